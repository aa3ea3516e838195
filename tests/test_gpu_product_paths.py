"""Products through each of their kernels and splits, alone and by group of rows:
every case asks which of them it gets, so that a changed choice shows here and
not as a kernel that nothing tests."""

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
from tests.test_gpu_products import built, clean, i32, whole_numbers  # noqa: F401

pytestmark = pytest.mark.gpu

PAIR, WIDE, SMALL = (256, 256), (128, 256), (128, 128)  # rows and columns of a tile


def widened(t, scale, k):
    return t.double() * scale.double().repeat_interleave(128, -1)[..., :k]


def exact(a, sa, w, sw):
    """The product in 64 bits, exact for whole_numbers(): the terms' magnitudes add up
    to less than 2^24 of the smallest unit, 2^-4, so that fp32 sums are exact too."""
    n, k = w.shape
    left, right = widened(a, sa, k), widened(w, sw.repeat_interleave(128, 0)[:n], k)
    assert float((left.abs() @ right.abs().t()).max()) * 16 < 2 ** 24
    return (left @ right.t()).float()


#: kernel, parts, rows, columns, K, the sizes none of the tiles' multiples (seven parts of
#: 128 x 256: eight, of which as many clusters run at a time, are never longer)
SPLITS = [(PAIR, 1, 700, 10400, 272), (PAIR, 2, 134, 6035, 5920), (PAIR, 3, 141, 4993, 3712), (PAIR, 4, 132, 3132, 5152),
          (WIDE, 1, 265, 9960, 144), (WIDE, 2, 41, 12085, 6208), (WIDE, 3, 41, 11457, 2736), (WIDE, 4, 42, 7330, 4416),
          (WIDE, 5, 41, 6172, 3488), (WIDE, 6, 42, 5238, 6080), (WIDE, 8, 41, 3705, 10800),
          (SMALL, 1, 300, 2000, 272), (SMALL, 2, 46, 6051, 1744), (SMALL, 3, 41, 5015, 1344), (SMALL, 4, 44, 100, 1344),
          (SMALL, 5, 44, 93, 1248), (SMALL, 6, 47, 97, 1472), (SMALL, 7, 41, 105, 1744), (SMALL, 8, 200, 250, 2000)]


@pytest.mark.parametrize("case", SPLITS, ids=str)
def test_every_kernel_and_split_is_exact(cuda_device, case):
    tile, parts, m, n, k = case
    a, sa, w, sw = whole_numbers(m, n, k, 1, torch.Generator().manual_seed(m + n + k), cuda_device)
    ref = exact(a, sa, w[0], sw[0])
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        wide = torch.full((m, n + 24), 9.0, dtype=dtype, device=cuda_device)  # gaps before and behind each row
        for out in (wide[:, 8:8 + n], wide[:, 9:9 + n]):  # aligned to 16 bytes, and not
            block = Q.make_matmul_params(a=a, a_scale=sa, w=w[0], w_scale=sw[0], out=out)
            assert Q.debug_matmul_plan(block) == (*tile, parts)
            out.fill_(7.0)
            Q.matmul(block)
            clean()
            assert torch.equal(out, ref.to(dtype))
            out.fill_(9.0)
            assert torch.all(wide == 9)


def ragged(sizes, first, behind):
    """(cu_rows, rows) of groups of these sizes, with rows before the first and behind the last."""
    cu = [first + int(v) for v in np.cumsum([0] + sizes)]
    return cu, cu[-1] + behind


#: group sizes around the tiles' rows, empty ones, single rows
AROUND = [0, 1, 255, 256, 257, 0, 0, 513, 127, 128, 129, 700, 31, 33]
GROUPED = {
    "pairs": (PAIR, *ragged(AROUND, 5, 9), 3000, 272),
    "pairs, some large": (PAIR, *ragged([1500, 0, 3, 1900, 900, 1, 0, 990], 0, 0), 1096, 400),
    "pairs, one group of rows": (PAIR, *ragged([0, 0, 2499, 0, 1, 0], 0, 0), 4104, 144),
    "wide, few rows": (WIDE, *ragged([i % 3 * (i % 5) for i in range(52)], 2, 3), 1100, 272),
    "wide": (WIDE, *ragged([16, 0, 33, 1, 128, 0, 129, 64, 257, 31, 90, 0, 65, 127, 300, 2, 0, 260, 95, 32, 5, 111, 250, 0], 7, 11), 1032, 528),
    "wide, around the tiles": (WIDE, *ragged([v // 2 for v in AROUND] * 3, 0, 40), 2056, 144),
    "small": (SMALL, *ragged([3, 0, 128, 129, 1, 40], 1, 2), 392, 656),
}


def grouped_case(name, dev, seed=0):
    tile, cu, m, n, k = GROUPED[name]
    a, sa, w, sw = whole_numbers(m, n, k, len(cu) - 1, torch.Generator().manual_seed(m + seed), dev)
    return tile, cu, m, n, a, sa, w, sw


def grouped_block(tile, a, sa, w, sw, cu, out):
    block = Q.make_matmul_params(a=a, a_scale=sa, w=w, w_scale=sw, cu_rows=cu, out=out)
    assert Q.debug_matmul_plan(block) == (*tile, 1)
    return block


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("name", sorted(GROUPED))
def test_grouped_kernels_are_exact(cuda_device, name, dtype):
    dev = cuda_device
    tile, cu, m, n, a, sa, w, sw = grouped_case(name, dev)
    out = torch.full((m, n), 7.0, dtype=dtype, device=dev)
    Q.matmul(grouped_block(tile, a, sa, w, sw, i32(cu, dev), out))
    clean()
    want = torch.full((m, n), 7.0, dtype=dtype, device=dev)
    for g in range(len(cu) - 1):
        at = slice(cu[g], cu[g + 1])
        if at.stop > at.start:
            want[at] = exact(a[at], sa[at], w[g], sw[g]).to(dtype)
    assert torch.equal(out, want)


@pytest.mark.parametrize("name", ["pairs", "wide", "wide, few rows"])
def test_rows_of_other_groups_do_not_reach_a_group(cuda_device, name):
    """Rows of every other group are NaN, by their codes or by their scales, and so are
    those outside all groups; a group's matrix that is NaN is that group's alone."""
    dev = cuda_device
    tile, cu, m, n, a, sa, w, sw = grouped_case(name, dev, 1)
    one = torch.full((m, n), 7.0, device=dev)
    Q.matmul(grouped_block(tile, a, sa, w, sw, i32(cu, dev), one))
    bad = torch.zeros(m, dtype=torch.bool, device=dev)
    a.view(torch.uint8)[:cu[0]] = 0x7F
    sa[cu[-1]:] = float("nan")
    for g in range(0, len(cu) - 1, 2):
        at = slice(cu[g], cu[g + 1])
        bad[at] = True
        if g % 6 == 0:
            a.view(torch.uint8)[at] = 0x7F
        elif g % 6 == 2:
            sa[at] = float("nan")
        else:
            w.view(torch.uint8)[g] = 0x7F
    two = torch.full((m, n), 7.0, device=dev)
    Q.matmul(grouped_block(tile, a, sa, w, sw, i32(cu, dev), two))
    clean()
    assert torch.isnan(two[bad]).all() and torch.equal(two[~bad], one[~bad])


@pytest.mark.parametrize("name", ["pairs", "wide"])
def test_bad_group_rows_are_cut_and_reported(cuda_device, name):
    """Entries that decrease or leave the rows: what is left of each group is computed,
    where only one group has a row its result is that group's."""
    dev = cuda_device
    tile, cu, m, n, a, sa, w, sw = grouped_case(name, dev, 2)
    for change in ({3: m + 1000}, {0: -4}, {4: cu[4] + 300, 6: 10}, {len(cu) - 1: 2 ** 31 - 1}):
        odd = list(cu)
        for i, v in change.items():
            odd[i] = v
        out = torch.full((m, n), 7.0, device=dev)
        Q.matmul(grouped_block(tile, a, sa, w, sw, i32(odd, dev), out))
        torch.cuda.synchronize()
        assert Q.device_status() == Q.FAULT_GROUP_ROWS
        owners = torch.zeros(m, dtype=torch.int64, device=dev)
        for g in range(len(odd) - 1):
            owners[min(max(odd[g], 0), m):max(min(odd[g + 1], m), 0)] += 1
        for g in range(len(odd) - 1):
            lo, hi = min(max(odd[g], 0), m), min(max(odd[g + 1], 0), m)
            if hi > lo:
                alone = owners[lo:hi] == 1
                assert torch.equal(out[lo:hi][alone], exact(a[lo:hi], sa[lo:hi], w[g], sw[g])[alone])
        assert torch.all(out[owners == 0] == 7)


@pytest.mark.parametrize("case", [c for c in SPLITS if c[1] > 1 and c[0] != SMALL], ids=str)
def test_split_products_repeat_bit_for_bit(cuda_device, case):
    tile, parts, m, n, k = case
    g = torch.Generator().manual_seed(k)
    a, sa = Q.quantize_rows(torch.randn(m, k, generator=g).to(cuda_device))
    w, _ = Q.quantize_rows(torch.randn(n, k, generator=g).to(cuda_device))
    sw = (0.5 + torch.rand(-(-n // 128), -(-k // 128), generator=g)).to(cuda_device)
    outs = [torch.full((m, n), float("nan"), device=cuda_device) for _ in range(4)]
    for out in outs:
        Q.matmul(Q.make_matmul_params(a=a, a_scale=sa, w=w, w_scale=sw, out=out))
    clean()
    assert all(torch.equal(outs[0], out) for out in outs[1:])


#: kernel, parts, rows, columns, K, columns before and behind: rows that begin at 16 bytes and
#: end between two
RAGGED = [(PAIR, 1, 700, 10403, 272, 8, 5), (PAIR, 1, 144, 11237, 48, 0, 3), (SMALL, 1, 82, 3, 288, 8, 5), (SMALL, 1, 213, 3251, 240, 4, 1),
          (SMALL, 1, 300, 1999, 272, 16, 1), (WIDE, 1, 265, 9961, 144, 8, 7), (SMALL, 4, 44, 99, 1344, 8, 5), (PAIR, 4, 132, 3131, 5152, 8, 5)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("case", RAGGED, ids=str)
def test_columns_beside_the_output_stay(cuda_device, case, dtype):
    tile, parts, m, n, k, before, behind = case
    a, sa, w, sw = whole_numbers(m, n, k, 1, torch.Generator().manual_seed(n), cuda_device)
    whole = torch.full((m, before + n + behind), float("nan"), dtype=dtype, device=cuda_device)
    assert whole.stride(0) * whole.element_size() % 16 == 0 and n * whole.element_size() % 16 != 0
    out = whole[:, before:before + n]
    block = Q.make_matmul_params(a=a, a_scale=sa, w=w[0], w_scale=sw[0], out=out)
    assert Q.debug_matmul_plan(block) == (*tile, parts)
    Q.matmul(block)
    clean()
    assert torch.equal(out, exact(a, sa, w[0], sw[0]).to(dtype))
    assert torch.isnan(whole[:, :before]).all() and torch.isnan(whole[:, before + n:]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_columns_beside_grouped_outputs_stay(cuda_device, dtype):
    dev = cuda_device
    cu, m = ragged([1500, 0, 3, 1900, 900, 1, 0, 990], 5, 9)
    n, k = 1099, 400
    a, sa, w, sw = whole_numbers(m, n, k, len(cu) - 1, torch.Generator().manual_seed(1), dev)
    whole = torch.full((m, n + 13), 7.0, dtype=dtype, device=dev)
    Q.matmul(grouped_block(PAIR, a, sa, w, sw, i32(cu, dev), whole[:, 8:8 + n]))
    clean()
    want = torch.full_like(whole, 7.0)
    for g in range(len(cu) - 1):
        at = slice(cu[g], cu[g + 1])
        if at.stop > at.start:
            want[at, 8:8 + n] = exact(a[at], sa[at], w[g], sw[g]).to(dtype)
    assert torch.equal(whole, want)
