"""GPU tests of the operators around the cache where a call is not the ordinary
one: tables with columns that hold no block, rows and queries that are not
finite, calls without tokens."""

import dataclasses

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
import workloads as W
from oracle import cache_oracle as C
from oracle import qsfm_oracle as O
from tests.harness import assert_parity, run_gpu
from tests.test_gpu_cache_operators import FORMATS, cache_values, i32, new_cache, table_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from compressed_mla_attention_gb300 import build

    build.build()
    Q.lib()


# ------------------------------------------------------------------ block tables
def table_step(dev, state, prev, lens, rows, ratio=1, num_blocks=None, inplace=True):
    """One call and the oracle's from the same state; returns the fault word and the slots."""
    table, free, count = state
    nb = len(free) if num_blocks is None else num_blocks
    ref = C.block_tables(table, prev, lens, free, count, ratio, rows, num_blocks=nb)
    t, f, n = i32(table, dev), i32(free, dev), i32([count], dev)
    out = None if inplace else i32([-99], dev)
    cu, res = i32(np.zeros(len(lens) + 1), dev), i32(np.zeros(len(lens)), dev)
    slots, pos = Q.update_block_tables(t, i32(prev, dev), i32(lens, dev), f, n, max_rows=rows, cu_rows=cu, residual=res,
                                       free_count_out=out, cmp_ratio=ratio, num_blocks=nb)
    torch.cuda.synchronize()
    fault = Q.device_status()
    assert np.array_equal(t.cpu().numpy(), ref[0])
    assert int((n if inplace else out)[0]) == ref[2]
    assert np.array_equal(f.cpu().numpy(), ref[1])
    for got, want in ((slots, ref[3]), (pos, ref[4]), (cu, ref[5]), (res, ref[6])):
        assert np.array_equal(got.cpu().numpy(), want)
    state[:] = ref[:3]
    return fault, ref[3]


def test_a_short_pool_recovers_every_block(cuda_device):
    """Two blocks for four wanted; both requests end; a new one takes a block."""
    state = [np.full((2, 4), -1, dtype=np.int32), np.array([5, 6, -7, -7], dtype=np.int32), 2]
    fault, _ = table_step(cuda_device, state, [0, 0], [300, 128], 428, num_blocks=16)
    assert fault == Q.FAULT_BLOCK_POOL and state[0].tolist() == [[6, 5, -1, -1], [-1] * 4]
    fault, _ = table_step(cuda_device, state, [300, 128], [0, 0], 1, num_blocks=16)
    assert fault == 0 and state[2] == 2 and state[1][:2].tolist() == [6, 5]
    fault, slots = table_step(cuda_device, state, [0, 0], [0, 100], 100, num_blocks=16)
    assert fault == 0 and slots.tolist() == [5 * 128 + i for i in range(100)]
    # a request that goes on in a column without a block is reported, and its rows are not stored
    state = [np.array([[6, -1]], dtype=np.int32), np.array([1, 2], dtype=np.int32), 2]
    fault, slots = table_step(cuda_device, state, [200], [201], 1, num_blocks=16)
    assert fault == Q.FAULT_ORI_BLOCK_ID and slots.tolist() == [-1]


def test_columns_behind_a_window_hold_no_block(cuda_device):
    state = [np.array([[-1, -1, -1, 7], [-1, 3, -1, -1]], dtype=np.int32), np.array([0, 1] + [-7] * 6, dtype=np.int32), 2]
    fault, slots = table_step(cuda_device, state, [500, 256], [0, 257], 1)
    assert fault == 0 and state[2] == 2 and slots.tolist() == [7 * 128]
    # one table row of 1000 columns, the last two blocks of it live; and a request that takes both
    table = np.full((2, 1000), -1, dtype=np.int32)
    table[0, 998:] = 4, 2
    state = [table, np.array([0, -7, -7, -7, -7], dtype=np.int32), 1]
    fault, _ = table_step(cuda_device, state, [128000, 0], [0, 300], 300)
    assert fault == 0 and state[0][1, :3].tolist() == [2, 4, 0] and state[2] == 0


def test_foreign_ids_are_reported_and_not_passed_on(cuda_device):
    for bad in (99, -2, 2 ** 31 - 1):
        state = [np.array([[3, bad], [-1, -1]], dtype=np.int32), np.array([1, 0, 0, 0], dtype=np.int32), 1]
        fault, _ = table_step(cuda_device, state, [256, 0], [0, 0], 1, num_blocks=16)
        assert fault == Q.FAULT_ORI_BLOCK_ID and state[2] == 2 and state[1][:2].tolist() == [1, 3]
    for bad in (99, -1):  # on the free list
        state = [np.full((1, 2), -1, dtype=np.int32), np.array([1, bad], dtype=np.int32), 2]
        fault, _ = table_step(cuda_device, state, [0], [256], 256, num_blocks=16)
        assert fault == Q.FAULT_ORI_BLOCK_ID and state[0].tolist() == [[-1, 1]] and state[2] == 0


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("name,batch,width,ratio,new_hi", [
    ("few", 3, 9, 1, 400), ("one CTA", 40, 30, 4, 700), ("wide rows", 12, 700, 1, 3000), ("many CTAs", 300, 40, 1, 2500),
    ("many requests", 3000, 5, 1, 150)])
def test_tables_with_holes_match_the_oracle(cuda_device, name, batch, width, ratio, new_hi, inplace):
    """Held columns of which some hold no block, or an id outside the pool."""
    r = np.random.RandomState(len(name))
    cap = width * 128 * ratio
    prev = r.randint(0, cap + 1, batch)
    lens = np.minimum(prev + r.randint(0, new_hi + 1, batch), cap)
    shrink = r.rand(batch) < 0.4
    lens[shrink] = (prev[shrink] * r.rand(shrink.sum())).astype(int) * r.randint(0, 2, shrink.sum())
    held = -(-(prev // ratio) // 128)
    pool = int(held.sum()) + batch
    perm, at = r.permutation(pool), 0
    table = r.randint(-5, pool, (batch, width)).astype(np.int32)
    for b in range(batch):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
        kind = r.randint(4)
        if kind == 1:  # behind a window
            table[b, :max(0, held[b] - 2)] = -1
        elif kind == 2:  # a short pool's, here and there
            table[b, :held[b]][r.rand(held[b]) < 0.5] = -1
        elif kind == 3 and held[b] and batch < 300:
            table[b, r.randint(held[b])] = r.choice([pool, -3])
    free = np.concatenate([perm[at:], np.full(at, -7)]).astype(np.int32)
    rows = int(np.maximum(lens // ratio - prev // ratio, 0).sum()) + 5
    table_step(cuda_device, [table, free, pool - at], prev, lens, rows, ratio=ratio, inplace=inplace)


def test_a_history_of_short_pools_loses_no_block(cuda_device):
    """Forty steps of a pool too small for its requests: after each, every
    block is in one table or on the list, once."""
    r = np.random.RandomState(7)
    batch, width, pool = 6, 8, 17
    state = [np.full((batch, width), -1, dtype=np.int32), r.permutation(pool).astype(np.int32), pool]
    prev, short = np.zeros(batch, dtype=int), 0
    for _ in range(40):
        lens = np.minimum(prev + r.randint(0, 300, batch), width * 128)
        lens[r.rand(batch) < 0.25] = 0
        fault, _ = table_step(cuda_device, state, prev, lens, int(np.maximum(lens - prev, 0).sum()) + 1)
        short += fault & Q.FAULT_BLOCK_POOL != 0
        used = [v for b, n in enumerate(lens) for v in state[0][b, :-(-n // 128)].tolist() if v >= 0]
        assert sorted(used + state[1][:state[2]].tolist()) == list(range(pool))
        prev = lens
    assert short > 5


# ------------------------------------------------------------------ rows that are not finite
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_broken_row_is_stored_as_one(cuda_device, fmt, dtype, norm):
    """NaN and infinities in key rows of every format: without the norm the
    element's scale group holds NaN, codes and scale (a bf16 element is as it is); with it a
    NaN breaks its whole row, and of a row with an infinity, whose norm divides by
    infinity, its group is NaN and the others are zeros. The rows beside are as
    without it."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(7, 512, generator=g)
    bad = [(1, 70, "nan"), (1, 300, "-inf"), (2, 511, "inf"), (4, 64, "nan"), (4, 500, "nan"), (5, 130, "-inf")]
    for row, at, v in bad:
        x[row, at] = float(v)
    dev, slots = cuda_device, torch.arange(7, dtype=torch.int32, device=cuda_device)
    stored = []
    for rows in (x, torch.where(torch.isfinite(x), x, 0.0)):
        cache, scale = new_cache(fmt, 1, dev)
        out = torch.empty(7, 512, dtype=torch.bfloat16, device=dev)
        Q.norm_rope_store(None, rows.to(dtype).to(dev), kv_cache=cache, kv_scale=scale, kv_out=out, slot_map=slots, norm_kv=norm)
        torch.cuda.synchronize()
        assert Q.device_status() == 0
        stored.append((cache_values(cache, scale, range(7)), out.double().cpu().numpy(),
                       O.pool_bytes(cache.cpu()).reshape(128, -1)[:7]))
    (held, out, raw), (clean, clean_out, _) = stored
    size = {"packed384": 16, "packed640": 64, "fp8_fp32_scales": 64, "bf16": 1}[fmt]
    broken = np.zeros((7, 512), dtype=bool)
    for row, at, v in bad:
        # the first 64 elements of a packed row are bf16 of their own
        broken[row, at // size * size:at // size * size + size] = True
    whole = [1, 4] if norm else []  # a NaN in the sum
    broken[whole] = True
    if fmt == "bf16" and not norm:
        assert np.array_equal(held, x.to(torch.bfloat16).double().numpy(), equal_nan=True)
        assert np.array_equal(out, held, equal_nan=True)
        return
    assert np.isnan(held[broken]).all() and np.isnan(out[broken]).all()
    zero = np.zeros_like(broken)
    if norm:
        zero[[2, 5]] = ~broken[[2, 5]]
    assert (held[zero] == 0).all() and (out[zero] == 0).all()
    rest = ~broken & ~zero
    assert np.array_equal(held[rest], clean[rest]) and np.array_equal(out[rest], clean_out[rest])
    if fmt == "fp8_fp32_scales":  # the attention must not read a number there, whatever it makes of the scale
        assert (raw[broken] & 0x7F == 0x7F).all()


# ------------------------------------------------------------------ calls without tokens
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_step_without_tokens(cuda_device, fmt):
    """Empty tensors, whose pointers are null: nothing is launched, nothing written."""
    dev = cuda_device
    none = torch.empty(0, dtype=torch.int32, device=dev)
    q, kv = (torch.empty(0, *s, dtype=torch.bfloat16, device=dev) for s in ((64, 512), (512,)))
    w = torch.ones(512, device=dev)
    at = dict(positions=none, cos_sin=table_of(10, 64, dev))
    cache, scale = new_cache(fmt, 1, dev)
    before = cache.clone()
    store = dict(kv_cache=cache, kv_scale=scale, slot_map=none, kv_weight=w)
    for got in (Q.norm_rope_store(q, kv, q_weight=w, kv_out=torch.empty(0, 512, dtype=torch.bfloat16, device=dev), **store, **at),
                Q.norm_rope_store(q, q_weight=w, **at), Q.norm_rope_store(q, q_out=torch.empty_like(q))):
        assert got.shape == (0, 64, 512)
    assert Q.norm_rope_store(None, kv, **store, **at) is None
    assert Q.norm_rope_store(None, kv[:, None], **store) is None
    torch.cuda.synchronize()
    assert Q.device_status() == 0 and torch.equal(cache, before)


# ------------------------------------------------------------------ attention over what is not finite
def nan_row(w, fmt, row):
    """w with a NaN in cmp row `row` of request 0."""
    kv = w.cmp_kv.clone()
    at = kv.view(-1, kv.shape[-1])[int(w.cmp_block_table[0, row // 128]) * 128 + row % 128]
    if fmt == "packed384":
        at[352 + 9] = 0x7F  # one scale
    elif fmt == "packed640":
        at[576 + 2] = 0xFF
    elif fmt == "fp8_fp32_scales":
        at[130] = 0x7F
    else:
        at[130] = float("nan")
    return dataclasses.replace(w, cmp_kv=kv)


# CTAs: units split over them (more than one part holds the row's unit), and not
@pytest.mark.parametrize("ctas", [16, 7, 1])
@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_rows_and_queries_show_in_every_plan(cuda_device, fmt, ctas):
    """A NaN in one row of one part makes its token's output and lse NaN, and a
    NaN in one head's query those of its head, however the tiles are cut; the
    rest is what it is without them."""
    w = W.build(f"nan {fmt}", layout="BSND", q_lens=[1, 1], s2=[70000, 50000], cmp_ratio=128, mode="HCA", kv_format=fmt, seed=5)
    o_ref, l_ref = O.reference(w, [0, 1])
    for row in (0, 200, 545):
        out, lse = run_gpu(nan_row(w, fmt, row), cuda_device, num_ctas=ctas, lse=True)
        assert np.isnan(out[0]).all() and np.isnan(lse[0]).all()
        out[0], lse[0] = o_ref[0], l_ref[0]
        assert_parity(out, lse, w, [0, 1], o_ref, l_ref)
    q = w.q.clone()
    q[0, 5, 17] = float("nan")
    if fmt != "fp8_fp32_scales":  # there one scale serves the 64 heads of a token: the other token alone is compared
        q[1, 63, 511] = float("nan")
    out, lse = run_gpu(dataclasses.replace(w, q=q), cuda_device, num_ctas=ctas, lse=True)
    for t, h in torch.isnan(q).any(2).nonzero().tolist():
        assert np.isnan(out[t, h]).all() and np.isnan(lse[t, h])
        out[t, h], lse[t, h] = o_ref[t, h], l_ref[t, h]
    tokens = [1] if fmt == "fp8_fp32_scales" else [0, 1]
    assert_parity(out, lse, w, tokens, o_ref[tokens], l_ref[tokens])


@pytest.mark.parametrize("ctas", [1, 5])
def test_a_first_tile_of_minus_infinities(cuda_device, ctas):
    """The window of each token is its own row, whose first element is -inf and
    meets a positive query: weight 0. The other rows' scores are all far below
    zero, some -350 against the first tile's, and count as they are."""
    w = W.build("4-bit minus inf", layout="TND", q_lens=[1, 1, 1], s2=[900, 700, 800], cmp_ratio=4, mode="CSA", k2=150,
                kv_format="packed384", seed=21, sinks=False, ori_win_left=0)
    q, ori, cmp = w.q.clone(), w.ori_kv.clone(), w.cmp_kv.clone()
    q[:, :, 0], q[:, :, 1] = 1.0, -8000.0
    first = torch.tensor([float("-inf"), 1.0], dtype=torch.bfloat16).view(torch.uint8)
    ori.view(-1, 384)[:, :4] = first
    cmp.view(-1, 384)[:, :4] = torch.tensor([0.5, 1.0], dtype=torch.bfloat16).view(torch.uint8)
    w = dataclasses.replace(w, q=q, ori_kv=ori, cmp_kv=cmp)
    out, lse = run_gpu(w, cuda_device, num_ctas=ctas, lse=True)
    for t in range(3):
        k = O.token_kv(w, t, t, 0)[1:]  # without the first row
        x = w.softmax_scale * (O.q_fp64(w, t) @ k.T)
        top = x.max(1, keepdims=True)
        p = np.exp(x - top)
        want = (p / p.sum(1, keepdims=True)) @ k
        # fp32 accumulation of 512 products of up to 8000: 512 roundings of 2^-24 of sum |q k|
        dx = 512 * 2.0 ** -24 * w.softmax_scale * (np.abs(O.q_fp64(w, t)) @ np.abs(k).T).max(1) + 2.0 ** -20
        bound = (2 * dx[:, None] + 2.0 ** -8 + len(k) * 2.0 ** -24) * ((p / p.sum(1, keepdims=True)) @ np.abs(k)) + 2.0 ** -8 * np.abs(want)
        assert (np.abs(out[t] - want) <= 1.01 * bound)[:, 1:].all()  # of element 0 the formula has 0 * -inf
        l = np.log(p.sum(1)) + top[:, 0]
        assert (np.abs(lse[t] - l) <= dx + len(k) * 2.0 ** -24 + 2.0 ** -20 * np.abs(l)).all()


@pytest.mark.parametrize("ctas", [64, 3])
@pytest.mark.parametrize("fmt", FORMATS)
def test_a_broken_row_shows_in_the_tokens_that_attend_it(cuda_device, fmt, ctas):
    """Stored by one call, read by the next: a NaN in a key row reaches the
    tokens whose window holds the row and no others."""
    dev, n, window, at = cuda_device, 40, 8, 20
    g = torch.Generator().manual_seed(9)
    x, q = torch.randn(n, 512, generator=g), torch.randn(n, 64, 512, generator=g).to(torch.bfloat16).to(dev)
    order = torch.arange(n, dtype=torch.int32, device=dev)
    runs = []
    for value in (0.5, float("nan")):
        x[at, 100] = value
        cache, scale = new_cache(fmt, 1, dev)
        Q.norm_rope_store(None, x.to(dev), kv_cache=cache, kv_scale=scale, slot_map=order, positions=order,
                          cos_sin=table_of(n, 64, dev))
        out, lse = Q.quant_sparse_flash_mla(q, cache, scale, i32([[0]], dev), i32([n], dev), layout="TND",
                                            cu_seqlens_q=i32([0, n], dev), ori_win_left=window - 1, num_ctas=ctas,
                                            return_softmax_lse=True)
        torch.cuda.synchronize()
        assert Q.device_status() == 0
        runs.append((out.float().cpu().numpy(), lse.cpu().numpy(), np.abs(cache_values(cache, scale, range(n)))))
    (clean, clean_lse, rows), (out, lse, _) = runs
    hit = np.zeros(n, dtype=bool)
    hit[at:at + window] = True
    assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    # the others: the same rows, the weights rounded to 8 bits against another reference, the output to 8 bits
    assert np.abs(out[~hit] - clean[~hit]).max() <= 4 * 2.0 ** -8 * rows.max()
    # 512 products in fp32, twice: less than 2^-13 of sum |q k| / sqrt(512) (below 40 for these rows)
    assert np.abs(lse[~hit] - clean_lse[~hit]).max() <= 40 * 2.0 ** -13


@pytest.mark.parametrize("ctas", [0, 1, 7])
def test_a_call_repeats_its_bits(cuda_device, ctas):
    """The same call gives the same bits, split units among them."""
    w = W.build("4-bit repeat", layout="TND", q_lens=[3, 1, 6], s2=[5000, 129, 20000], cmp_ratio=4, mode="CSA", k2=512,
                kv_format="packed384", seed=31)
    out, lse = run_gpu(w, cuda_device, num_ctas=ctas, lse=True)
    for _ in range(20):
        again, again_lse = run_gpu(w, cuda_device, num_ctas=ctas, lse=True)
        assert np.array_equal(out, again) and np.array_equal(lse, again_lse)
