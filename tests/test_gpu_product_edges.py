"""8-bit products where their arithmetic could leave the formula."""

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
from oracle import product_oracle as P
from oracle import qsfm_oracle as O
from tests.test_gpu_products import SCALE_REL, built, check_quantised, clean, f64, i32, values  # noqa: F401

pytestmark = pytest.mark.gpu

LARGEST = float(np.finfo(np.float32).max)
BORDERS = (O.E4M3FN_TABLE[1:127] + O.E4M3FN_TABLE[:126]) / 2


def next_to(y):
    """y in fp32 with the numbers before and behind."""
    y = np.asarray(y, dtype=np.float32)
    return np.concatenate((np.nextafter(y, np.float32(0)), y, np.nextafter(y, np.float32(np.inf))))


def groups_of(top, y):
    """Groups of 128 whose first element is `top`, the others y in turn, signs mixed."""
    y = np.concatenate((y, np.zeros(-len(y) % 127, dtype=np.float32))).reshape(-1, 127)
    y = y * np.where(np.arange(127) % 3 == 0, -1, 1).astype(np.float32)
    return np.concatenate((np.full((len(y), 1), top, dtype=np.float32), y), 1)


def check_computed(codes, scale, y):
    """check_quantised() of elements that 64 bits round too: y and A are carried to 2^-48
    of themselves, and what is compared to 2^-47 (three sums of terms below 2^-23, each in
    fp32), so that within 2^-45 of a border, the fp64 roundings among it, either of its codes may be taken."""
    want, _ = P.quantize(y, False)
    a = np.abs(y).reshape(len(y), -1, 128).max(2).repeat(128, 1)
    near = np.abs(np.abs(y * 448 / a)[..., None] / BORDERS - 1) < 2.0 ** -45
    got = values(codes)
    free = near.any(2) & (got != want)
    lower, upper = O.E4M3FN_TABLE[near.argmax(2)], O.E4M3FN_TABLE[near.argmax(2) + 1]
    assert np.all((np.abs(got) == lower)[free] | (np.abs(got) == upper)[free])
    assert np.array_equal(np.signbit(got)[free], np.signbit(y)[free])
    assert np.array_equal(got[~free], want[~free])
    assert np.all(np.abs(f64(scale) / (a[:, ::128] / 448) - 1) <= SCALE_REL["gated"])


def still(n, dim, dev):
    """A table whose angles are all 0."""
    return torch.cat((torch.ones(n, dim // 2), torch.zeros(n, dim // 2)), 1).to(dev)


# ------------------------------------------------------------------ quantised rows
@pytest.mark.parametrize("top", [LARGEST, 1.75 * 2.0 ** 126, 1.3 * 2.0 ** 120, 1.9 * 2.0 ** 119, 2.0 ** 101, 2.0 ** 100], ids=str)
def test_borders_near_the_largest_numbers(cuda_device, top):
    top = float(np.float32(top))
    x = torch.from_numpy(groups_of(top, next_to(BORDERS * (top / 448)))).to(cuda_device)
    codes, scale = Q.quantize_rows(x)
    clean()
    check_quantised(codes, scale, f64(x), False, "plain")
    zero = torch.zeros(len(x), dtype=torch.int32, device=cuda_device)
    for inter in (True, False):
        codes, scale = Q.quantize_rows(x, positions=zero, cos_sin=still(1, 64, cuda_device), rope_offset=64, interleaved=inter)
        clean()
        check_quantised(codes, scale, f64(x), False, "rotate")
    small = x / 16
    for spread in (0.0, 0.25):  # of equal gates the borders of x are y's
        gate = 8 + spread * torch.rand(x.shape, generator=torch.Generator().manual_seed(1)).to(cuda_device)
        codes, scale = Q.quantize_rows(small, gate=gate)
        clean()
        check_computed(codes, scale, f64(small) * P.silu(f64(gate)))


@pytest.mark.parametrize("inter", [True, False])
def test_power_of_two_scales_of_tiny_turned_rows(cuda_device, inter):
    """The largest element is a little above 1.75 2^j, its fp32 value is not: the
    exponent is one more, and is clipped after that."""
    at = list(range(-126, -85, 3)) + [-94, -93, -92, -91, 3, 106, 107]
    x = torch.zeros(len(at), 128)
    other = 1 if inter else 32
    for i, j in enumerate(at):
        x[i, 64], x[i, 64 + other] = 1.75 * 2.0 ** j, -1.75 * 2.0 ** j
    table = torch.cat((torch.ones(1, 32), torch.full((1, 32), 2.0 ** -26)), 1)
    codes, scale = Q.quantize_rows(x.to(cuda_device), positions=i32([0] * len(at), cuda_device), cos_sin=table.to(cuda_device),
                                   rope_offset=64, interleaved=inter, pow2_scale=True)
    clean()
    cos, sin = f64(table[:, :32]).repeat(len(at), 0), f64(table[:, 32:]).repeat(len(at), 0)
    y = P.turn(f64(x)[:, None], cos, sin, 64, inter, False)[:, 0]
    assert np.all(y.max(1) > 1.75 * 2.0 ** np.array(at, dtype=float)) and np.all(y.astype(np.float32).max(1) == x.numpy().max(1))
    check_quantised(codes, scale, y, True, "rotate")


def test_groups_below_the_least_maximum(cuda_device):
    """Where all elements are below 1e-12, that is A: the number itself, not the fp32
    number next to it (one element in fp32 lies between the borders of the two)."""
    for top in (0.0, 9e-13, 2e-17, float(np.float32(1e-12)), float(np.nextafter(np.float32(1e-12), np.float32(1)))):
        y = next_to(BORDERS * (1e-12 / 448))
        x = torch.from_numpy(groups_of(top, y[y <= max(top, 9e-13)])).to(cuda_device)
        codes, scale = Q.quantize_rows(x)
        clean()
        check_quantised(codes, scale, f64(x), False, "plain")
        zero = torch.zeros(len(x), dtype=torch.int32, device=cuda_device)
        codes, scale = Q.quantize_rows(x, positions=zero, cos_sin=still(1, 128, cuda_device))
        clean()
        check_quantised(codes, scale, f64(x), False, "rotate")


#: cosine, sine, and a pair (a, b) of bf16 whose a cos - b sin lies within 2^-25 above 1,
#: and in fp32, within its roundings, below
ABOVE_ONE = [("0x1.6346e4p-3", "-0x1.f83cb8p-1", -0.00130462646484375, 1.015625),
             ("-0x1.433022p-2", "-0x1.e5d4a2p-1", 0.002471923828125, 1.0546875),
             ("-0x1.1cb348p-2", "0x1.ebd03cp-1", 0.0201416015625, -1.046875),
             ("-0x1.c867eap-2", "0x1.ca54c4p-1", 0.00018310546875, -1.1171875),
             ("-0x1.536868p-1", "0x1.7f55f6p-1", 0.000331878662109375, -1.3359375)]


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_turned_element_just_above_the_largest_other(cuda_device, dtype, inter):
    """An element that is not turned is 1; a turned one is larger by less than what its
    fp32 value may be off: elements on a border of A = 1 lie below the border of A."""
    x = torch.zeros(len(ABOVE_ONE), 128)
    table = torch.zeros(len(ABOVE_ONE), 64)
    # 448 y = m, the border of two codes: m a multiple of 7
    ties = [(m / 448) * 2.0 ** -e for m in (21.0, 28 / 2.0 ** 12) for e in range(0, 9)]
    for i, (c, s, a, b) in enumerate(ABOVE_ONE):
        x[i, 0] = 1.0
        x[i, 1:1 + len(ties)] = torch.tensor(ties)
        x[i, 64], x[i, 65 if inter else 96] = a, b
        table[i, 0], table[i, 32] = float.fromhex(c), float.fromhex(s)
    assert torch.equal(x.to(torch.bfloat16).float(), x)
    x = x.to(dtype)
    codes, scale = Q.quantize_rows(x.to(cuda_device), positions=i32(range(len(x)), cuda_device),
                                   cos_sin=table.to(cuda_device), rope_offset=64, interleaved=inter)
    clean()
    y = P.turn(f64(x)[:, None], *np.split(f64(table), 2, axis=1), 64, inter, False)[:, 0]
    if dtype != torch.float16:  # fp16 holds a less exactly
        assert np.all(y[:, 64] > 1) and np.all(y[:, 64] < 1 + 2.0 ** -25) and np.all(np.abs(y).max(1) == y[:, 64])
    check_quantised(codes, scale, y, False, "rotate")


def test_numbers_below_the_normal_ones_in_gated_rows(cuda_device):
    """silu of a small gate is half of it, and of a large one the gate: what is left of a
    gate or an element of few bits counts in full."""
    g = torch.Generator().manual_seed(5)
    large = 1e30 * torch.randn(40, 256, generator=g)
    small = torch.randint(1, 2000, (40, 256), generator=g) * 2.0 ** -149
    small[::2] *= -1
    small[1] = 2.0 ** -149
    small[2] = 1e-30
    for dtype in (torch.float32, torch.bfloat16):
        for x, gate in ((large, small), (small, 20 + large.abs())):
            x, gate = x.to(dtype), gate.to(dtype)
            for pow2 in (False, True):
                codes, scale = Q.quantize_rows(x.to(cuda_device), gate=gate.to(cuda_device), pow2_scale=pow2)
                clean()
                check_quantised(codes, scale, f64(x) * P.silu(f64(gate)), pow2, "gated")


def test_computed_elements_above_the_largest_number(cuda_device):
    """A turned or gated element that fp32 does not hold, and a term of a turned one, make
    their group NaN, and no other."""
    def check(codes, scale):
        clean()
        assert torch.isnan(scale).tolist() == [[True, False], [False, False]]
        assert torch.all(codes[0, :128] == 0x7F) and not torch.any(codes[0, 128:] & 0x7F == 0x7F) and not torch.any(codes[1] & 0x7F == 0x7F)

    for factor in (0.8, 1.2):  # a c - b s above the largest number; both terms above it and 0 left
        x = torch.randn(2, 256, generator=torch.Generator().manual_seed(2))
        x[0, 64], x[0, 65] = 3e38, -3e38 if factor < 1 else 3e38
        table = torch.cat((torch.ones(1, 32), torch.zeros(1, 32)), 1)
        table[0, 0] = table[0, 32] = factor
        zero = torch.zeros(2, dtype=torch.int32, device=cuda_device)
        for pow2 in (False, True):
            check(*Q.quantize_rows(x.to(cuda_device), positions=zero, cos_sin=table.to(cuda_device), rope_offset=64, pow2_scale=pow2))
    x, gate = torch.randn(2, 256, generator=torch.Generator().manual_seed(3)), torch.ones(2, 256)
    x[0, 7], gate[0, 7] = -3e38, 20.0
    for pow2 in (False, True):
        check(*Q.quantize_rows(x.to(cuda_device), gate=gate.to(cuda_device), pow2_scale=pow2))


# ------------------------------------------------------------------ products
#: rows, columns, K
SHAPES = [(40, 260, 1040), (5, 130, 128), (300, 10130, 144), (700, 10400, 272), (141, 4993, 3712), (41, 6172, 3488)]


def codes_of(v, dev):
    return v.float().to(torch.float8_e4m3fn).to(dev)


def scaled_by_fp32(a, sa, w, sw):
    """The definition in 64 bits, a block's two scales multiplied in fp32, with the sum of
    the terms' magnitudes."""
    out, mag = (torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64, device=a.device) for _ in range(2))
    rows = torch.arange(w.shape[0], device=a.device) // 128
    for b in range(-(-a.shape[1] // 128)):
        u, v = a[:, 128 * b:128 * b + 128].double(), w[:, 128 * b:128 * b + 128].double()
        s = (sa[:, b, None] * sw[rows, b][None]).double()
        out += s * (u @ v.t())
        mag += s.abs() * (u.abs() @ v.abs().t())
    return out, mag


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("ends", ["largest", "least"])
def test_scales_whose_product_is_at_the_ends_of_fp32(cuda_device, shape, ends):
    """Products of two scales from 2^125 to 2^127 of small codes, and from 2^-126 to 2^-124 of
    large ones, each scale far from the other: every result is a number of fp32."""
    dev, (m, n, k), g = cuda_device, shape, torch.Generator().manual_seed(shape[1])
    kb, nb = -(-k // 128), -(-n // 128)
    mant = lambda *s: 1 + torch.rand(*s, generator=g)  # noqa: E731
    if ends == "largest":  # codes up to 3 x 2^-9: a result is below K 9 2^-18 2^128
        a, w = (codes_of(torch.randint(-3, 4, s, generator=g) * 2.0 ** -9, dev) for s in ((m, k), (n, k)))
        sa, sw = mant(m, kb).to(dev) * 2.0 ** 119, mant(nb, kb).to(dev) * 2.0 ** 6
    else:  # codes of 256 and more: a block's sum is above 2^20, and so exact in fp32 terms
        a, w = (codes_of(256 + 32 * torch.randint(0, 7, s, generator=g), dev) for s in ((m, k), (n, k)))
        sa, sw = mant(m, kb).to(dev) * 2.0 ** -100, mant(nb, kb).to(dev) * 2.0 ** -26
    out = Q.scaled_matmul(a, sa, w, sw, out_dtype=torch.float32)
    clean()
    ref, mag = scaled_by_fp32(a, sa, w, sw)
    # a block's sum is exact (whole numbers of a unit, below 2^24 of them); a rounding each of the
    # product with the scales' and of the sum, for every block
    assert torch.isfinite(out).all() and torch.all((out.double() - ref).abs() <= (1 + kb) * 2.0 ** -24 * 1.01 * mag)


def test_scales_whose_product_leaves_fp32(cuda_device):
    """The product of a block's scales is fp32's: inf where it is larger than its largest
    number, rounded to its steps of 2^-149 where it is small."""
    dev = cuda_device
    a = torch.zeros(6, 256, device=dev)
    a[:, :128] = 1.0
    a[0, 1:128:2] = -1.0  # a sum of 0
    a[5, :128] = 448.0
    w = torch.ones(130, 256, device=dev)
    a, w = codes_of(a, dev), codes_of(w, dev)
    sa, sw = torch.ones(6, 2, device=dev), torch.ones(2, 2, device=dev)
    for first, second in ((2.0 ** 119, 2.0 ** 9), (2.0 ** -100, 2.0 ** -50), (1.3 * 2.0 ** -75, 1.7 * 2.0 ** -72), (-2.0 ** 100, 2.0 ** 100)):
        sa[:, 0], sw[:, 0] = first, second
        sa[1, 0] = 2.0 ** -3
        out = Q.scaled_matmul(a, sa, w, sw, out_dtype=torch.float32)
        clean()
        want = (sa[:, :1] * sw[0, 0]).double() * torch.tensor([0, 128, 128, 128, 128, 448 * 128], device=dev)[:, None].double()
        assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(want.float(), nan=7.0).expand(6, 130))
    assert torch.isnan(out[0]).all() and torch.isinf(out[2:]).all() and torch.isfinite(out[1]).all()
