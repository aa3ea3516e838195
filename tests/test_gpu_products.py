"""GPU parity of the 8-bit products (rows quantised per 128 elements, scaled
products, products by group of rows) with the fp64 oracle, each alone and in
the order a step runs them around the indexer and the attention."""

import threading

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
from oracle import product_oracle as P
from oracle import qsfm_oracle as O

pytestmark = pytest.mark.gpu

#: Scales against the formula's, relative: their own rounding (1 unit of 2^-24),
#: and those of a computed A: rotated 3, gated 9 + 1.25 |gate| (exp's argument
#: 1.25 |gate|, its result 4, 1 + e 1, the reciprocal 2, two products), where
#: the gates of the largest elements are below 12.
SCALE_REL = {"plain": 2.0 ** -24, "rotate": 4 * 2.0 ** -24, "gated": 25 * 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    from compressed_mla_attention_gb300 import build

    build.build()
    Q.lib()


def clean():
    torch.cuda.synchronize()
    assert Q.device_status() == 0


def i32(v, dev):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).to(dev)


def values(codes):
    return O.E4M3FN_TABLE[codes.view(torch.uint8).cpu().numpy().astype(int)]


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ quantised rows
def table_of(n, dim, dev):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().to(dev)


def check_quantised(codes, scale, y, pow2, kind):
    """Codes equal to the formula's in 64 bits, scales within their roundings."""
    want, s = P.quantize(y, pow2)
    got = values(codes).reshape(y.shape)
    assert np.array_equal(got, want, equal_nan=True), f"{(got != want).sum()} of {got.size} codes differ"
    got = f64(scale)
    assert np.array_equal(np.isnan(got), np.isnan(s))
    live = ~np.isnan(s)
    if pow2:
        assert np.array_equal(got[live], s[live])
    else:
        assert np.all(np.abs(got[live] / s[live] - 1) <= SCALE_REL[kind])


DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (rows, heads, elements of a head)
PLAIN = [(1, 1, 16), (1, 1, 4096), (3, 1, 144), (7, 1, 1008), (5, 64, 128), (257, 3, 256), (1000, 1, 5120), (2, 128, 512)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("shape", PLAIN, ids=str)
def test_quantized_rows_are_the_formulas(cuda_device, shape, dtype, pow2):
    g = torch.Generator().manual_seed(sum(shape))
    x = (torch.randn(*shape, generator=g) * torch.exp(torch.randn(shape[0], 1, 1, generator=g))).to(dtype).to(cuda_device)
    x[0, 0, 5] *= 30
    codes, scale = Q.quantize_rows(x, pow2_scale=pow2)
    clean()
    assert codes.shape == x.shape and scale.shape == (shape[0], -(-shape[1] * shape[2] // 128))
    check_quantised(codes, scale, f64(x).reshape(shape[0], -1), pow2, "plain")


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_quantized_borders(cuda_device, dtype):
    """Elements on the borders of two codes, and next to them: every quotient of
    short significands, with largest elements whose scale is not a power of two."""
    top = torch.arange(128, 256, dtype=torch.float64)
    x = torch.arange(128, 256, dtype=torch.float64)[None] * 2.0 ** -torch.arange(0, 20)[:, None, None]
    x = torch.minimum(x, top[None, :, None]).clone()  # [20, 128 tops, 128]
    x[:, :, 0] = top
    x = x.reshape(-1, 128)
    if dtype == torch.float32:  # with the neighbours in fp32 of each
        up = x.float() * (1 + 2.0 ** -23)
        x = torch.cat((x.float(), up, x.float() * (1 - 2.0 ** -24))).double()
    x = (x * 2.0 ** -7).to(dtype)
    for pow2 in (False, True):
        codes, scale = Q.quantize_rows(x.to(cuda_device), pow2_scale=pow2)
        clean()
        check_quantised(codes, scale, f64(x), pow2, "plain")


def test_quantized_extremes(cuda_device):
    """Zeros, denormals, the largest values, infinities and NaN, each a matter of
    its own group."""
    x = torch.randn(16, 512, generator=torch.Generator().manual_seed(3))
    x[0] = 0
    x[1] = -0.0
    x[2, :128] = 1e-30
    x[3, :128] = 3e-39
    x[4, 128:256] = 3.3e38
    x[5, 7] = float("inf")
    x[6, 300] = float("-inf")
    x[7, 511] = float("nan")
    x[8] = float("nan")
    x[9, ::3] = 3e38
    for dtype in (torch.float32, torch.bfloat16):
        for pow2 in (False, True):
            y = x.to(dtype)
            codes, scale = Q.quantize_rows(y.to(cuda_device), pow2_scale=pow2)
            clean()
            check_quantised(codes, scale, f64(y), pow2, "plain")
    assert torch.isnan(scale[5, 0]) and torch.isfinite(scale[5, 1:]).all()


ROTATE = [dict(heads=64, dim=128, offset=64), dict(heads=64, dim=512, offset=448, inter=False, inverse=True),
          dict(heads=2, dim=256, offset=0, inverse=True), dict(heads=3, dim=128, rope=128, inter=False),
          dict(heads=1, dim=256, rope=32, offset=96), dict(heads=1, dim=208, rope=64, offset=128, inter=False),
          dict(heads=5, dim=128, rope=32, offset=96, inter=False)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("case", ROTATE, ids=str)
def test_rotated_rows_are_the_formulas(cuda_device, case, dtype, pow2):
    o = dict(dict(rope=64, offset=0, inter=True, inverse=False), **case)
    n = 37
    g = torch.Generator().manual_seed(o["dim"])
    x = torch.randn(n, o["heads"], o["dim"], generator=g).to(dtype)
    pos = torch.randint(0, 4000, (n,), generator=g)
    pos[0], pos[1] = 0, 3999
    x[2] = 0
    x[2, 0, o["offset"]] = 1.0  # alone in its group: A is its turned pair's
    table = table_of(4000, o["rope"], cuda_device)
    codes, scale = Q.quantize_rows(x.to(cuda_device), positions=i32(pos, cuda_device), cos_sin=table,
                                   rope_offset=o["offset"], interleaved=o["inter"], inverse=o["inverse"], pow2_scale=pow2)
    clean()
    cos, sin = np.split(f64(table)[pos.numpy()], 2, axis=1)
    y = P.turn(f64(x), cos, sin, o["offset"], o["inter"], o["inverse"])
    check_quantised(codes, scale, y.reshape(n, -1), pow2, "rotate")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("shape", [(1, 1, 2048), (301, 1, 1424), (9, 4, 384)], ids=str)
def test_gated_rows_are_the_formulas(cuda_device, shape, dtype, pow2):
    """Gate and up projection as the two halves of one product's rows."""
    t, h, d = shape
    g = torch.Generator().manual_seed(d)
    both = (2 * torch.randn(t, h, 2 * d, generator=g)).to(dtype)
    both[0, 0, :8] = torch.tensor([-30.0, 30, 0, -0.0, -86, 80, 1e-4, -1e-4])
    both = both.to(cuda_device)
    gate, x = both[:, :, :d], both[:, :, d:]
    if h == 1:
        gate, x = gate[:, 0], x[:, 0]
    codes, scale = Q.quantize_rows(x, gate=gate, pow2_scale=pow2)
    clean()
    y = f64(x) * P.silu(f64(gate))
    check_quantised(codes, scale, y.reshape(t, -1), pow2, "gated")


def test_gate_that_is_not_finite(cuda_device):
    x, gate = torch.ones(4, 256), torch.ones(4, 256)
    gate[0, 0], gate[1, 0], gate[2, 200], x[3, 0] = float("inf"), float("-inf"), float("nan"), float("nan")
    gate[:, 5] = -200.0
    codes, scale = Q.quantize_rows(x.to(cuda_device), gate=gate.to(cuda_device))
    clean()
    assert torch.isnan(scale).tolist() == [[True, False], [True, False], [False, True], [True, False]]
    assert codes[2, 5].item() in (0, 0x80)


def test_gathered_and_padded_rows(cuda_device):
    dev, g = cuda_device, torch.Generator().manual_seed(8)
    x = torch.randn(50, 1040, generator=g).to(torch.bfloat16)
    index = torch.randint(0, 50, (333,), generator=g)
    index[::7] = -1
    codes = torch.full((333, 1040), 0x5A, dtype=torch.uint8, device=dev)
    scale = torch.full((333, 9), 7.0, device=dev)
    Q.quantize_rows(x.to(dev), row_index=i32(index, dev), codes=codes, scale=scale)
    clean()
    live = (index >= 0).numpy()
    check_quantised(codes[live], scale[live], f64(x)[index.numpy()[live]], False, "plain")
    assert torch.all(codes[~live] == 0x5A) and torch.all(scale[~live] == 7)
    # an index past the source rows, a position past the table: reported, not read
    c, s = Q.quantize_rows(x.to(dev), row_index=i32([3, 50, 2 ** 31 - 1, 4], dev))
    torch.cuda.synchronize()
    assert Q.device_status() == Q.FAULT_ROW_INDEX
    assert not c[1:3].any() and not s[1:3].any()
    check_quantised(c[[0, 3]], s[[0, 3]], f64(x)[[3, 4]], False, "plain")
    c, s = Q.quantize_rows(x[:4].to(dev), positions=i32([-1, 9, 10, 0], dev), cos_sin=table_of(10, 64, dev))
    torch.cuda.synchronize()
    assert Q.device_status() == Q.FAULT_POSITION
    assert not c[[0, 2]].any() and s[[1, 3]].all() and not s[[0, 2]].any()


def test_strided_rows_and_empty_ones(cuda_device):
    dev, g = cuda_device, torch.Generator().manual_seed(9)
    big = torch.randn(6, 9, 640, generator=g).to(torch.float16).to(dev)
    for x in (big[::2, :, 128:512], big.transpose(0, 1)[:, :, :256], big[:, 4, 16:160], big[:, :, :128].expand(6, 9, 128)):
        codes, scale = Q.quantize_rows(x)
        clean()
        check_quantised(codes, scale, f64(x).reshape(x.shape[0], -1), False, "plain")
    one = torch.randn(1, 256, generator=g).to(dev)
    codes, scale = Q.quantize_rows(one.expand(5, 256))  # a broadcast row: stride 0
    clean()
    assert torch.equal(codes, codes[:1].expand(5, 256))
    codes, scale = Q.quantize_rows(big[:0])
    assert codes.shape == (0, 9, 640) and scale.shape == (0, 45)
    codes, scale = Q.quantize_rows(big[0], row_index=torch.zeros(0, dtype=torch.int32, device=dev))
    assert codes.shape == (0, 640)


def test_one_row_of_any_stride(cuda_device):
    x = torch.randn(3, 261, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(cuda_device)
    x = x[:1, :256]  # 522 bytes to the next row, which there is not
    codes, scale = Q.quantize_rows(x, gate=x)
    again, _ = Q.quantize_rows(x.clone(), gate=x.clone())
    assert torch.equal(codes, again)
    out = Q.scaled_matmul(codes, scale, codes, scale)
    clean()
    assert out.shape == (1, 1)


def test_rows_past_2_to_the_31_elements(cuda_device):
    """Offsets that do not fit 31 bits: input, codes and a product's output."""
    dev, n = cuda_device, 66000
    if torch.cuda.mem_get_info(dev)[0] < 30 << 30:
        pytest.skip("not enough memory")
    x = torch.empty(n, 32768, dtype=torch.bfloat16, device=dev)
    x[:-3] = 1.0
    x[-3:] = torch.randn(3, 32768, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(dev)
    codes, scale = Q.quantize_rows(x)
    last, last_scale = Q.quantize_rows(x[-3:].clone())
    assert torch.equal(codes[-3:], last) and torch.equal(scale[-3:], last_scale)
    turned = dict(cos_sin=table_of(100, 64, dev), rope_offset=64, inverse=True)
    at = torch.arange(n, dtype=torch.int32, device=dev) % 100
    Q.quantize_rows(x.view(n, 64, 512), positions=at, codes=codes, scale=scale, **turned)
    last, last_scale = Q.quantize_rows(x[-3:].clone().view(3, 64, 512), positions=at[-3:].clone(), **turned)
    assert torch.equal(codes[-3:], last.view(3, -1)) and torch.equal(scale[-3:], last_scale)
    del x
    a, sa = codes[:, :128], scale[:, :1]  # strided rows
    w, sw = last.view(-1, 128)[:256].repeat(128, 1), torch.ones(256, 1, device=dev)
    out = Q.scaled_matmul(a, sa, w, sw)
    small = Q.scaled_matmul(a[-3:].clone(), sa[-3:].clone(), w, sw)
    clean()
    assert out.numel() > 2 ** 31 and torch.equal(out[-3:], small)


def test_index_into_no_rows(cuda_device):
    c, s = Q.quantize_rows(torch.empty(0, 256, device=cuda_device), row_index=i32([0, -1], cuda_device))
    torch.cuda.synchronize()
    assert Q.device_status() == Q.FAULT_ROW_INDEX and not c.any() and not s.any()


# ------------------------------------------------------------------ products
def whole_numbers(m, n, k, groups, g, dev):
    """Codes of whole numbers within -8 .. 8 and scales that are powers of two: every
    product and every sum below 2^24 units is exact in fp32, in any order. (128
    products within 64 sum up to 2^13; with scales of 2^-2 .. 2^1 each, blocks
    of 2^-4 .. 2^2 times that add up to at most ceil(K / 128) 2^19 of the
    smallest unit: 2^24 for 32 blocks in the worst case.)"""
    e4m3 = lambda *s: torch.randint(-8, 9, s, generator=g).float().to(torch.float8_e4m3fn).to(dev)  # noqa: E731
    power = lambda *s: (2.0 ** torch.randint(-2, 2, s, generator=g)).to(dev)  # noqa: E731
    kb, nb = -(-k // 128), -(-n // 128)
    return e4m3(m, k), power(m, kb), e4m3(groups, n, k), power(groups, nb, kb)


def real_numbers(m, n, k, groups, g, dev):
    a, sa = Q.quantize_rows(torch.randn(m, k, generator=g).to(dev))
    w, _ = Q.quantize_rows(torch.randn(groups * n, k, generator=g).to(dev))
    sw = (0.5 + torch.rand(groups, -(-n // 128), -(-k // 128), generator=g)).to(dev)
    return a, sa, w.view(groups, n, k), sw


def exact_product(a, sa, w, sw):
    """The products in 64 bits with what their sums' roundings scale with."""
    return P.product(values(a), f64(sa), values(w), f64(sw))


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def tolerance(ref, mag, kb, dtype):
    """Half a step of the output; of the fp32 sums: the two scales' product and the
    block's product with it (2 units of 2^-24), one unit for each block added, and
    for a block's 128 products in fp32 accumulators that may cut instead of round
    (2 units for each of them), all relative to the terms' magnitudes."""
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0  # half the smallest step of fp16
    return HALF_STEP[dtype] * np.abs(ref) + (2 + kb + 256) * 2.0 ** -24 * mag * 1.01 + tiny


#: rows, columns, K: each row tile of the kernel with one less, one more; odd sizes
SHAPES = [(1, 128, 128), (1, 1, 16), (1, 4096, 2048), (2, 129, 144), (15, 100, 272), (16, 128, 1024), (17, 200, 256), (31, 384, 400),
          (33, 130, 128), (64, 512, 1040), (65, 127, 2064), (127, 640, 384), (128, 256, 512), (129, 257, 640), (200, 96, 4096),
          (256, 384, 256), (257, 512, 128), (500, 1000, 1296), (777, 1000, 2064), (1500, 260, 784)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_of_whole_numbers_are_exact(cuda_device, shape, dtype):
    m, n, k = shape
    a, sa, w, sw = whole_numbers(m, n, k, 1, torch.Generator().manual_seed(m + n + k), cuda_device)
    out = Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=dtype)
    clean()
    ref, _ = exact_product(a, sa, w[0], sw[0])
    assert out.dtype == dtype and torch.equal(out.cpu(), torch.from_numpy(ref).to(torch.float32).to(dtype))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_products_match_the_oracle(cuda_device, shape):
    m, n, k = shape
    a, sa, w, sw = real_numbers(m, n, k, 1, torch.Generator().manual_seed(m + n + k), cuda_device)
    ref, mag = exact_product(a, sa, w[0], sw[0])
    for dtype in DTYPES:
        out = Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=dtype)
        clean()
        assert np.all(np.abs(f64(out) - ref) <= tolerance(ref, mag, sa.shape[1], dtype))


#: few rows over a long K (split over many parts, odd numbers of them among them), pairs of
#: row tiles, many row tiles; columns that end inside a tile
LARGE = [(1, 4096, 32768), (48, 2048, 16384), (16, 8192, 1024), (130, 4096, 8192), (256, 4096, 16384), (200, 2000, 4112),
         (300, 640, 16400), (640, 2000, 4112), (2100, 1800, 1040), (5000, 520, 272), (1500, 1500, 4096), (9000, 264, 144)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large_products_of_whole_numbers_are_exact(cuda_device, shape, dtype):
    """Against torch's product in 64 bits, which is exact for these. The sums of the
    terms' magnitudes stay below 2^24 of the smallest unit, 2^-4, so that fp32 sums
    are exact in any order."""
    m, n, k = shape
    a, sa, w, sw = whole_numbers(m, n, k, 1, torch.Generator().manual_seed(m + n + k), cuda_device)
    wide = torch.full((m, n + 8), 9.0, dtype=dtype, device=cuda_device)  # rows with a gap behind them
    Q.scaled_matmul(a, sa, w[0], sw[0], out=wide[:, :n])
    clean()
    left = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    right = w[0].double() * sw[0].double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    assert float((left.abs() @ right.abs().t()).max()) * 16 < 2 ** 24
    assert torch.equal(wide[:, :n], (left @ right.t()).float().to(dtype))
    assert torch.all(wide[:, n:] == 9)


def test_products_repeat_bit_for_bit(cuda_device):
    for m, n, k in ((3, 512, 4096), (200, 384, 8192), (600, 512, 1024)):
        a, sa, w, sw = real_numbers(m, n, k, 1, torch.Generator().manual_seed(m), cuda_device)
        one = Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(one, Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=torch.float32))
    clean()


@pytest.mark.parametrize("m", [3, 40, 300])
def test_products_of_strided_tensors(cuda_device, m):
    """Rows inside wider rows, scales by column, an output between other columns;
    what surrounds them stays."""
    dev, g = cuda_device, torch.Generator().manual_seed(m)
    n, k = 200, 272
    a, sa, w, sw = whole_numbers(m, n, k, 1, g, dev)
    ref, _ = exact_product(a, sa, w[0], sw[0])
    wide_a = torch.full((m, 512), 0x7F, dtype=torch.uint8, device=dev)  # NaN codes
    wide_a[:, 128:128 + k] = a.view(torch.uint8)
    wide_w = torch.full((n, 320), 0x7F, dtype=torch.uint8, device=dev)
    wide_w[:, 16:16 + k] = w[0].view(torch.uint8)
    by_column = torch.full((sa.shape[1], m + 5), float("nan"), device=dev)
    by_column[:, :m] = sa.t()
    out = torch.full((m, n + 7), 5.0, dtype=torch.bfloat16, device=dev)
    got = Q.scaled_matmul(wide_a[:, 128:128 + k], by_column[:, :m].t(), wide_w[:, 16:16 + k], sw[0], out=out[:, 3:3 + n])
    clean()
    assert got.data_ptr() == out[:, 3:].data_ptr()
    assert torch.equal(out[:, 3:3 + n].cpu(), torch.from_numpy(ref).float().to(torch.bfloat16))
    assert torch.all(out[:, :3] == 5) and torch.all(out[:, 3 + n:] == 5)


@pytest.mark.parametrize("m", [5, 100, 400])
def test_products_of_what_is_not_finite(cuda_device, m):
    """A NaN in a row's code or scale is a matter of that row, one in a matrix's row
    of that column; scales of inf and 0 give what the sum gives."""
    dev, g = cuda_device, torch.Generator().manual_seed(m)
    a, sa, w, sw = whole_numbers(m, 300, 512, 1, g, dev)
    clean_out = Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=torch.float32)
    a.view(torch.uint8)[2, 200] = 0x7F
    sa[3, 1] = float("nan")
    w.view(torch.uint8)[0, 130, 17] = 0xFF
    out = Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=torch.float32)
    clean()
    bad = torch.zeros(m, 300, dtype=torch.bool)
    bad[2:4] = True
    bad[:, 130] = True
    assert torch.equal(torch.isnan(out).cpu(), bad)
    assert torch.equal(out.cpu()[~bad], clean_out.cpu()[~bad])
    sw[0, 2] = 0.0
    sw[0, 1, 0] = float("inf")
    out = Q.scaled_matmul(a, sa, w[0], sw[0], out_dtype=torch.float32)
    clean()
    assert torch.all(out[4:, 256:] == 0) and not torch.isfinite(out[4:, 128:256]).any()


def test_products_of_no_rows(cuda_device):
    a, sa, w, sw = whole_numbers(1, 128, 128, 1, torch.Generator().manual_seed(0), cuda_device)
    assert Q.scaled_matmul(a[:0], sa[:0], w[0], sw[0]).shape == (0, 128)
    e = i32([0, 0], cuda_device)
    assert Q.grouped_scaled_matmul(a[:0], sa[:0], w, sw, e).shape == (0, 128)
    out = Q.grouped_scaled_matmul(a, sa, w, sw, e)
    clean()
    assert not out.any()


# ------------------------------------------------------------------ products by group
GROUPS = {
    "one group": ([0, 40], 200, 272, 40),
    "each a row": (list(range(0, 34)), 130, 256, 33),
    "empty ones": ([0, 0, 5, 5, 5, 70, 70], 256, 400, 70),
    "all empty": ([0] * 9, 128, 128, 12),
    "before and behind": ([7, 20, 20, 150], 384, 128, 163),
    "one large": ([0, 2, 3, 700, 701], 250, 528, 701),
    "around the tiles": ([0, 15, 31, 48, 111, 175, 240, 367, 495, 624, 879, 1135, 1392], 136, 144, 1400),
    "many": (list(np.cumsum([0] + [(7 * i) % 5 for i in range(300)])), 64, 128, 600),
    "the most": (list(np.minimum(np.arange(1025) // 3, 200)), 32, 16, 200),
    "pairs": ([0, 256, 511, 1100, 1101, 1900], 392, 656, 1930),
    "pairs of many": ([3] + [3 + 300 * (i + 1) - 7 * i for i in range(12)], 128, 400, 3700),
}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped_products_of_whole_numbers_are_exact(cuda_device, name, dtype):
    cu, n, k, m = GROUPS[name]
    dev = cuda_device
    a, sa, w, sw = whole_numbers(m, n, k, len(cu) - 1, torch.Generator().manual_seed(m), dev)
    out = torch.full((m, n), 7.0, dtype=dtype, device=dev)
    Q.grouped_scaled_matmul(a, sa, w, sw, i32(cu, dev), out=out)
    clean()
    ref, _ = P.grouped(values(a), f64(sa), values(w), f64(sw), cu, np.full((m, n), 7.0))
    assert torch.equal(out.cpu(), torch.from_numpy(ref).float().to(dtype))


def test_grouped_products_match_the_oracle(cuda_device):
    cu, n, k, m = [0, 300, 300, 310, 520], 384, 1040, 530
    a, sa, w, sw = real_numbers(m, n, k, 4, torch.Generator().manual_seed(4), cuda_device)
    ref, mag = P.grouped(values(a), f64(sa), values(w), f64(sw), cu, np.zeros((m, n)))
    for dtype in DTYPES:
        out = Q.grouped_scaled_matmul(a, sa, w, sw, i32(cu, cuda_device), out_dtype=dtype)
        clean()
        assert np.all(np.abs(f64(out) - ref) <= tolerance(ref, mag, sa.shape[1], dtype))
        assert not out[520:].any()


def test_rows_of_other_groups_do_not_reach_a_group(cuda_device):
    """NaN rows of one group, and rows outside all groups, lie in the tiles of others."""
    dev = cuda_device
    a, sa, w, sw = whole_numbers(90, 128, 256, 3, torch.Generator().manual_seed(6), dev)
    cu = i32([0, 20, 50, 80], dev)
    one = Q.grouped_scaled_matmul(a, sa, w, sw, cu)
    a.view(torch.uint8)[20:50] = 0x7F
    sa[80:] = float("nan")
    two = Q.grouped_scaled_matmul(a, sa, w, sw, cu)
    clean()
    assert torch.equal(one[:20], two[:20]) and torch.equal(one[50:], two[50:]) and torch.isnan(two[20:50]).all()


def test_bad_group_rows_are_cut_and_reported(cuda_device):
    dev = cuda_device
    a, sa, w, sw = whole_numbers(60, 130, 256, 4, torch.Generator().manual_seed(7), dev)
    for cu, live in (([0, 20, 10, 10, 60], {0: (0, 20), 3: (10, 60)}), ([-5, 20, 30, 50, 90], {0: (0, 20), 1: (20, 30), 2: (30, 50), 3: (50, 60)}),
                     ([70, 80, 80, 2 ** 31 - 1, -2 ** 31], {})):
        out = torch.full((60, 130), 7.0, device=dev)
        Q.grouped_scaled_matmul(a, sa, w, sw, i32(cu, dev), out=out)
        torch.cuda.synchronize()
        assert Q.device_status() == Q.FAULT_GROUP_ROWS
        rows = np.zeros(60, dtype=int)
        for lo, hi in live.values():
            rows[lo:hi] += 1
        for e, (lo, hi) in live.items():
            ref, _ = exact_product(a[lo:hi], sa[lo:hi], w[e], sw[e])
            alone = rows[lo:hi] == 1
            assert np.array_equal(f64(out)[lo:hi][alone], ref[alone])
        assert torch.all(out[torch.from_numpy(rows == 0).to(dev)] == 7)


# ------------------------------------------------------------------ streams, graphs, steps
def test_products_as_the_first_call_of_a_thread(cuda_device):
    """Host threads that have not used CUDA before, each on a stream of its own, at
    once; the first call of the process is the main thread's."""
    dev = cuda_device
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(300, 1024, generator=gen).to(dev)
    w = torch.randint(0, 120, (512, 1024), generator=gen, dtype=torch.uint8).to(dev)
    sw = torch.rand(4, 8, generator=gen).to(dev)
    codes, scale = Q.quantize_rows(x)
    want = [Q.scaled_matmul(codes[:m], scale[:m], w, sw) for m in (1, 300)]
    torch.cuda.synchronize(dev)
    outs = [[torch.zeros_like(v) for v in want] for _ in range(4)]
    streams = [torch.cuda.Stream(dev) for _ in outs]
    errors = []

    def run(out, stream):
        try:
            params = [
                Q.make_matmul_params(a=codes[: v.shape[0]], a_scale=scale[: v.shape[0]], w=w, w_scale=sw, out=v)
                for v in out
            ]
            for _ in range(20):
                for p in params:
                    Q.matmul(p, stream=stream)
        except Exception as e:  # (an exception of a thread would be lost)
            errors.append(e)

    threads = [threading.Thread(target=run, args=a) for a in zip(outs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize(dev)
    assert not errors, errors
    assert all(torch.equal(g, v) for out in outs for g, v in zip(out, want))
    assert Q.device_status() == 0


def test_other_streams_and_captured_calls(cuda_device):
    """Calls on streams of their own, two at once; a captured step replayed on
    other inputs in the same buffers, between eager calls."""
    dev, g = cuda_device, torch.Generator().manual_seed(12)
    x = torch.randn(40, 1024, generator=g).to(torch.bfloat16).to(dev)
    w, _ = Q.quantize_rows(torch.randn(512, 1024, generator=g).to(dev))
    sw = torch.rand(4, 8, generator=g).to(dev)

    def step(rows):
        codes, scale = Q.quantize_rows(rows)
        return Q.scaled_matmul(codes, scale, w, sw)

    want, other = step(x), step(-2 * x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for s, rows in zip(streams * 2, (x, -2 * x) * 2):
        s.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(s):
            got.append(step(rows))
    own = torch.cuda.Stream(dev)
    own.wait_stream(torch.cuda.current_stream(dev))
    codes, scale = Q.quantize_rows(x, stream=own)
    got.append(Q.scaled_matmul(codes, scale, w, sw, stream=own))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want if i % 2 == 0 else other) for i, v in enumerate(got))

    buf = x.clone()
    codes, scale, out = (torch.zeros(40, 1024, dtype=torch.uint8, device=dev), torch.zeros(40, 8, device=dev),
                         torch.zeros(40, 512, dtype=torch.bfloat16, device=dev))
    blocks = (Q.make_quantize_params(x=buf, codes=codes, scale=scale),
              Q.make_matmul_params(a=codes, a_scale=scale, w=w, w_scale=sw, out=out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.quantize(blocks[0])
        Q.matmul(blocks[1])
    for rows, ref in ((x, want), (-2 * x, other), (x, want)):
        buf.copy_(rows)
        graph.replay()
        assert torch.equal(step(rows), ref)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    clean()


def test_step_of_the_indexer_and_the_projections(cuda_device):
    """A decode step as a model runs it: hidden rows quantised and projected to the
    indexer's queries, those rotated and quantised into what lightning_indexer takes,
    the attention over the rows that it picks, its output turned back, quantised and
    projected, and the experts' products; each against its oracle on what it got."""
    dev, g = cuda_device, torch.Generator().manual_seed(20)
    n, hidden, heads = 6, 1024, 64
    x = torch.randn(n, hidden, generator=g).to(torch.bfloat16).to(dev)

    def matrix(rows, k):
        codes, _ = Q.quantize_rows(torch.randn(rows, k, generator=g).to(dev))
        return codes, (0.5 + torch.rand(-(-rows // 128), -(-k // 128), generator=g)).to(dev) / 448 / k ** 0.5

    def project(codes, scale, m):
        out = Q.scaled_matmul(codes, scale, *m)
        ref, mag = exact_product(codes, scale, *m)
        assert np.all(np.abs(f64(out) - ref) <= tolerance(ref, mag, scale.shape[1], torch.bfloat16))
        return out

    hx, hs = Q.quantize_rows(x)
    check_quantised(hx, hs, f64(x), False, "plain")
    table = table_of(5000, 64, dev)
    s2, pos = i32([900, 2000], dev), i32([897, 898, 899, 1997, 1998, 1999], dev)
    iq = project(hx, hs, matrix(heads * 128, hidden)).view(n, heads, 128)
    query, query_scale = Q.quantize_rows(iq, positions=pos, cos_sin=table, rope_offset=64)
    cos, sin = np.split(f64(table)[pos.cpu().numpy()], 2, axis=1)
    check_quantised(query, query_scale, P.turn(f64(iq), cos, sin, 64, True, False).reshape(n, -1), False, "rotate")
    # keys of the indexer: a head of 128 elements, one scale each, paged
    keys = torch.randn(8 * 128, 128, generator=g).to(dev)
    key, key_scale = Q.quantize_rows(keys)
    tab = torch.randperm(8, generator=g).int().view(2, 4).to(dev)
    idx, _ = Q.lightning_indexer(query.view(2, 3, heads, 128), query_scale, torch.rand(n, heads, generator=g).to(dev),
                                 key.view(8, 128, 1, 128), key_scale.view(8, 128, 1), tab, i32([225, 500], dev), layout="BSND",
                                 topk=64, mask_mode=3, cmp_ratio=4)
    q = project(hx, hs, matrix(heads * 512, hidden)).view(n, heads, 512)
    kv = torch.randn(40, 128, 1, 512, generator=g).to(torch.bfloat16).to(dev)
    ori_tab = torch.arange(32, dtype=torch.int32, device=dev).view(2, 16)
    cmp_tab = 32 + torch.arange(8, dtype=torch.int32, device=dev).view(2, 4)
    o, _ = Q.quant_sparse_flash_mla(q.view(2, 3, heads, 512), kv, None, ori_tab, s2, cmp_kv=kv, cmp_block_table=cmp_tab,
                                    cmp_sparse_indices=idx.view(2, 3, 1, 64), cmp_ratio=4)
    o = o.view(n, heads, 512)
    codes, scale = Q.quantize_rows(o, positions=pos, cos_sin=table, rope_offset=0, inverse=True)
    check_quantised(codes, scale, P.turn(f64(o), cos, sin, 0, True, True).reshape(n, -1), False, "rotate")
    y = project(codes.view(n, -1), scale, matrix(hidden, heads * 512))
    # two of four experts for each token, rows in the experts' order, gathered as they are quantised
    choice = torch.stack([torch.randperm(4, generator=g)[:2] for _ in range(n)]).flatten()
    order = torch.argsort(choice, stable=True)
    cu = i32([0] + torch.bincount(choice, minlength=4).cumsum(0).tolist(), dev)
    index = i32(order // 2, dev)
    ey, es = Q.quantize_rows(y, row_index=index)
    check_quantised(ey, es, f64(y)[(order // 2).numpy()], False, "plain")
    up = [matrix(512, hidden) for _ in range(4)]
    w, ws = torch.stack([m[0] for m in up]), torch.stack([m[1] for m in up])
    both = Q.grouped_scaled_matmul(ey, es, w, ws, cu)
    ref, mag = P.grouped(values(ey), f64(es), values(w), f64(ws), cu.tolist(), np.zeros((2 * n, 512)))
    assert np.all(np.abs(f64(both) - ref) <= tolerance(ref, mag, 8, torch.bfloat16))
    ay, as_ = Q.quantize_rows(both[:, 256:], gate=both[:, :256])
    check_quantised(ay, as_, f64(both[:, 256:]) * P.silu(f64(both[:, :256])), False, "gated")
    clean()
