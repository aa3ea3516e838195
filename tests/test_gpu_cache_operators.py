"""GPU parity of the operators around the cache (block tables, norm + rotation
+ store of rows, attention over 4-bit rows) with the fp64 oracles, each alone
and in the order a serving step runs them."""

import dataclasses

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
import workloads as W
from oracle import cache_oracle as C
from oracle import qsfm_oracle as O
from tests.harness import LSE_ATOL, assert_parity, run_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from compressed_mla_attention_gb300 import build

    build.build()
    Q.lib()


def i32(v, dev):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).to(dev)


# ------------------------------------------------------------------ block tables
def table_case(seed, batch, width, ratio, prev_hi, new_hi, end=0.2, begin=0.2, pool=None):
    r = np.random.RandomState(seed)
    prev = r.randint(0, prev_hi + 1, batch)
    prev[r.rand(batch) < begin] = 0
    lens = prev + r.randint(0, new_hi + 1, batch)
    shrink = r.rand(batch) < 0.2
    lens[shrink] = prev[shrink] // 2
    lens[r.rand(batch) < end] = 0
    held = -(-(prev // ratio) // 128)
    pool = pool if pool is not None else int(held.sum() + batch * width)
    perm = r.permutation(pool)
    table = r.randint(-5, 1000, (batch, width))  # behind the held columns: whatever was there
    at = 0
    for b in range(batch):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.concatenate([perm[at:], np.full(at, -7)])
    return table, prev, lens, free, pool - at


TABLES = {
    "one": dict(batch=1, width=4, ratio=1, prev_hi=300, new_hi=100),
    "decode": dict(batch=128, width=40, ratio=1, prev_hi=4000, new_hi=2),
    "compressed": dict(batch=70, width=16, ratio=4, prev_hi=6000, new_hi=900),
    "ratio 128": dict(batch=33, width=3, ratio=128, prev_hi=30000, new_hi=5000),
    "chunks": dict(batch=100, width=60, ratio=1, prev_hi=5000, new_hi=1500),
    "many": dict(batch=5000, width=6, ratio=1, prev_hi=400, new_hi=200),
    "fresh": dict(batch=17, width=30, ratio=1, prev_hi=0, new_hi=3500),
}


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("name", sorted(TABLES))
def test_block_tables_match_the_oracle(cuda_device, name, inplace):
    kw = TABLES[name]
    table, prev, lens, free, count = table_case(len(name), **kw)
    rows = int(np.maximum(lens // kw["ratio"] - prev // kw["ratio"], 0).sum()) + 5
    ref = C.block_tables(table, prev, lens, free, count, kw["ratio"], rows)
    dev = cuda_device
    t, f, n = i32(table, dev), i32(free, dev), i32([count], dev)
    out = None if inplace else i32([-99], dev)
    cu, res, slots = i32(np.zeros(len(lens) + 1), dev), i32(np.zeros(len(lens)), dev), i32(np.full(rows + 3, 77), dev)
    s, pos = Q.update_block_tables(t, i32(prev, dev), i32(lens, dev), f, n, slot_map=slots[:rows],
                                   positions=torch.empty(rows, dtype=torch.int32, device=dev), cu_rows=cu,
                                   residual=res, free_count_out=out, cmp_ratio=kw["ratio"])
    torch.cuda.synchronize()
    assert Q.device_status() == 0
    assert np.array_equal(t.cpu().numpy(), ref[0])
    assert int((n if inplace else out)[0]) == ref[2] and (inplace or int(n[0]) == count)
    assert np.array_equal(f.cpu().numpy(), ref[1])
    for got, want in ((s, ref[3]), (pos, ref[4]), (cu, ref[5]), (res, ref[6])):
        assert np.array_equal(got.cpu().numpy(), want)
    assert slots[rows:].tolist() == [77] * 3  # behind the map: left as it was


def test_block_tables_without_a_request(cuda_device):
    e = torch.empty(0, dtype=torch.int32, device=cuda_device)
    n = i32([3], cuda_device)
    s, pos = Q.update_block_tables(e.view(0, 4), e, e, i32([0, 1, 2], cuda_device), n, max_rows=700)
    assert set(s.tolist()) == {-1} and set(pos.tolist()) == {-1} and int(n[0]) == 3


def test_block_tables_report_bad_data(cuda_device):
    dev = cuda_device
    # two blocks are free and five wanted: in order, then none
    t, n = i32(np.full((2, 4), 9), dev), i32([2], dev)
    s, _ = Q.update_block_tables(t, i32([0, 0], dev), i32([300, 256], dev), i32([5, 6, 0, 0], dev), n, max_rows=556,
                                 num_blocks=16)
    s = s.cpu().numpy()
    assert Q.device_status() == Q.FAULT_BLOCK_POOL
    assert t.tolist() == [[6, 5, -1, 9], [-1, -1, 9, 9]] and int(n[0]) == 0
    assert s[0] == 6 * 128 and s[255] == 5 * 128 + 127 and set(s[256:].tolist()) == {-1}
    # more rows than the map holds, a request wider than its table row, ids outside the pool
    t, n = i32(np.full((1, 2), -1), dev), i32([4], dev)
    s, pos = Q.update_block_tables(t, i32([0], dev), i32([1000], dev), i32([0, 1, 2, 99], dev), n, max_rows=300,
                                   num_blocks=16)
    s = s.cpu().numpy()
    assert Q.device_status() == Q.FAULT_SLOT | Q.FAULT_ORI_TABLE_COL | Q.FAULT_ORI_BLOCK_ID
    assert t.tolist() == [[-1, 2]] and int(n[0]) == 2
    assert set(s[:128].tolist()) == {-1} and s[128] == 256 and set(s[256:].tolist()) == {-1}
    # the list cannot take more than it holds; a count past it is cut
    t, n = i32([[1, 2]], dev), i32([7], dev)
    f = i32([3, 4, 5], dev)
    Q.update_block_tables(t, i32([256], dev), i32([0], dev), f, n, max_rows=1, num_blocks=16)
    torch.cuda.synchronize()
    assert Q.device_status() == Q.FAULT_BLOCK_POOL and int(n[0]) == 3 and f.tolist() == [3, 4, 5]


def test_block_tables_of_absurd_lengths_stay_in_bounds(cuda_device):
    """2^31 - 1 tokens in each of 5000 requests: the row counts stop at the
    largest int instead of wrapping."""
    dev, big = cuda_device, 2 ** 31 - 1
    t, n = i32(np.zeros((5000, 2)), dev), i32([4], dev)
    s, pos = Q.update_block_tables(t, i32(np.zeros(5000), dev), i32(np.full(5000, big), dev), i32([0, 1, 2, 3], dev), n,
                                   max_rows=600)
    s, pos = s.cpu().numpy(), pos.cpu().numpy()
    assert Q.device_status() == Q.FAULT_SLOT | Q.FAULT_ORI_TABLE_COL | Q.FAULT_BLOCK_POOL
    assert np.array_equal(pos, np.arange(600)) and s[0] == 3 * 128 and s[255] == 2 * 128 + 127 and s[256] == -1
    s, _ = Q.update_block_tables(t, i32([-5] * 5000, dev), i32([-1] * 5000, dev), i32([0, 1, 2, 3], dev), n, max_rows=9)
    torch.cuda.synchronize()
    assert Q.device_status() == 0 and set(s.tolist()) == {-1}


# ------------------------------------------------------------------ rows
FORMATS = ["packed384", "packed640", "fp8_fp32_scales", "bf16"]


def new_cache(fmt, blocks, dev, fill=0xAB):
    if fmt == "bf16":
        return torch.full((blocks, 128, 1, 512), 3.0, dtype=torch.bfloat16, device=dev), None
    width = {"packed384": 384, "packed640": 640, "fp8_fp32_scales": 512}[fmt]
    scale = torch.full((blocks, 128, 1, 8), 5.0, device=dev) if fmt == "fp8_fp32_scales" else None
    return torch.full((blocks, 128, 1, width), fill, dtype=torch.uint8, device=dev), scale


def cache_values(cache, scale, slots):
    """K~ fp64 of the rows at slots, by the attention's oracle."""
    flat = O.pool_bytes(cache.cpu())
    flat = flat.reshape(-1, flat.shape[-1])[slots]
    return O.decode_rows(flat, None if scale is None else scale.cpu().numpy().reshape(-1, 8)[slots])


def table_of(n, dim, dev):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float().to(dev)


#: Rounding of y in fp32, relative to the row's elements (for a rotated one, to
#: the length of its pair): half the sum's 21 roundings, the mean + eps, rsqrtf
#: (2 ulp), two products and, rotated, two more and a difference: less than
#: 10.5 + 0.5 + 4 + 2 + 3 = 20 units of 2^-24.
Y_REL = 20 * 2.0 ** -24


def reference_rows(x, weight, pos, table, offset, interleaved, norm=True, eps=1e-6):
    """y fp64 [n, 512] of rows x [n, 512], and the length its error scales with."""
    y, mag = np.zeros((len(x), 512)), np.zeros((len(x), 512))
    w = None if weight is None else weight.double().cpu().numpy()
    tab = None if table is None else table.double().cpu().numpy()
    x = x.double().cpu().numpy()
    for i in range(len(x)):
        if pos is not None and pos[i] < 0:
            continue
        c, s = (None, None) if tab is None else np.split(tab[pos[i]], 2)
        plain = C.norm_rope(x[i], w, eps, norm, None, None, 0, True)
        y[i] = C.norm_rope(x[i], w, eps, norm, c, s, offset, interleaved)
        mag[i] = np.abs(plain)
        if tab is not None:
            half = len(c)
            a = offset + (2 * np.arange(half) if interleaved else np.arange(half))
            b = a + 1 if interleaved else a + half
            mag[i][a] = mag[i][b] = np.abs(plain[a]) + np.abs(plain[b])
    return y, mag


def check_stored(cache, scale, fmt, slots, y, mag):
    """Stored rows against fp64 rows y: each value is one that some y within
    Y_REL of the reference is stored as."""
    got = cache_values(cache, scale, slots)
    tol = Y_REL * mag
    bf = 2.0 ** -8 * np.abs(y) + tol * 1.01
    if fmt == "bf16":
        assert np.all(np.abs(got - y) <= bf)
        return
    if fmt == "fp8_fp32_scales":
        raw = cache.cpu().numpy().reshape(-1, 512)[slots]
        step = np.repeat(scale.cpu().numpy().astype(np.float64).reshape(-1, 8)[slots], 64, axis=1)
        amax = np.abs(y.reshape(-1, 8, 64)).max(2)
        rel = np.repeat(tol.reshape(-1, 8, 64).max(2) / amax + 2.0 ** -23, 64, axis=1)
        assert np.all(np.abs(step / np.repeat(amax / 448, 64, axis=1) - 1) <= rel)
        code = O.E4M3FN_TABLE[raw.astype(int)]
        half = np.maximum(2.0 ** -10, np.abs(y / step) * 2.0 ** -4)
        assert np.all(np.abs(code - y / step) <= half * (1 + 1e-5) + (tol / step) * 1.01 + 448 * rel)
        return
    assert np.all((np.abs(got - y) <= bf)[:, :64])
    raw = cache.cpu().numpy().reshape(-1, cache.shape[-1])[slots].astype(int)
    z, tz = y[:, 64:], tol[:, 64:]
    if fmt == "packed640":
        assert np.all(raw[:, 583:] == 0)
        amax = np.abs(z.reshape(-1, 7, 64)).max(2)
        power = 2.0 ** (raw[:, 576:583] - 127.0)
        slack = 1 + tz.reshape(-1, 7, 64).max(2) / amax
        assert np.all(amax <= 448 * power * slack) and np.all(amax * slack > 224 * power)
        step = np.repeat(power, 64, axis=1)
        code = O.E4M3FN_TABLE[raw[:, 128:576]]
        assert np.all(np.abs(code - z / step) <= np.maximum(2.0 ** -10, np.abs(z / step) * 2.0 ** -4) * (1 + 1e-5) + tz / step * 1.01)
        return
    assert np.all(raw[:, 381:] == 0)
    top, e = np.abs(y).max(1), raw[:, 380] - 127
    slack = 1 + tol.max(1) / top
    assert np.all(top * slack >= 2.0 ** (e + 10.0)) and np.all(top / slack < 2.0 ** (e + 11.0))
    want = np.abs(z.reshape(-1, 28, 16)).max(2) / 6 / 2.0 ** e[:, None]
    s = O.E4M3FN_TABLE[raw[:, 352:380]]
    ulp = np.maximum(2.0 ** -10, want * 2.0 ** -4)  # at least half a step of e4m3
    assert np.all(np.abs(s - want) <= ulp * (1 + 1e-5) + 2.0 ** -22 * want + tz.reshape(-1, 28, 16).max(2) / 2.0 ** e[:, None])
    step = np.repeat(s * 2.0 ** e[:, None], 16, axis=1)
    two = raw[:, 128:352]
    code = np.empty_like(z)
    code[:, 0::2], code[:, 1::2] = O.E2M1_TABLE[two & 15], O.E2M1_TABLE[two >> 4]
    live = step > 0
    assert np.all(code[~live] == 0)
    q, c, t = (z[live] / step[live]), code[live], (tz[live] / step[live]) * 1.01 + 1e-9
    # the interval of quotients that a code stands for
    mags = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    k = np.searchsorted(mags, np.abs(c))
    lo = np.where(k == 0, -0.25, np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5])[k])
    hi = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, np.inf])[k]
    m = np.where(k == 0, np.abs(q), q * np.sign(c))
    assert np.all(m >= lo - t) and np.all(m <= hi + t)


ROWS = {
    "single token": dict(n=1),
    "decode": dict(n=37, heads=64, weights=torch.bfloat16, fused=True),
    "128 heads, halves, last elements": dict(n=9, heads=128, inter=False, offset=448),
    "one head": dict(n=300, heads=1, inter=False, padded=11),
    "fp16": dict(n=20, heads=3, dtype=torch.float16, padded=3, fused=True),
    "fp32": dict(n=21, heads=5, dtype=torch.float32, offset=448, weights=torch.bfloat16),
    "rope of 32": dict(n=12, heads=2, dim=32, offset=64, inter=False),
    "rope of 128": dict(n=12, heads=2, dim=128, offset=128),
    "rope of 256": dict(n=12, heads=2, dim=256, offset=256, inter=False),
    "no rope": dict(n=12, heads=2, dim=0),
    "no norm": dict(n=12, heads=2, norm=False),
    "no weights": dict(n=12, heads=2, weights=None),
    "rows only": dict(n=1500, heads=0),
}


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("name", sorted(ROWS))
def test_norm_rope_store_matches_the_oracle(cuda_device, name, fmt):
    o = dict(dict(heads=64, dtype=torch.bfloat16, weights=torch.float32, dim=64, offset=0, inter=True, norm=True, padded=0,
                  fused=False), **ROWS[name])
    dev, n, heads = cuda_device, o["n"], o["heads"]
    g = torch.Generator().manual_seed(len(name))
    x = (2 * torch.randn(n, heads + 1, 512, generator=g)).to(o["dtype"]).to(dev)
    if o["fused"]:
        q, kv = x[:, :heads], x[:, heads]
    else:
        q, kv = x[:, :heads].contiguous(), x[:, heads:].contiguous()
    w = [None, None] if o["weights"] is None else [(1 + 0.3 * torch.randn(512, generator=g)).to(o["weights"]).to(dev) for _ in range(2)]
    table = table_of(3000, o["dim"], dev) if o["dim"] else None
    pos = torch.randint(0, 3000, (n,), generator=g).int()
    blocks = n // 64 + 2
    slots = torch.randperm(blocks * 128, generator=g)[:n].int()
    if n > 2:
        slots[1] = -1  # not stored, but its queries and values are made
    if o["padded"]:
        pos[-o["padded"]:] = -1
    cache, scale = new_cache(fmt, blocks, dev)
    before = cache.clone()
    kv_out = torch.full((n, 512), 7.0, dtype=torch.bfloat16, device=dev)
    q_out = torch.full((n, heads, 512), 7.0, dtype=torch.bfloat16, device=dev) if heads else None
    got = Q.norm_rope_store(q if heads else None, kv, q_out=q_out, kv_cache=cache, kv_scale=scale, kv_out=kv_out,
                            slot_map=slots.to(dev), positions=pos.to(dev), cos_sin=table, q_weight=w[0] if heads else None,
                            kv_weight=w[1], eps=1e-5, rope_offset=o["offset"], interleaved=o["inter"], norm_q=o["norm"],
                            norm_kv=o["norm"])
    torch.cuda.synchronize()
    assert Q.device_status() == 0
    live = pos.numpy() >= 0
    args = (pos.numpy(), table, o["offset"], o["inter"], o["norm"], 1e-5)
    if heads:
        assert got is q_out
        flat = q.reshape(n * heads, 512)
        y, mag = reference_rows(flat, w[0], np.repeat(pos.numpy(), heads), *args[1:])
        out = got.double().cpu().numpy().reshape(n * heads, 512)
        alive = np.repeat(live, heads)
        assert np.all(out[~alive] == 7.0)
        assert np.all((np.abs(out - y) <= 2.0 ** -8 * np.abs(y) + 1.01 * Y_REL * mag)[alive])
    y, mag = reference_rows(kv.reshape(n, 512), w[1], *args)
    stored = live & (slots.numpy() >= 0)
    check_stored(cache, scale, fmt, slots.numpy()[stored], y[stored], mag[stored])
    others = np.setdiff1d(np.arange(blocks * 128), slots.numpy()[stored])
    assert torch.equal(cache.view(blocks * 128, -1)[others], before.view(blocks * 128, -1)[others])
    if scale is not None:
        assert torch.all(scale.view(-1, 8)[others] == 5.0)
    values = kv_out.double().cpu().numpy()
    assert np.all(values[~live] == 7.0)
    held = cache_values(cache, scale, slots.numpy()[stored])
    if fmt == "fp8_fp32_scales":
        assert np.all(np.abs(values[stored] - held) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(held))
    else:
        assert np.array_equal(values[stored], held)


def half_even(x, bits, lowest=0.0):
    """x to `bits` significant bits, none finer than `lowest`, ties to even."""
    with np.errstate(divide="ignore"):
        unit = np.maximum(np.exp2(np.floor(np.log2(np.abs(x))) + 1 - bits), lowest)
    return np.where(x == 0, 0, np.round(x / np.where(x == 0, 1, unit)) * unit)


def formula_rows(y, fmt):
    """The values that rows y [n, 512] are held as, by the formats' definitions in 64 bits."""
    if fmt == "bf16":
        return half_even(y, 8)
    n = len(y)
    if fmt == "fp8_fp32_scales":
        t = y.reshape(n, 8, 64)
        scale = np.abs(t).max(2, keepdims=True) / 448
        return (half_even(t / scale, 4, 2.0 ** -9) * scale).reshape(n, 512)
    rope = half_even(y[:, :64], 8)
    if fmt == "packed640":
        t = y[:, 64:].reshape(n, 7, 64)
        scale = np.exp2(np.ceil(np.log2(np.abs(t).max(2, keepdims=True) / 448)))
        return np.concatenate((rope, (half_even(t / scale, 4, 2.0 ** -9) * scale).reshape(n, 448)), 1)
    t = y[:, 64:].reshape(n, 28, 16)
    power = np.exp2(np.floor(np.log2(np.abs(y).max(1))) - 10)[:, None, None]
    scale = half_even(np.abs(t).max(2, keepdims=True) / 6 / power, 4, 2.0 ** -9) * power
    return np.concatenate((rope, (np.clip(half_even(t / scale, 2, 0.5), -6, 6) * scale).reshape(n, 448)), 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_stored_rows_are_the_formulas(cuda_device, fmt, dtype):
    """Every stored element is the rounding of the exact one. The kernel carries
    y to about 2^-40 of the products it is made of, so of the 600,000 elements
    one in 10^5 trials would be so near a rounding border; fp32 alone is off
    in some ten (bf16)."""
    dev, n = cuda_device, 1200
    g = torch.Generator().manual_seed(21)
    kv = (2 * torch.randn(n, 512, generator=g)).to(dtype).to(dev)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(dev)
    pos = torch.randint(0, 3000, (n,), generator=g).int()
    slots = torch.randperm(1280, generator=g)[:n].int()
    for inter, offset in ((True, 0), (False, 448)):
        cache, scale = new_cache(fmt, 10, dev)
        out = torch.empty(n, 512, dtype=torch.bfloat16, device=dev)
        Q.norm_rope_store(None, kv, kv_cache=cache, kv_scale=scale, kv_out=out, slot_map=slots.to(dev), positions=pos.to(dev),
                          cos_sin=table_of(3000, 64, dev), kv_weight=w, rope_offset=offset, interleaved=inter)
        torch.cuda.synchronize()
        y, _ = reference_rows(kv, w, pos.numpy(), table_of(3000, 64, dev), offset, inter, eps=float(np.float32(1e-6)))
        want, got = formula_rows(y, fmt), cache_values(cache, scale, slots.numpy())
        if fmt == "fp8_fp32_scales":
            # the codes are the formula's; the root of fp8 rows, common to a group and its scale, is fp32's: 15 of the
            # 20 units in Y_REL, and three roundings (two products, the scale's own)
            exact = np.abs(y.reshape(n, 8, 64)).max(2) / 448
            codes = cache_values(cache, torch.ones_like(scale), slots.numpy())
            assert np.array_equal(codes, half_even(y / np.repeat(exact, 64, axis=1), 4, 2.0 ** -9))
            held = scale.cpu().double().numpy().reshape(-1, 8)[slots.numpy()]
            assert np.all(np.abs(held - exact) <= Y_REL * exact)
        else:
            assert np.array_equal(got, want)
            assert np.array_equal(out.double().cpu().numpy(), want)


def test_key_rows_without_a_cache(cuda_device):
    """kv_out alone: the rows in bf16."""
    g = torch.Generator().manual_seed(22)
    kv = torch.randn(70, 512, generator=g).to(cuda_device)
    out = torch.empty(70, 512, dtype=torch.bfloat16, device=cuda_device)
    pos = torch.arange(70, dtype=torch.int32)
    Q.norm_rope_store(None, kv, kv_out=out, positions=pos.to(cuda_device), cos_sin=table_of(70, 64, cuda_device))
    torch.cuda.synchronize()
    y, _ = reference_rows(kv, None, pos.numpy(), table_of(70, 64, cuda_device), 0, True, eps=float(np.float32(1e-6)))
    assert np.array_equal(out.double().cpu().numpy(), half_even(y, 8))


@pytest.mark.parametrize("fmt", ["packed384", "packed640"])
def test_rows_as_they_are_are_stored_bit_for_bit(cuda_device, fmt):
    """Without norm and rotation the quantisation of bf16 rows is exact,
    halves of a step among them."""
    g = torch.Generator().manual_seed(3)
    x = torch.cat((torch.randn(200, 512, generator=g) * torch.logspace(-9, 9, 200)[:, None],
                   torch.randint(-12, 13, (100, 512), generator=g).float(), torch.zeros(2, 512))).to(torch.bfloat16)
    x[201, 64:80], x[202] = 0, x[202] * 2.0 ** -120
    dev, n = cuda_device, x.shape[0]
    cache, _ = new_cache(fmt, 3, dev)
    Q.norm_rope_store(None, x.to(dev), kv_cache=cache, slot_map=torch.arange(n, dtype=torch.int32, device=dev), norm_kv=False)
    torch.cuda.synchronize()
    got = cache.cpu().numpy().reshape(-1, cache.shape[-1])[:n]
    if fmt == "packed384":
        ref = np.stack([C.pack384(r, O.E2M1_TABLE[:8], O.E4M3FN_TABLE[:127]) for r in x.double().numpy()])
        assert np.array_equal(got[:, 352:], ref[:, 352:])
        assert np.array_equal(O.decode_rows(got, None), O.decode_rows(ref, None))
        assert np.array_equal(got[:, :128], ref[:, :128])
    else:
        ref = W._quantize_packed_rows(x.float()).numpy()
        keep = np.arange(200)  # behind them tiles of zeros, whose exponent means nothing
        assert np.array_equal(O.decode_rows(got[keep], None), O.decode_rows(ref[keep], None))


def test_rows_that_are_not_finite(cuda_device):
    """A scale group with an infinity or a NaN stores NaN; the others and the
    row's neighbours are as without it."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(4, 512, generator=g)
    x[1, 70], x[1, 500], x[2, 300] = float("inf"), float("nan"), -float("inf")
    dev = cuda_device
    for fmt, size in (("packed384", 16), ("packed640", 64)):
        out = torch.empty(4, 512, dtype=torch.bfloat16, device=dev)
        cache, _ = new_cache(fmt, 1, dev)
        Q.norm_rope_store(None, x.to(dev), kv_cache=cache, kv_out=out, norm_kv=False,
                          slot_map=torch.arange(4, dtype=torch.int32, device=dev))
        clean = torch.where(torch.isfinite(x), x, 0.0)
        ref, ref_cache = torch.empty_like(out), new_cache(fmt, 1, dev)[0]
        Q.norm_rope_store(None, clean.to(dev), kv_cache=ref_cache, kv_out=ref, norm_kv=False,
                          slot_map=torch.arange(4, dtype=torch.int32, device=dev))
        torch.cuda.synchronize()
        bad = (~torch.isfinite(x))[:, 64:].view(4, -1, size).any(2).repeat_interleave(size, 1)
        bad = torch.cat((torch.zeros(4, 64, dtype=torch.bool), bad), 1)
        o, r = out.cpu().float(), ref.cpu().float()
        assert torch.all(torch.isnan(o[bad])) and torch.equal(o[~bad], r[~bad])


def test_bad_positions_and_slots_are_skipped(cuda_device):
    dev = cuda_device
    g = torch.Generator().manual_seed(5)
    kv, q = torch.randn(5, 512, generator=g).to(dev), torch.randn(5, 2, 512, generator=g).to(dev)
    cache, _ = new_cache("packed384", 1, dev)
    before = cache.clone()
    q_out = torch.full((5, 2, 512), 7.0, dtype=torch.bfloat16, device=dev)
    Q.norm_rope_store(q, kv, q_out=q_out, kv_cache=cache, cos_sin=table_of(10, 64, dev),
                      positions=i32([0, 10, 2 ** 31 - 1, -1, 9], dev), slot_map=i32([128, 0, 1, 2, 2 ** 31 - 1], dev))
    torch.cuda.synchronize()
    assert Q.device_status() == Q.FAULT_POSITION | Q.FAULT_SLOT
    assert torch.equal(cache, before)
    assert torch.all(q_out[1:4] == 7) and torch.all((q_out[[0, 4]] != 7).any(2))


def test_in_place_queries_and_views(cuda_device):
    """q_out = q gives the bits of separate buffers; so does a head slice of a
    wider tensor."""
    dev = cuda_device
    g = torch.Generator().manual_seed(6)
    q = torch.randn(50, 64, 512, generator=g).to(torch.bfloat16).to(dev)
    kw = dict(positions=torch.arange(50, dtype=torch.int32, device=dev), cos_sin=table_of(64, 64, dev))
    a = Q.norm_rope_store(q, **kw)
    wide = torch.zeros(50, 70, 512, dtype=torch.bfloat16, device=dev)
    wide[:, 3:67] = q
    assert torch.equal(a, Q.norm_rope_store(wide[:, 3:67], **kw))
    assert torch.equal(a, Q.norm_rope_store(q, q_out=q, **kw)) and torch.equal(a, q)


# ------------------------------------------------------------------ attention over 4-bit rows
ATTN = {
    "tiny csa decode": dict(layout="BSND", q_lens=[1, 1], s2=[4096, 4096], cmp_ratio=4, mode="CSA", k2=512, n_valid=384),
    "csa decode": dict(layout="BSND", q_lens=[2] * 6, s2=[5000, 20000, 4100, 999, 129, 2], cmp_ratio=4, mode="CSA", k2=512),
    "swa ragged": dict(layout="TND", q_lens=[1, 130, 0, 57, 300], s2=[1, 130, 40, 1000, 300]),
    "hca decode": dict(layout="BSND", q_lens=[1] * 3, s2=[70000, 128, 127], cmp_ratio=128, mode="HCA"),
    "hca 128 heads": dict(layout="TND", q_lens=[3, 5], s2=[3000, 40000], cmp_ratio=128, mode="HCA", n1=128),
    "csa chunks 128 heads": dict(layout="TND", q_lens=[70, 33, 1], s2=[9000, 400, 33], cmp_ratio=4, mode="CSA", k2=512, n1=128),
    "k2 1024": dict(layout="BSND", q_lens=[2] * 2, s2=[30000, 9000], cmp_ratio=4, mode="CSA", k2=1024),
    "k2 100": dict(layout="BSND", q_lens=[3] * 2, s2=[300, 9000], cmp_ratio=8, mode="CSA", k2=100),
    "padded and empty": dict(layout="BSND", q_lens=[2] * 4, s2=[0, 2, 600, 5000], cmp_ratio=4, mode="CSA", k2=512,
                             seqused_q=[2, 0, 1, 2]),
    "no mask": dict(layout="TND", q_lens=[2, 3], s2=[200, 333], ori_mask_mode=0, ori_win_left=-1, ori_win_right=-1),
    "bsnd kv picks": dict(layout="BSND", q_lens=[2, 2], s2=[900, 900], cmp_ratio=4, mode="CSA", k2=100, layout_kv="BSND",
                          ori_k1=64, kv_pad=5),
    "tnd kv hca": dict(layout="TND", q_lens=[4, 9], s2=[2000, 5000], cmp_ratio=8, mode="HCA", layout_kv="TND"),
    "no sinks": dict(layout="TND", q_lens=[5], s2=[777], cmp_ratio=4, mode="CSA", k2=128, sinks=False),
    "peaked": dict(layout="TND", q_lens=[40], s2=[2000], cmp_ratio=4, mode="CSA", k2=512, q_scale=8.0),
}


def four_bit_tolerance(out, lse, w, tokens):
    """4-bit rows and queries are exact in the products' bf16 operands, so
    only fp32 sums, the weights' rounding to bf16 (2^-8 of each, relative to
    sum_j w_j |v_j|) and the output's remain."""
    o_ref, l_ref = O.reference(w, tokens)
    tb, tp = w.token_batch(), w.token_pos()
    for i, t in enumerate(tokens):
        k = O.token_kv(w, t, int(tb[t]), int(tp[t]))
        if k is None or len(k) == 0:
            assert np.all(out[t] == 0) and np.all(lse[t] == -np.inf)
            continue
        q = O.q_fp64(w, t)
        x = w.softmax_scale * (q @ k.T)
        # fp32 accumulation of 512 products: 512 roundings of the running sum, of 2^-24 of sum |q k|
        dx = 512 * 2.0 ** -24 * w.softmax_scale * (np.abs(q) @ np.abs(k).T).max(1) + 2.0 ** -20
        sink = -np.inf if w.sinks is None else w.sinks.double().numpy()
        m = np.maximum(x.max(1), sink)
        p = np.exp(x - m[:, None])
        p /= (p.sum(1) + np.exp(sink - m))[:, None]
        bound = (2 * dx[:, None] + 2.0 ** -8 + len(k) * 2.0 ** -24) * (p @ np.abs(k)) + 2.0 ** -8 * np.abs(o_ref[i])
        assert np.all(np.abs(out[t] - o_ref[i]) <= 1.01 * bound + 1e-12), (t, np.abs(out[t] - o_ref[i]).max())
        assert np.all(np.abs(lse[t] - l_ref[i]) <= dx + len(k) * 2.0 ** -24 + 2.0 ** -20 * np.abs(l_ref[i]))


@pytest.mark.parametrize("ctas", [0, 5])
@pytest.mark.parametrize("name", sorted(ATTN))
def test_four_bit_attention_matches_the_oracle(cuda_device, name, ctas):
    w = W.build(f"4-bit {name}", kv_format="packed384", seed=len(name), **ATTN[name])
    out, lse = run_gpu(w, cuda_device, num_ctas=ctas, lse=True)
    tokens = W.subset_tokens(w, 60, seed=1).tolist()
    four_bit_tolerance(out, lse, w, tokens)


def test_four_bit_attention_follows_the_bytes(cuda_device):
    """Scales, exponents and codes over their whole range, one row per token:
    the output is the row itself (to the softmax's rounding)."""
    r = np.random.RandomState(0)
    n = 128
    rows = np.zeros((n, 384), dtype=np.uint8)
    rope = torch.randn(n, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    rows[:, :128] = rope.view(torch.uint8).numpy()
    rows[:, 128:352] = r.randint(0, 256, (n, 224))
    rows[:, 352:380] = r.randint(0, 127, (n, 28)) | (r.randint(0, 2, (n, 28)) << 7)  # negative scales too
    rows[:, 380] = 127 + r.randint(-30, 20, n)
    w = W.build("bytes", layout="TND", q_lens=[n], s2=[n], kv_format="packed384", sinks=False, ori_win_left=0,
                ori_win_right=0, softmax_scale=0.0, seed=1)
    pool = np.zeros(w.ori_kv.shape, dtype=np.uint8)
    pool[int(w.ori_block_table[0, 0]), :, 0] = rows
    w = dataclasses.replace(w, ori_kv=torch.from_numpy(pool))
    out, lse = run_gpu(w, cuda_device, lse=True)
    want = torch.from_numpy(O.decode_rows(rows, None)).to(torch.bfloat16).double().numpy()
    assert np.array_equal(out, np.repeat(want[:, None], 64, axis=1)) and np.all(np.abs(lse) <= LSE_ATOL)


@pytest.mark.parametrize("ctas", [1, 3])
def test_four_bit_units_leave_one_another_alone(cuda_device, ctas):
    """Queries that are tiny, huge, infinite or NaN, in heads of some tokens: the
    units worked on after them by the same CTA, and their other heads, are what
    they are without them."""
    w = W.build("4-bit odd queries", layout="TND", q_lens=[50, 40], s2=[300, 40], cmp_ratio=4, mode="CSA", k2=256,
                kv_format="packed384", seed=11)
    q, odd = w.q.clone(), {}
    for t, h, v in ((3, 0, float("inf")), (4, 1, float("nan")), (5, 2, float("-inf")), (20, 63, float("nan")),
                    (60, 31, float("inf")), (61, 0, float("nan"))):
        q[t, h, 17 * h % 512] = v
        odd.setdefault(t, []).append(h)
    q[8] *= 2.0 ** 60
    q[9] *= 2.0 ** -60
    q[30, ::2] *= -(2.0 ** 40)
    w = dataclasses.replace(w, q=q)
    out, lse = run_gpu(w, cuda_device, num_ctas=ctas, lse=True)
    for t, heads in odd.items():
        assert not np.isfinite(out[t, heads]).any() and not np.isfinite(lse[t, heads]).any()
        # their products are not finite in the oracle either: the other heads against a query of ones there
        q[t, heads] = 1.0
    w = dataclasses.replace(w, q=q)
    tokens = list(range(w.total_t))
    o_ref, l_ref = O.reference(w, tokens)
    for t, heads in odd.items():
        out[t, heads], lse[t, heads] = o_ref[t, heads], l_ref[t, heads]
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    four_bit_tolerance(out, lse, w, tokens)


@pytest.mark.parametrize("ctas", [0, 1, 5])
def test_four_bit_units_without_rows_in_a_row(cuda_device, ctas):
    """More units without rows one after the other than any ring holds, at the
    start, between others, and at the end."""
    s2 = [0] * 9 + [300, 0, 0, 128, 7] + [0] * 12 + [40] + [0] * 3
    w = W.build("4-bit empty units", layout="TND", q_lens=[2] * len(s2), s2=s2, cmp_ratio=4, mode="CSA", k2=64,
                kv_format="packed384", seed=12)
    out, lse = run_gpu(w, cuda_device, num_ctas=ctas, lse=True)
    four_bit_tolerance(out, lse, w, list(range(w.total_t)))


def test_four_bit_rows_through_the_other_entry_points(cuda_device):
    """The pass without a workspace gives the bits of the one with, and the
    gather exports the rows' bytes."""
    w = W.build("4-bit entries", layout="TND", q_lens=[5, 3], s2=[700, 9000], cmp_ratio=4, mode="CSA", k2=512,
                kv_format="packed384", seed=13)
    args = W.device_inputs(w, cuda_device)
    args.pop("return_softmax_lse")
    out, plan = torch.empty_like(args["q"]), torch.empty(Q.METADATA_INTS, dtype=torch.int32, device=cuda_device)
    lse = torch.empty(w.total_t, 64, device=cuda_device)
    p = Q.make_params(attn_out=out, softmax_lse=lse, metadata=plan, return_lse=True, num_ctas=24, **args)
    Q.metadata(p, plan)
    size = Q.workspace_size(p)
    assert size > 0  # fewer tokens than CTAs: the scratch is used
    Q.forward(p, torch.empty(size, dtype=torch.uint8, device=cuda_device))
    want = out.clone(), lse.clone()
    out.fill_(float("nan")), lse.fill_(float("nan"))
    Q.forward_noalloc(p)
    torch.cuda.synchronize()
    assert Q.device_status() == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    tokens = [0, 4, 5, 7]
    new = lambda *s, t=torch.int32: torch.empty(*s, dtype=t, device=cuda_device)  # noqa: E731
    rows, ids, counts = new(4, 1280, 384, t=torch.uint8), new(4, 1280), new(4)
    Q.debug_gather(p, i32(tokens, cuda_device), 1280, rows, None, ids, counts)
    torch.cuda.synchronize()
    assert Q.device_status() == 0
    tb, tp = w.token_batch(), w.token_pos()
    for j, t in enumerate(tokens):
        k = O.token_kv(w, t, int(tb[t]), int(tp[t]))
        got = rows[j, :int(counts[j])][(ids[j, :int(counts[j])] >= 0).nonzero()[:, 0]].cpu().numpy()
        assert np.array_equal(O.decode_rows(got, None), k)


def test_four_bit_full_decode_batch(cuda_device):
    w = W.config(2, kv_format="packed384")
    out, lse = run_gpu(w, cuda_device, lse=True)
    tokens = W.subset_tokens(w, 40, seed=3).tolist()
    four_bit_tolerance(out, lse, w, tokens)
    assert_parity(out, lse, w, tokens)


# ------------------------------------------------------------------ together
class Serving:
    """The state a serving loop keeps: lengths, tables, pools, buffers of the
    largest step. step() only launches, so that it can be captured."""

    def __init__(self, dev, batch, width, ratio, max_t, heads=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
        self.g, self.dev, self.batch, self.ratio, self.max_t, self.heads = g, dev, batch, ratio, max_t, heads
        self.prev, self.lens = new(batch), new(batch)
        self.pools, self.tables, self.free, self.count = [], [], [], []
        for r in (1, ratio):
            blocks = batch * width
            self.pools.append(new_cache("packed384", blocks, dev)[0])
            self.tables.append(torch.full((batch, -(-width // r)), -1, dtype=torch.int32, device=dev))
            self.free.append(torch.randperm(blocks, generator=g).int().to(dev))
            self.count.append(i32([blocks], dev))
        self.x = torch.zeros(max_t, heads + 1, 512, dtype=torch.bfloat16, device=dev)
        self.cx = torch.zeros(max_t, 512, dtype=torch.bfloat16, device=dev)
        self.w = [(1 + 0.2 * torch.randn(512, generator=g)).to(dev) for _ in range(2)]
        self.table = table_of(width * 128, 64, dev)
        self.sinks = torch.randn(heads, generator=g).to(dev)
        self.slots, self.pos = [new(max_t), new(max_t)], [new(max_t), new(max_t)]
        self.cu, self.residual = new(batch + 1), new(batch)
        self.idx = torch.full((max_t, 1, 64), -1, dtype=torch.int32, device=dev)
        self.q = torch.zeros(max_t, heads, 512, dtype=torch.bfloat16, device=dev)
        self.out = torch.zeros_like(self.q)
        self.lse = torch.zeros(max_t, heads, device=dev)
        self.plan = new(Q.METADATA_INTS)
        rows = dict(cos_sin=self.table, kv_weight=self.w[1])
        self.launches = [
            Q.make_block_table_params(block_table=self.tables[0], prev_lens=self.prev, lens=self.lens, free_list=self.free[0],
                                      free_count=self.count[0], slot_map=self.slots[0], positions=self.pos[0], cu_rows=self.cu),
            Q.make_block_table_params(block_table=self.tables[1], prev_lens=self.prev, lens=self.lens, free_list=self.free[1],
                                      free_count=self.count[1], slot_map=self.slots[1], positions=self.pos[1],
                                      residual=self.residual, cmp_ratio=ratio)]
        self.rows = [
            Q.make_norm_rope_params(q=self.x[:, :heads], q_out=self.q, kv=self.x[:, heads], kv_cache=self.pools[0],
                                    slot_map=self.slots[0], positions=self.pos[0], q_weight=self.w[0], **rows),
            Q.make_norm_rope_params(kv=self.cx, kv_cache=self.pools[1], slot_map=self.slots[1], positions=self.pos[1], **rows)]
        self.attn = Q.make_params(
            q=self.q, attn_out=self.out, ori_kv=self.pools[0], ori_scale=None, ori_block_table=self.tables[0],
            seqused_ori_kv=self.lens, layout="TND", cmp_kv=self.pools[1], cmp_block_table=self.tables[1],
            cmp_sparse_indices=self.idx, cu_seqlens_q=self.cu, cmp_residual_kv=self.residual, sinks=self.sinks,
            metadata=self.plan, softmax_lse=self.lse, cmp_ratio=ratio, return_lse=True)
        self.attn.total_t = 1  # few tokens are split over the SMs and need the workspace
        size = Q.workspace_size(self.attn)
        self.attn.total_t = max_t
        self.work = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)

    def feed(self, prev, lens):
        """New lengths, projections and picks for the next step."""
        n = max(0, sum(max(0, b - a) for a, b in zip(prev, lens)))
        self.n = n
        self.prev.copy_(i32(prev, self.dev)), self.lens.copy_(i32(lens, self.dev))
        self.x.copy_(torch.randn(self.x.shape, generator=self.g)), self.cx.copy_(torch.randn(self.cx.shape, generator=self.g))
        idx, t = np.full((self.max_t, 1, 64), -1), 0
        for a, b in zip(prev, lens):
            for p in range(a, b):
                seen = (p + 1) // self.ratio
                k = min(64, seen)
                idx[t, 0, :k] = torch.randperm(max(seen, 1), generator=self.g)[:k].numpy()
                t += 1
        self.idx.copy_(i32(idx, self.dev))

    def step(self, stream=None):
        for launch in self.launches:
            Q.block_tables(launch, stream)
        for launch in self.rows:
            Q.norm_rope(launch, stream)
        Q.metadata(self.attn, self.plan, stream)
        Q.forward(self.attn, self.work, stream)

    def check(self, prev, lens):
        torch.cuda.synchronize()
        assert Q.device_status() == 0
        n, dev = self.n, self.dev
        pos = self.pos[0].cpu().numpy()
        assert np.array_equal(pos[:n], np.concatenate([np.arange(a, b) for a, b in zip(prev, lens)] + [[]]))
        # stage 1: blocks of live requests are distinct and the counts add up
        for k, r in enumerate((1, self.ratio)):
            used = [int(v) for b, m in enumerate(lens) for v in self.tables[k][b, :-(-(m // r) // 128)].tolist()]
            free = self.free[k][:int(self.count[k][0])].tolist()
            assert sorted(used + free) == list(range(self.pools[k].shape[0]))
        # stage 2: the queries and the new rows
        y, mag = reference_rows(self.x[:n, 0], self.w[0], pos, self.table, 0, True)
        assert np.all(np.abs(self.q[:n, 0].double().cpu().numpy() - y) <= 2.0 ** -8 * np.abs(y) + 1.01 * Y_REL * mag)
        y, mag = reference_rows(self.x[:n, self.heads], self.w[1], pos, self.table, 0, True)
        check_stored(self.pools[0], None, "packed384", self.slots[0].cpu().numpy()[:n], y, mag)
        # stage 3: the attention over the caches as they are now
        q_lens = np.array([max(0, b - a) for a, b in zip(prev, lens)])
        w = W.build("shape only", layout="TND", q_lens=q_lens, s2=[max(m, 1) for m in lens], kv_format="packed384",
                    cmp_ratio=self.ratio, mode="CSA", k2=64, seed=0)
        w = dataclasses.replace(
            w, q=self.q[:n].cpu(), ori_kv=self.pools[0].cpu(), cmp_kv=self.pools[1].cpu(),
            ori_block_table=self.tables[0].cpu(), cmp_block_table=self.tables[1].cpu(),
            seqused_ori_kv=self.lens.cpu(), cmp_sparse_indices=self.idx[:n].cpu(), cmp_residual_kv=self.residual.cpu(),
            sinks=self.sinks.cpu(), cu_seqlens_q=self.cu.cpu())
        tokens = W.subset_tokens(w, 40, seed=n).tolist()
        four_bit_tolerance(self.out.float().cpu().numpy(), self.lse.cpu().numpy(), w, tokens)


STEPS = [([0, 0, 0, 0], [300, 5, 0, 129]), ([300, 5, 0, 129], [301, 6, 200, 130]), ([301, 6, 200, 130], [302, 0, 201, 131]),
         ([302, 0, 201, 131], [303, 127, 202, 132]), ([303, 127, 202, 132], [290, 130, 0, 133])]


def test_a_serving_loop_of_several_steps(cuda_device):
    """Prompts, decode steps, an ended, a new and a shortened request."""
    s = Serving(cuda_device, batch=4, width=8, ratio=4, max_t=440)
    for prev, lens in STEPS:
        s.feed(prev, lens)
        # the token count of a TND call is its buffers': steps with fewer tokens leave the rest to padding
        s.attn.total_t = s.n
        s.step()
        s.check(prev, lens)


def test_a_captured_step_replays_on_new_lengths(cuda_device):
    """One graph of tables, rows, plan and attention, replayed while lengths,
    projections and picks change; and a second graph on another stream in
    between, with buffers of its own."""
    loops = [Serving(cuda_device, batch=4, width=8, ratio=4, max_t=4, seed=k) for k in range(2)]
    for s in loops:
        s.feed([0] * 4, [0] * 4)
        s.step()  # the first call outside of a capture
    torch.cuda.synchronize()
    graphs = []
    for s in loops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    lens = [0] * 4
    for k in range(6):
        new = [n + 1 for n in lens]
        for s in loops:
            s.feed(lens, new)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s in loops:
            s.check(lens, new)
        lens = new if k != 3 else [0] + new[1:]
        if k == 3:  # request 0 ends: a step of its own, without tokens
            for s in loops:
                s.feed(new, lens)
                torch.cuda.synchronize()
                for launch in s.launches:
                    Q.block_tables(launch)
                torch.cuda.synchronize()


def test_rows_on_another_stream(cuda_device):
    """The calls run on the stream that they are given, outputs allocated for it."""
    dev = cuda_device
    s = torch.cuda.Stream()
    g = torch.Generator().manual_seed(8)
    q = torch.randn(600, 64, 512, generator=g).to(torch.bfloat16).to(dev)
    kw = dict(positions=torch.arange(600, dtype=torch.int32, device=dev), cos_sin=table_of(600, 64, dev))
    want = Q.norm_rope_store(q, **kw)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        got = Q.norm_rope_store(q, stream=stream, **kw)
        s.synchronize()
        assert torch.equal(got, want)
        args = [i32(v, dev) for v in ([[-1]], [0], [9], [4, 5], [2])]
        torch.cuda.synchronize()  # the inputs are made on the current stream
        slots, _ = Q.update_block_tables(*args, max_rows=10, stream=stream, num_blocks=6)
        s.synchronize()
        assert slots.tolist() == [640 + i for i in range(9)] + [-1]
