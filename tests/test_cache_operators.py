"""The operators around the cache on the CPU: struct layouts, refusals (every
call below is rejected before any CUDA call) and pins of their oracle."""

import ctypes

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
import workloads as W
from oracle import cache_oracle as C
from oracle import qsfm_oracle as O
from tests.test_abi import test_struct_layout_matches_c as struct_layout
from tests.test_abi import _valid, lib  # noqa: F401

INVALID, UNSUPPORTED = 1, 2


@pytest.mark.parametrize("cls,cname", [(Q.NormRopeParams, "qsfm_norm_rope_params"),
                                       (Q.BlockTableParams, "qsfm_block_table_params")])
def test_struct_layouts_match_c(tmp_path, cls, cname):
    struct_layout(tmp_path, cls, cname)


def test_defaults(lib):  # noqa: F811
    p, b = Q.NormRopeParams(), Q.BlockTableParams()
    lib.qsfm_norm_rope_params_init(ctypes.byref(p))
    lib.qsfm_block_table_params_init(ctypes.byref(b))
    assert (p.dim, p.norm_q, p.norm_kv, p.kv_layout) == (512, 1, 1, 0) and abs(p.eps - 1e-6) < 1e-12
    assert (b.cmp_ratio, b.block_size) == (1, 128)
    assert lib.qsfm_norm_rope_store(None, None) == INVALID
    assert lib.qsfm_update_block_tables(None, None) == INVALID


# fake device addresses far enough apart that no two tensors overlap
Q_AT, QO_AT, KV_AT, KVO_AT, CACHE_AT, SCALE_AT, W_AT, POS_AT, TAB_AT = (0x1000000 * (i + 1) for i in range(9))


def norm_rope_valid(lib):  # noqa: F811
    p = Q.NormRopeParams()
    lib.qsfm_norm_rope_params_init(ctypes.byref(p))
    p.tokens, p.heads, p.num_blocks, p.kv_layout = 4, 64, 8, Q.KV_PACKED384
    p.rope_dim, p.max_positions = 64, 100
    p.q_token_stride, p.q_head_stride, p.kv_token_stride = 64 * 512, 512, 512
    p.q, p.q_out, p.kv, p.kv_out, p.kv_cache = Q_AT, QO_AT, KV_AT, KVO_AT, CACHE_AT
    p.q_weight, p.kv_weight, p.positions, p.slot_map, p.cos_sin = W_AT, W_AT + 4096, POS_AT, POS_AT + 4096, TAB_AT
    return p


NORM_ROPE = [
    ("dim 256", dict(dim=256), UNSUPPORTED),
    ("dim 0", dict(dim=0), INVALID),
    ("negative tokens", dict(tokens=-1), INVALID),
    ("element type", dict(in_type=3), INVALID),
    ("negative eps", dict(eps=-1.0), INVALID),
    ("nan eps", dict(eps=float("nan")), INVALID),
    ("too many rows", dict(tokens=1 << 25), UNSUPPORTED),
    ("neither q nor kv", dict(q=None, kv=None), INVALID),
    ("q without heads", dict(heads=0), INVALID),
    ("q without q_out", dict(q_out=None), INVALID),
    ("heads without q", dict(q=None), INVALID),
    ("cache without kv", dict(kv=None), INVALID),
    ("kv without an output", dict(kv_cache=None, kv_out=None, slot_map=None), INVALID),
    ("rope of 48", dict(rope_dim=48), UNSUPPORTED),
    ("rope of 512", dict(rope_dim=512), UNSUPPORTED),
    ("rope past the row", dict(rope_offset=480), INVALID),
    ("rope not at a multiple", dict(rope_offset=32), UNSUPPORTED),
    ("negative offset", dict(rope_offset=-64), INVALID),
    ("no table", dict(cos_sin=None), INVALID),
    ("empty table", dict(max_positions=0), INVALID),
    ("no positions", dict(positions=None), INVALID),
    ("table without rope", dict(rope_dim=0), INVALID),
    ("row format", dict(kv_layout=4), INVALID),
    ("no slots", dict(slot_map=None), INVALID),
    ("no blocks", dict(num_blocks=0), INVALID),
    ("scale with 4-bit rows", dict(kv_scale=SCALE_AT), INVALID),
    ("fp8 rows without scale", dict(kv_layout=0), INVALID),
    ("2^31 rows", dict(num_blocks=1 << 24), UNSUPPORTED),
    ("slots without a cache", dict(kv_cache=None), INVALID),
    ("q stride of 4 bytes", dict(q_head_stride=514), INVALID),
    ("negative stride", dict(kv_token_stride=-512), INVALID),
    ("q not 16-byte aligned", dict(q=Q_AT + 8), INVALID),
    ("weight not 16-byte aligned", dict(kv_weight=W_AT + 4), INVALID),
    ("table not 16-byte aligned", dict(cos_sin=TAB_AT + 4), INVALID),
    ("positions not 4-byte aligned", dict(positions=POS_AT + 2), INVALID),
    ("q_out shifted inside q", dict(q_out=Q_AT + 1024), INVALID),
    ("q_out = q with gaps", dict(q_out=Q_AT, q_token_stride=65 * 512), INVALID),
    ("q_out = q of fp16", dict(q_out=Q_AT, in_type=1), INVALID),
    ("kv_out = kv", dict(kv_out=KV_AT), INVALID),
    ("kv_out inside q", dict(kv_out=Q_AT + 4096), INVALID),
    ("cache over the slots", dict(slot_map=CACHE_AT + 64), INVALID),
    ("cache over kv_out", dict(kv_out=CACHE_AT + 64), INVALID),
]


@pytest.mark.parametrize("why,change,code", NORM_ROPE, ids=[c[0] for c in NORM_ROPE])
def test_norm_rope_refusals(lib, why, change, code):  # noqa: F811
    p = norm_rope_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    assert lib.qsfm_norm_rope_store(ctypes.byref(p), None) == code


@pytest.mark.parametrize("change", [{}, dict(q_out=Q_AT), dict(q=None, q_out=None, heads=0, q_weight=None),
                                    dict(kv=None, kv_cache=None, kv_out=None, slot_map=None, kv_weight=None),
                                    dict(rope_dim=0, cos_sin=None, positions=None)],
                         ids=["all", "in place", "kv only", "q only", "norm only"])
def test_norm_rope_valid_calls_pass_the_checks(lib, change):  # noqa: F811
    """With no tokens a valid call returns before anything is launched."""
    p = norm_rope_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    p.tokens = 0
    assert lib.qsfm_norm_rope_store(ctypes.byref(p), None) == 0


def block_tables_valid(lib):  # noqa: F811
    p = Q.BlockTableParams()
    lib.qsfm_block_table_params_init(ctypes.byref(p))
    p.batch, p.max_blocks, p.num_blocks, p.free_capacity, p.max_rows = 4, 16, 64, 64, 100
    for i, f in enumerate(("block_table", "prev_lens", "lens", "free_list", "free_count", "slot_map", "positions",
                           "cu_rows", "residual", "free_count_out")):
        setattr(p, f, 0x10000 * (i + 1))
    return p


TABLES = [
    ("negative batch", dict(batch=-1), INVALID),
    ("no columns", dict(max_blocks=0), INVALID),
    ("no blocks", dict(num_blocks=0), INVALID),
    ("negative capacity", dict(free_capacity=-1), INVALID),
    ("negative rows", dict(max_rows=-1), INVALID),
    ("ratio 0", dict(cmp_ratio=0), INVALID),
    ("ratio 129", dict(cmp_ratio=129), INVALID),
    ("block size 64", dict(block_size=64), UNSUPPORTED),
    ("block size 0", dict(block_size=0), INVALID),
    ("8193 requests", dict(batch=8193), UNSUPPORTED),
    ("2^31 rows", dict(num_blocks=1 << 24), UNSUPPORTED),
    ("2^30 columns", dict(max_blocks=1 << 30), UNSUPPORTED),
    ("table of 2^31 entries", dict(batch=8192, max_blocks=1 << 18), UNSUPPORTED),
    ("too many new rows", dict(max_rows=(1 << 30) + 1), UNSUPPORTED),
    ("no count", dict(free_count=None), INVALID),
    ("no free list", dict(free_list=None), INVALID),
    ("no table", dict(block_table=None), INVALID),
    ("no lengths", dict(lens=None), INVALID),
    ("no previous lengths", dict(prev_lens=None), INVALID),
    ("no slots", dict(slot_map=None), INVALID),
    ("lengths not aligned", dict(lens=0x30002), INVALID),
    ("slots over positions", dict(positions=0x60010), INVALID),
    ("cu_rows over the lengths", dict(cu_rows=0x30000), INVALID),
    ("count inside the free list", dict(free_count=0x40004), INVALID),
]


@pytest.mark.parametrize("why,change,code", TABLES, ids=[c[0] for c in TABLES])
def test_block_table_refusals(lib, why, change, code):  # noqa: F811
    p = block_tables_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    assert lib.qsfm_update_block_tables(ctypes.byref(p), None) == code


def test_four_bit_rows_take_no_scale_tensors(lib):  # noqa: F811
    p = _valid(lib)
    p.kv_layout = Q.KV_PACKED384
    assert lib.qsfm_forward(ctypes.byref(p), None, 0, None) == INVALID  # ori_scale given
    p.ori_scale = None
    n = ctypes.c_size_t(0)
    p.max_s1 = 8
    assert lib.qsfm_forward_workspace_size(ctypes.byref(p), ctypes.byref(n)) == 0


@pytest.mark.parametrize("bad", [dict(q=torch.zeros(2, 4, 512)), dict(kv=torch.zeros(2, 512, dtype=torch.float64)),
                                 dict(kv=torch.zeros(2, 500)), dict(q=torch.zeros(2, 512)), {},
                                 dict(kv=torch.zeros(512, 2).t()),
                                 dict(kv=torch.zeros(2, 512), positions=torch.zeros(2, dtype=torch.int64)),
                                 dict(kv=torch.zeros(2, 512), positions=torch.zeros(3, dtype=torch.int32)),
                                 dict(kv=torch.zeros(2, 512), kv_weight=torch.zeros(512, dtype=torch.float16)),
                                 dict(kv=torch.zeros(2, 512), kv_cache=torch.zeros(2, 64, 1, 384, dtype=torch.uint8))],
                         ids=["cpu", "fp64", "width", "q rank", "nothing", "columns", "int64 positions",
                              "positions length", "fp16 weight", "block of 64"])
def test_norm_rope_binding_refuses(lib, bad):  # noqa: F811
    with pytest.raises((ValueError, Q.QsfmError)):
        if "q" in bad:
            bad = dict(bad, q_out=torch.zeros(bad["q"].shape, dtype=torch.bfloat16))
        Q.make_norm_rope_params(**bad)


def test_block_table_binding_refuses(lib):  # noqa: F811
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    good = dict(block_table=i(2, 8), prev_lens=i(2), lens=i(2), free_list=i(16), free_count=i(1), slot_map=i(4))
    for change in (dict(prev_lens=i(3)), dict(free_count=i(2)), dict(block_table=i(8, 2).t()), dict(lens=i(2).long()),
                   dict(positions=i(5)), {}):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            Q.make_block_table_params(**dict(good, **change))
    with pytest.raises(ValueError):
        Q.update_block_tables(i(2, 8), i(2), i(2), i(16), i(1))  # neither slot_map nor max_rows


# ------------------------------------------------------------------ oracle
def test_e2m1_and_e4m3_tables():
    assert O.E2M1_TABLE.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, O.E4M3FN_TABLE[:127])


def test_hand_made_four_bit_row():
    row = np.zeros((1, 384), dtype=np.uint8)
    row[0, 0:4] = [0x80, 0x3F, 0x00, 0xC0]   # bf16 1.0, -2.0
    row[0, 128], row[0, 136] = 0x7F, 0x21    # codes 15, 7 (group 0) and 1, 2 (group 1)
    row[0, 352], row[0, 353] = 0x38, 0x40    # scales 1 and 2
    row[0, 380] = 126                        # 2^-1
    y = O.decode_rows(row, None)[0]
    assert y[0] == 1 and y[1] == -2
    assert y[64] == -3 and y[65] == 3 and y[80] == 0.5 and y[81] == 1.0
    assert np.count_nonzero(y) == 6


def test_generator_rows_are_the_oracles():
    """The seeded generator's quantiser and the oracle's, written apart, give
    the same bytes; halves of a step occur (bf16 inputs)."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 512, generator=g) * torch.logspace(-6, 3, 40)[:, None]
    x[7] = 0
    x[8, 64:80] = 0
    x = torch.cat((x, x.to(torch.bfloat16).float(), torch.randint(-12, 13, (40, 512), generator=g).float()))
    got = W._quantize_packed384_rows(x).numpy()
    for i in range(x.shape[0]):
        ref = C.pack384(x[i].double().numpy(), O.E2M1_TABLE[:8], O.E4M3FN_TABLE[:127])
        assert np.array_equal(O.decode_rows(got[i:i + 1], None), O.decode_rows(ref[None], None)), i
        assert np.array_equal(got[i, 352:], ref[352:]), i


def test_four_bit_rows_are_near_their_input():
    """|K~ - x| of a 4-bit element: half a step of its code times the scale,
    at most scale (between 4 and 6), plus what the scale's own rounding cuts
    off above 6: 6 * 2^-4 of it; amax / 6 within 2^-4 of the scale."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(64, 512, generator=g)
    y = O.decode_rows(W._quantize_packed384_rows(x).numpy(), None)
    x = x.double().numpy()
    assert np.abs(y[:, :64] - x[:, :64]).max() <= 2.0 ** -8 * np.abs(x[:, :64]).max()
    amax = np.repeat(np.abs(x[:, 64:].reshape(64, 28, 16)).max(2), 16, axis=1)
    assert np.all(np.abs(y[:, 64:] - x[:, 64:]) <= amax / 6 * (1 + 2.0 ** -4) + 1e-9)


def test_norm_rope_oracle_closed_forms():
    x = np.arange(1.0, 513.0)
    y = C.norm_rope(x, None, 0.0, True, None, None, 0, True)
    assert abs(np.mean(y * y) - 1) < 1e-12
    cos, sin = np.cos(np.linspace(0, 3, 32)), np.sin(np.linspace(0, 3, 32))
    for inter in (True, False):
        z = C.norm_rope(x, None, 0.0, False, cos, sin, 448, inter)
        back = C.norm_rope(z, None, 0.0, False, cos, -sin, 448, inter)
        assert np.allclose(back, x, atol=1e-9) and np.array_equal(z[:448], x[:448]) and not np.allclose(z, x)
    z = C.norm_rope(x, None, 0.0, False, np.zeros(32), np.ones(32), 0, True)  # a quarter turn
    assert np.array_equal(z[:4], [-2, 1, -4, 3])
    z = C.norm_rope(x, None, 0.0, False, np.zeros(32), np.ones(32), 0, False)
    assert np.array_equal(z[[0, 32]], [-33, 1])


def test_block_table_oracle_by_hand():
    table = np.array([[4, 5, -1], [6, -1, -1], [-1, -1, -1]], dtype=np.int32)
    free = np.array([0, 1, 2, 3, 9, 9, 9], dtype=np.int32)
    t, f, n, slots, pos, cu, res = C.block_tables(table, [200, 100, 0], [0, 130, 3], free, 4, 1, 40)
    # request 0 gives 4 and 5 back; request 1 takes 5, request 2 takes 4
    assert t[1].tolist() == [6, 5, -1] and t[2, 0] == 4 and n == 4 and f[:4].tolist() == [0, 1, 2, 3]
    assert slots[:33].tolist() == [6 * 128 + i for i in range(100, 128)] + [640, 641] + [512, 513, 514]
    assert pos[:33].tolist() == list(range(100, 130)) + [0, 1, 2] and set(slots[33:].tolist()) == {-1}
    assert cu.tolist() == [0, 0, 30, 33] and res.tolist() == [0, 0, 0]
    t, f, n, slots, pos, cu, res = C.block_tables(table, [200, 100, 0], [20, 100, 0], free, 4, 1, 0)
    assert n == 5 and f[:5].tolist() == [0, 1, 2, 3, 5]
