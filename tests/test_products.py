"""The 8-bit products on the CPU: struct layouts, refusals (every call below is
rejected before any CUDA call) and pins of their oracle."""

import ctypes

import numpy as np
import pytest
import torch

import compressed_mla_attention_gb300 as Q
from oracle import product_oracle as P
from oracle import qsfm_oracle as O
from tests.test_abi import lib  # noqa: F401
from tests.test_abi import test_struct_layout_matches_c as struct_layout

INVALID, UNSUPPORTED = 1, 2


@pytest.mark.parametrize("cls,cname", [(Q.QuantizeParams, "qsfm_quantize_params"), (Q.MatmulParams, "qsfm_matmul_params")])
def test_struct_layouts_match_c(tmp_path, cls, cname):
    struct_layout(tmp_path, cls, cname)


def test_defaults(lib):  # noqa: F811
    q, m = Q.QuantizeParams(), Q.MatmulParams()
    lib.qsfm_quantize_params_init(ctypes.byref(q))
    lib.qsfm_matmul_params_init(ctypes.byref(m))
    assert (q.heads, q.rows, q.x) == (1, 0, None) and (m.groups, m.rows, m.out_type, m.a) == (1, 0, 0, None)
    assert lib.qsfm_quantize_rows(None, None) == INVALID and lib.qsfm_scaled_matmul(None, None) == INVALID


# fake device addresses far enough apart that no two tensors overlap
X, GATE, INDEX, POS, TABLE, CODES, SCALE = (0x10000000 * (i + 1) for i in range(7))


def quantize_valid(lib):  # noqa: F811
    p = Q.QuantizeParams()
    lib.qsfm_quantize_params_init(ctypes.byref(p))
    p.rows, p.source_rows, p.heads, p.dim = 4, 4, 64, 512
    p.x_row_stride, p.x_head_stride = 64 * 512, 512
    p.rope_dim, p.rope_offset, p.max_positions = 64, 448, 100
    p.x, p.positions, p.cos_sin, p.codes, p.scale = X, POS, TABLE, CODES, SCALE
    return p


GATED = dict(gate=GATE, gate_row_stride=64 * 512, gate_head_stride=512, rope_dim=0, cos_sin=None, positions=None)
QUANTIZE = [
    ("negative rows", dict(rows=-1), INVALID),
    ("negative source rows", dict(source_rows=-1), INVALID),
    ("no heads", dict(heads=0), INVALID),
    ("no elements", dict(dim=0), INVALID),
    ("element type", dict(in_type=3), INVALID),
    ("K of 8", dict(heads=1, dim=8, rope_dim=0, rope_offset=0, cos_sin=None), UNSUPPORTED),
    ("heads of 64", dict(dim=64, rope_offset=0), UNSUPPORTED),
    ("too many groups", dict(rows=1 << 25, source_rows=1 << 25), UNSUPPORTED),
    ("K past 2^30", dict(heads=1 << 22), UNSUPPORTED),
    ("rope of 48", dict(rope_dim=48, rope_offset=0), UNSUPPORTED),
    ("rope of 256", dict(rope_dim=256, rope_offset=0), UNSUPPORTED),
    ("rope past the head", dict(rope_offset=512), INVALID),
    ("rope not at a multiple", dict(rope_offset=32), UNSUPPORTED),
    ("negative offset", dict(rope_offset=-64), INVALID),
    ("no codes", dict(codes=None), INVALID),
    ("no scale", dict(scale=None), INVALID),
    ("no x", dict(x=None), INVALID),
    ("source rows without an index", dict(source_rows=5), INVALID),
    ("no table", dict(cos_sin=None), INVALID),
    ("empty table", dict(max_positions=0), INVALID),
    ("no positions", dict(positions=None), INVALID),
    ("table without rope", dict(rope_dim=0), INVALID),
    ("gate and rope", dict(gate=GATE, gate_row_stride=64 * 512, gate_head_stride=512), INVALID),
    ("stride of 4 bytes", dict(x_head_stride=514), INVALID),
    ("negative stride", dict(x_row_stride=-512), INVALID),
    ("stride past 2^31", dict(x_row_stride=1 << 31), UNSUPPORTED),
    ("gate's stride", dict(GATED, gate_row_stride=514), INVALID),
    ("gate's negative stride", dict(GATED, gate_head_stride=-512), INVALID),
    ("x not 16-byte aligned", dict(x=X + 8), INVALID),
    ("codes not 16-byte aligned", dict(codes=CODES + 8), INVALID),
    ("table not 16-byte aligned", dict(cos_sin=TABLE + 4), INVALID),
    ("scale not 4-byte aligned", dict(scale=SCALE + 2), INVALID),
    ("index not 4-byte aligned", dict(row_index=INDEX + 1), INVALID),
    ("codes over x", dict(codes=X + 4096), INVALID),
    ("scale over the positions", dict(scale=POS), INVALID),
    ("scale over the codes", dict(scale=CODES + 64), INVALID),
    ("codes over the gate", dict(GATED, codes=GATE), INVALID),
]


@pytest.mark.parametrize("why,change,code", QUANTIZE, ids=[c[0] for c in QUANTIZE])
def test_quantize_refusals(lib, why, change, code):  # noqa: F811
    p = quantize_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    assert lib.qsfm_quantize_rows(ctypes.byref(p), None) == code


@pytest.mark.parametrize("change", [{}, GATED, dict(row_index=INDEX, source_rows=2), dict(heads=1, dim=16, rope_dim=0, rope_offset=0, cos_sin=None)],
                         ids=["rotation", "gate", "index", "16 elements"])
def test_quantize_valid_calls_pass_the_checks(lib, change):  # noqa: F811
    """With no rows a valid call returns before anything is launched."""
    p = quantize_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    p.rows = p.source_rows = 0
    assert lib.qsfm_quantize_rows(ctypes.byref(p), None) == 0


A, AS, W, WS, CU, OUT = (0x10000000 * (i + 1) for i in range(6))


def matmul_valid(lib):  # noqa: F811
    p = Q.MatmulParams()
    lib.qsfm_matmul_params_init(ctypes.byref(p))
    p.rows, p.n, p.k, p.groups = 40, 200, 1040, 3
    p.a_row_stride, p.w_row_stride, p.w_group_stride, p.out_row_stride = 1040, 1040, 1040 * 200, 200
    p.a_scale_row_stride, p.a_scale_col_stride = 9, 1
    p.a, p.a_scale, p.w, p.w_scale, p.cu_rows, p.out = A, AS, W, WS, CU, OUT
    return p


MATMUL = [
    ("negative rows", dict(rows=-1), INVALID),
    ("no columns", dict(n=0), INVALID),
    ("no elements", dict(k=0), INVALID),
    ("no groups", dict(groups=0), INVALID),
    ("output type", dict(out_type=3), INVALID),
    ("K of 1032", dict(k=1032), UNSUPPORTED),
    ("1025 groups", dict(groups=1025), UNSUPPORTED),
    ("2^24 rows", dict(rows=1 << 24), UNSUPPORTED),
    ("2^24 columns", dict(n=1 << 24), UNSUPPORTED),
    ("K of 2^24", dict(k=1 << 24), UNSUPPORTED),
    ("too many tiles", dict(rows=(1 << 24) - 1, n=(1 << 24) - 1), UNSUPPORTED),
    ("groups without cu_rows", dict(cu_rows=None), INVALID),
    ("no a", dict(a=None), INVALID),
    ("no a_scale", dict(a_scale=None), INVALID),
    ("no w", dict(w=None), INVALID),
    ("no w_scale", dict(w_scale=None), INVALID),
    ("no out", dict(out=None), INVALID),
    ("a not 16-byte aligned", dict(a=A + 8), INVALID),
    ("w not 16-byte aligned", dict(w=W + 8), INVALID),
    ("out not aligned to its elements", dict(out=OUT + 1), INVALID),
    ("fp32 out not aligned", dict(out=OUT + 2, out_type=2), INVALID),
    ("a_scale not aligned", dict(a_scale=AS + 2), INVALID),
    ("cu_rows not aligned", dict(cu_rows=CU + 2), INVALID),
    ("rows of a that overlap", dict(a_row_stride=1024), INVALID),
    ("rows of a at 1048 bytes", dict(a_row_stride=1048), INVALID),
    ("matrices that overlap", dict(w_group_stride=1040 * 199), INVALID),
    ("rows of w that overlap", dict(w_row_stride=16), INVALID),
    ("negative stride of a_scale", dict(a_scale_row_stride=-1), INVALID),
    ("rows of out that overlap", dict(out_row_stride=199), INVALID),
    ("a stride of 2^37", dict(w_group_stride=1 << 37), UNSUPPORTED),
    ("a scale stride of 2^36", dict(a_scale_row_stride=1 << 36), UNSUPPORTED),
    ("out over a", dict(out=A + 1024), INVALID),
    ("out over the matrices", dict(out=W + 2 * 1040 * 200), INVALID),
    ("out over a_scale", dict(out=AS + 64), INVALID),
    ("out over w_scale", dict(out=WS), INVALID),
    ("out over cu_rows", dict(out=CU + 12), INVALID),
]


@pytest.mark.parametrize("why,change,code", MATMUL, ids=[c[0] for c in MATMUL])
def test_matmul_refusals(lib, why, change, code):  # noqa: F811
    p = matmul_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    assert lib.qsfm_scaled_matmul(ctypes.byref(p), None) == code


def test_matmul_without_rows(lib):  # noqa: F811
    p = matmul_valid(lib)
    p.rows, p.a, p.out = 0, None, None
    assert lib.qsfm_scaled_matmul(ctypes.byref(p), None) == 0


def test_quantize_binding_refuses(lib):  # noqa: F811
    z, u8 = torch.zeros, torch.uint8
    good = dict(x=z(4, 256, dtype=torch.bfloat16), codes=z(4, 256, dtype=u8), scale=z(4, 2))
    i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    for change in (dict(x=z(4, 256, dtype=torch.float64)), dict(x=z(4)), dict(x=z(256, 4).t()),
                   dict(gate=z(4, 256)), dict(gate=z(4, 128, dtype=torch.bfloat16)), dict(codes=z(4, 255, dtype=u8)),
                   dict(codes=z(4, 256, dtype=torch.int8)), dict(scale=z(4, 3)), dict(scale=z(2, 4).t()),
                   dict(row_index=i(5)), dict(positions=i(3)), dict(positions=i(4).long()), dict(cos_sin=z(10)),
                   {}):  # the last: not on a CUDA device
        with pytest.raises(ValueError):
            Q.make_quantize_params(**dict(good, **change))


def test_matmul_binding_refuses(lib):  # noqa: F811
    z, u8 = torch.zeros, torch.uint8
    good = dict(a=z(5, 256, dtype=u8), a_scale=z(5, 2), w=z(130, 256, dtype=u8), w_scale=z(2, 2), out=z(5, 130))
    grouped = dict(good, w=z(3, 130, 256, dtype=u8), w_scale=z(3, 2, 2), cu_rows=z(4, dtype=torch.int32))
    for base, change in ((good, dict(a=z(5, 256))), (good, dict(a=z(5, 1, 256, dtype=u8))), (good, dict(w=z(130, 128, dtype=u8))),
                         (good, dict(a=z(256, 5, dtype=u8).t())), (good, dict(a_scale=z(5, 3))), (good, dict(w_scale=z(3, 2))),
                         (good, dict(out=z(5, 131))), (good, dict(out=z(5, 130, dtype=torch.float64))),
                         (good, dict(w=z(3, 130, 256, dtype=u8))), (good, dict(out=z(130, 5).t())), (good, {}),
                         (grouped, dict(w=z(130, 256, dtype=u8))), (grouped, dict(cu_rows=z(3, dtype=torch.int32))),
                         (grouped, dict(cu_rows=z(4, dtype=torch.int64))), (grouped, dict(w_scale=z(2, 2))), (grouped, {})):
        with pytest.raises(ValueError):
            Q.make_matmul_params(**dict(base, **change))
    with pytest.raises(ValueError):
        Q.scaled_matmul(good["a"], good["a_scale"], good["w"], good["w_scale"], out=good["out"], out_dtype=torch.bfloat16)


# ------------------------------------------------------------------ oracle
def test_e4m3_rounding_is_the_tables():
    """Every code's value stays, every border goes to the even code, what lies on
    either side of it to its own."""
    v = O.E4M3FN_TABLE[:127]
    assert np.array_equal(P.e4m3(v), v) and np.array_equal(P.e4m3(-v), -v)
    mid = (v[1:] + v[:-1]) / 2
    even = np.where(np.arange(126) % 2 == 0, v[:-1], v[1:])
    assert np.array_equal(P.e4m3(mid), even)
    assert np.array_equal(P.e4m3(mid * (1 + 1e-12)), v[1:]) and np.array_equal(P.e4m3(mid * (1 - 1e-12)), v[:-1])
    assert P.e4m3(460.0) == 448 and P.e4m3(-1e9) == -448


def test_quantize_oracle_by_hand():
    y = np.zeros((1, 144))
    y[0, 3], y[0, 7], y[0, 130] = 448.0, -17.0, 3.5
    codes, scales = P.quantize(y, False)
    # -17 lies between -16 and -18: the even code
    assert scales.tolist() == [[1.0, 3.5 / 448]] and codes[0, 3] == 448 and codes[0, 7] == -16 and codes[0, 130] == 448
    codes, scales = P.quantize(y, True)
    assert scales.tolist() == [[1.0, 2.0 ** -7]] and codes[0, 130] == 448
    codes, scales = P.quantize(y * 1.001, True)
    assert scales.tolist() == [[2.0, 2.0 ** -6]] and codes[0, 130] == 224
    y[0, 5] = np.inf
    codes, scales = P.quantize(y, False)
    assert np.isnan(codes[0, :128]).all() and np.isnan(scales[0, 0]) and codes[0, 130] == 448
    codes, scales = P.quantize(np.zeros((2, 128)), False)
    assert not codes.any() and np.all(scales == 1e-12 / 448)


def test_turn_oracle_turns_back():
    r = np.random.RandomState(0)
    y, angle = r.randn(5, 3, 256), r.rand(5, 32) * 7
    for inter in (True, False):
        z = P.turn(y, np.cos(angle), np.sin(angle), 128, inter, False)
        assert np.array_equal(z[:, :, :128], y[:, :, :128]) and not np.allclose(z[:, :, 128:192], y[:, :, 128:192])
        assert np.allclose(P.turn(z, np.cos(angle), np.sin(angle), 128, inter, True), y)
        assert np.allclose((z ** 2).sum(2), (y ** 2).sum(2))
    quarter = P.turn(np.arange(1.0, 129.0).reshape(1, 1, 128), np.zeros((1, 32)), np.ones((1, 32)), 0, True, False)
    assert quarter[0, 0, :4].tolist() == [-2, 1, -4, 3]


def test_product_oracle_is_the_dense_product():
    r = np.random.RandomState(1)
    a, w = r.randint(-5, 6, (7, 300)).astype(float), r.randint(-5, 6, (200, 300)).astype(float)
    sa, sw = r.rand(7, 3), r.rand(2, 3)
    dense = (a * np.repeat(sa, 128, 1)[:, :300]) @ (w * np.repeat(np.repeat(sw, 128, 0), 128, 1)[:200, :300]).T
    out, mag = P.product(a, sa, w, sw)
    assert np.allclose(out, dense) and np.all(mag >= np.abs(out) * (1 - 1e-12))
    got, _ = P.grouped(a, sa, np.stack([w, -w, w]), np.stack([sw] * 3), [1, 3, 3, 6], np.full((7, 200), 9.0))
    assert np.all(got[[0, 6]] == 9) and np.allclose(got[1:6], dense[1:6])
