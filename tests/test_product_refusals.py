"""Refusals of the 8-bit products' binding on the CPU, each by its own check: the tensors
stand for tensors of one CUDA device, so that the unchanged block is accepted."""

import ctypes
import os
import re

import pytest
import torch

import compressed_mla_attention_gb300 as Q
from tests.test_abi import lib  # noqa: F401

U8, I32, BF16 = torch.uint8, torch.int32, torch.bfloat16


@pytest.fixture
def accept(monkeypatch, lib):  # noqa: F811
    monkeypatch.setattr(Q, "_one_device", lambda tensors: torch.device("cuda", 0))


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def rows():
    return dict(x=z(4, 256, dtype=BF16), codes=z(4, 256, dtype=U8), scale=z(4, 2))


def heads():
    return dict(x=z(4, 2, 256, dtype=BF16), codes=z(4, 2, 256, dtype=U8), scale=z(4, 4), gate=None,
                row_index=None, positions=z(4, dtype=I32), cos_sin=z(9, 64))


QUANTIZE = {
    "x type": (rows, dict(x=z(4, 256, dtype=torch.float64)), "x and gate must have one type"),
    "x of one axis": (rows, dict(x=z(4, dtype=BF16)), "x has shape"),
    "x of four axes": (rows, dict(x=z(4, 1, 1, 256, dtype=BF16)), "x has shape"),
    "x by columns": (rows, dict(x=z(256, 4, dtype=BF16).t()), "x must have contiguous rows"),
    "gate type": (rows, dict(gate=z(4, 256)), "x and gate must have one type"),
    "gate shape": (rows, dict(gate=z(4, 128, dtype=BF16)), "gate has shape"),
    "gate with heads": (rows, dict(gate=z(4, 2, 128, dtype=BF16)), "gate has shape"),
    "gate by columns": (rows, dict(gate=z(256, 4, dtype=BF16).t()), "gate must have contiguous rows"),
    "codes width": (rows, dict(codes=z(4, 255, dtype=U8)), "codes has shape"),
    "codes rows": (rows, dict(codes=z(3, 256, dtype=U8)), "codes has shape"),
    "codes type": (rows, dict(codes=z(4, 256, dtype=torch.int8)), "codes has type"),
    "codes strided": (rows, dict(codes=z(4, 512, dtype=U8)[:, :256]), "codes must be contiguous"),
    "codes of other heads": (heads, dict(codes=z(4, 4, 128, dtype=U8)), "codes has shape"),
    "scale width": (rows, dict(scale=z(4, 3)), "scale has shape"),
    "scale rows": (rows, dict(scale=z(5, 2)), "scale has shape"),
    "scale type": (rows, dict(scale=z(4, 2, dtype=torch.float64)), "scale has type"),
    "scale by columns": (rows, dict(scale=z(2, 4).t()), "scale must be contiguous"),
    "index type": (rows, dict(row_index=z(4, dtype=torch.int64)), "row_index has type"),
    "index of two axes": (rows, dict(row_index=z(4, 1, dtype=I32)), "row_index has shape"),
    "index strided": (rows, dict(row_index=z(8, dtype=I32)[::2]), "row_index must be contiguous"),
    "more indexes than codes": (rows, dict(row_index=z(5, dtype=I32)), "codes has shape"),
    "positions count": (heads, dict(positions=z(3, dtype=I32)), "positions has shape"),
    "positions type": (heads, dict(positions=z(4, dtype=torch.int64)), "positions has type"),
    "positions strided": (heads, dict(positions=z(8, dtype=I32)[::2]), "positions must be contiguous"),
    "table of one axis": (heads, dict(cos_sin=z(64)), "cos_sin has shape"),
    "table type": (heads, dict(cos_sin=z(9, 64, dtype=BF16)), "cos_sin has type"),
    "table strided": (heads, dict(cos_sin=z(9, 128)[:, :64]), "cos_sin must be contiguous"),
}


def product():
    return dict(a=z(5, 256, dtype=U8), a_scale=z(5, 2), w=z(130, 256, dtype=U8), w_scale=z(2, 2), out=z(5, 130))


def grouped():
    return dict(product(), w=z(3, 130, 256, dtype=U8), w_scale=z(3, 2, 2), cu_rows=z(4, dtype=I32))


MATMUL = {
    "a type": (product, dict(a=z(5, 256)), "a has type"),
    "w type": (product, dict(w=z(130, 256, dtype=torch.int8)), "w has type"),
    "a of three axes": (product, dict(a=z(5, 1, 256, dtype=U8)), r"a must be \[M, K\]"),
    "w of another K": (product, dict(w=z(130, 128, dtype=U8)), r"w must be \[N, K\] with K = 256"),
    "w with groups": (product, dict(w=z(3, 130, 256, dtype=U8)), r"w must be \[N, K\]"),
    "a by columns": (product, dict(a=z(256, 5, dtype=U8).t()), "a must have contiguous rows"),
    "w by columns": (product, dict(w=z(256, 130, dtype=U8).t()), "w must have contiguous rows"),
    "out by columns": (product, dict(out=z(130, 5).t()), "out must have contiguous rows"),
    "a_scale width": (product, dict(a_scale=z(5, 3)), r"a_scale must be float32 \[5, 2\]"),
    "a_scale rows": (product, dict(a_scale=z(4, 2)), r"a_scale must be float32 \[5, 2\]"),
    "a_scale type": (product, dict(a_scale=z(5, 2, dtype=BF16)), r"a_scale must be float32 \[5, 2\]"),
    "w_scale shape": (product, dict(w_scale=z(3, 2)), "w_scale has shape"),
    "w_scale type": (product, dict(w_scale=z(2, 2, dtype=BF16)), "w_scale has type"),
    "w_scale by columns": (product, dict(w_scale=z(2, 2).t()), "w_scale must be contiguous"),
    "out width": (product, dict(out=z(5, 131)), r"out must be .* \[5, 130\]"),
    "out rows": (product, dict(out=z(4, 130)), r"out must be .* \[5, 130\]"),
    "out type": (product, dict(out=z(5, 130, dtype=torch.float64)), r"out must be .* \[5, 130\]"),
    "groups without an axis": (grouped, dict(w=z(130, 256, dtype=U8)), r"w must be \[groups, N, K\]"),
    "grouped w_scale": (grouped, dict(w_scale=z(2, 2)), "w_scale has shape"),
    "w_scale of fewer groups": (grouped, dict(w_scale=z(2, 2, 2)), "w_scale has shape"),
    "cu_rows count": (grouped, dict(cu_rows=z(3, dtype=I32)), "cu_rows has shape"),
    "cu_rows type": (grouped, dict(cu_rows=z(4, dtype=torch.int64)), "cu_rows has type"),
    "cu_rows strided": (grouped, dict(cu_rows=z(8, dtype=I32)[::2]), "cu_rows must be contiguous"),
}


@pytest.mark.parametrize("name", sorted(QUANTIZE))
def test_quantize_binding_refuses_by_its_own_check(accept, name):
    base, change, message = QUANTIZE[name]
    Q.make_quantize_params(**base())
    with pytest.raises(ValueError, match="^" + message):
        Q.make_quantize_params(**dict(base(), **change))


@pytest.mark.parametrize("name", sorted(MATMUL))
def test_matmul_binding_refuses_by_its_own_check(accept, name):
    base, change, message = MATMUL[name]
    Q.make_matmul_params(**base())
    with pytest.raises(ValueError, match="^" + message):
        Q.make_matmul_params(**dict(base(), **change))


@pytest.mark.parametrize("make,base", [(Q.make_quantize_params, rows), (Q.make_matmul_params, product), (Q.make_matmul_params, grouped)],
                         ids=["quantize", "product", "grouped"])
def test_tensors_outside_a_device_are_refused(lib, make, base):  # noqa: F811
    with pytest.raises(ValueError, match="every tensor must be on one CUDA device"):
        make(**base())


def test_output_of_another_type_than_asked_for_is_refused(accept):
    p = product()
    with pytest.raises(ValueError, match="^out has type torch.float32, not torch.bfloat16"):
        Q.scaled_matmul(p["a"], p["a_scale"], p["w"], p["w_scale"], out=p["out"], out_dtype=BF16)


def test_block_holds_what_it_was_given(accept):
    """The sizes, strides and pointers that reach the library."""
    wide = z(7, 640, dtype=BF16)
    x, gate = wide[::2, :256], wide[::2, 384:]
    p = Q.make_quantize_params(x=x, gate=gate, codes=z(5, 256, dtype=U8), scale=z(5, 2), row_index=z(5, dtype=I32), pow2_scale=True).params
    assert (p.rows, p.source_rows, p.heads, p.dim, p.in_type, p.pow2_scale, p.rope_dim) == (5, 4, 1, 256, Q.ELEM_TYPE["torch.bfloat16"], 1, 0)
    assert (p.x_row_stride, p.x_head_stride, p.gate_row_stride, p.gate_head_stride) == (1280, 0, 1280, 0)
    assert (p.x, p.gate) == (x.data_ptr(), gate.data_ptr()) and p.positions is None and p.cos_sin is None
    h = heads()
    p = Q.make_quantize_params(**h, rope_offset=192, interleaved=False, inverse=True).params
    assert (p.rows, p.source_rows, p.heads, p.dim, p.rope_dim, p.rope_offset, p.interleaved, p.inverse, p.max_positions) == (4, 4, 2, 256, 64, 192, 0, 1, 9)
    g = grouped()
    out, scale = z(5, 200)[:, 3:133], z(2, 9)[:, :5].t()
    p = Q.make_matmul_params(**dict(g, out=out, a_scale=scale, a=z(5, 512, dtype=U8)[:, 256:])).params
    assert (p.rows, p.n, p.k, p.groups, p.out_type) == (5, 130, 256, 3, Q.ELEM_TYPE["torch.float32"])
    assert (p.a_row_stride, p.w_row_stride, p.w_group_stride, p.a_scale_row_stride, p.a_scale_col_stride, p.out_row_stride) == \
        (512, 256, 130 * 256, 1, 9, 200)
    assert p.out == out.data_ptr() and p.cu_rows == g["cu_rows"].data_ptr()


def test_plan_query_refuses(lib):  # noqa: F811
    """As the product itself, before any CUDA call; and without rows or a place for the answer."""
    from tests.test_products import matmul_valid

    out = [ctypes.c_int32() for _ in range(3)]
    refs = [ctypes.byref(v) for v in out]
    assert lib.qsfm_debug_matmul_plan(None, *refs) == 1
    p = matmul_valid(lib)
    for i in range(3):
        assert lib.qsfm_debug_matmul_plan(ctypes.byref(p), *(None if j == i else refs[j] for j in range(3))) == 1
    p.k = 1032
    assert lib.qsfm_debug_matmul_plan(ctypes.byref(p), *refs) == 2
    p = matmul_valid(lib)
    p.rows = 0
    assert lib.qsfm_debug_matmul_plan(ctypes.byref(p), *refs) == 1


@pytest.mark.parametrize("rows,n,groups,code", [((1 << 24) - 1, 1 << 18, 1, 1), (1 << 20, 1 << 23, 1, 1), (1 << 20, 1 << 23, 1024, 1),
                                                (1, (1 << 24) - 1, 1024, 1), (1 << 21, 1 << 23, 1, 2), ((1 << 24) - 1, 1 << 20, 1, 2)])
def test_sizes_are_limited_by_the_smallest_tiles(lib, rows, n, groups, code):  # noqa: F811
    """2^30 tiles of 128 x 128 outputs, and one for each group beside: more is not
    supported, less goes on to the next check (here of pointers that are not there)."""
    from tests.test_products import matmul_valid

    p = matmul_valid(lib)
    p.rows, p.n, p.groups, p.a = rows, n, groups, None
    assert lib.qsfm_scaled_matmul(ctypes.byref(p), None) == code


def test_weights_quantised_as_the_usage_text_does():
    """The README's function: codes and scales of its 128 x 128 elements, the last ones fewer."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    names = {"torch": torch}
    exec(re.search(r"```python\n(def quantised_matrix.*?)```", text, re.S).group(1), names)
    w = torch.randn(200, 400, generator=torch.Generator().manual_seed(0))
    w[129, 300] = 50.0
    codes, scale = names["quantised_matrix"](w.to(BF16))
    assert codes.shape == (200, 400) and scale.shape == (2, 4) and codes.is_contiguous() and scale.is_contiguous()
    wide = scale.repeat_interleave(128, 0)[:200].repeat_interleave(128, 1)[:, :400]
    assert scale[1, 2] == 50.0 / 448 and codes[129, 300].float() == 448
    # half a step of 3 bits, relative, or of the least step 2^-9, and the division's rounding
    assert torch.all((codes.float() * wide - w.to(BF16).float()).abs() <= (2.0 ** -4 * w.abs() + 2.0 ** -10 * wide) * (1 + 2.0 ** -7))
