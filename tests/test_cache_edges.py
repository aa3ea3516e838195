"""The operators around the cache where a table, a batch or a script is not the
ordinary one (CPU): the oracle of block tables over columns and lists that hold
no block, calls without tokens, the entry script."""

import ast
import ctypes
import os

import numpy as np
import pytest

import compressed_mla_attention_gb300 as Q
from oracle import cache_oracle as C
from tests.test_abi import lib  # noqa: F401
from tests.test_cache_operators import norm_rope_valid

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ------------------------------------------------------------------ block tables
def test_oracle_gives_back_blocks_alone():
    """A short pool leaves -1 in the table; the request's end gives back the
    blocks that it has, and the next request takes one of them."""
    table, free = np.full((3, 2), -1, dtype=np.int32), np.array([5, -7, -7, -7, -7, -7], dtype=np.int32)
    table, free, n, slots, *_ = C.block_tables(table, [0, 0, 0], [128, 128, 0], free, 1, 1, 256)
    assert table[:2, 0].tolist() == [5, -1] and n == 0 and set(slots[128:].tolist()) == {-1}
    table, free, n, slots, *_ = C.block_tables(table, [128, 128, 0], [128, 0, 128], free, n, 1, 128)
    assert table[2, 0] == -1 and n == 0 and set(slots.tolist()) == {-1}  # request 1 had none to give
    table, free, n, slots, *_ = C.block_tables(table, [128, 0, 128], [0, 0, 0], free, n, 1, 0)
    assert n == 1 and free[0] == 5
    table, free, n, slots, *_ = C.block_tables(table, [0, 0, 0], [0, 3, 0], free, n, 1, 3)
    assert n == 0 and slots.tolist() == [640, 641, 642]


def test_oracle_gives_back_what_a_window_left():
    table, free = np.array([[-1, -1, -1, 7]], dtype=np.int32), np.array([0, 1, -7, -7, -7, -7, -7, -7], dtype=np.int32)
    _, f, n, *_ = C.block_tables(table, [500], [0], free, 2, 1, 0)
    assert n == 3 and f.tolist() == [0, 1, 7, -7, -7, -7, -7, -7]


def test_oracle_passes_no_foreign_id_on():
    """Ids outside the pool, in a column given back or on the list, are not blocks."""
    table, free = np.array([[3, 99], [-1, -1]], dtype=np.int32), np.array([1, 44, 0, 0], dtype=np.int32)
    t, f, n, slots, *_ = C.block_tables(table, [256, 0], [0, 256], free, 2, 1, 256)
    assert t[1].tolist() == [3, -1] and n == 1 and f[0] == 1
    assert slots[:128].tolist() == [3 * 128 + i for i in range(128)] and set(slots[128:].tolist()) == {-1}


# ------------------------------------------------------------------ calls without tokens
TOKEN_POINTERS = ("q", "q_out", "kv", "kv_out", "positions", "slot_map")


@pytest.mark.parametrize("change", [{}, dict(heads=0, q_weight=None), dict(kv_cache=None, kv_weight=None),
                                    dict(rope_dim=0, cos_sin=None)], ids=["all", "kv only", "q only", "norm only"])
def test_no_tokens_with_null_pointers(lib, change):  # noqa: F811
    """Empty tensors have null pointers: with no tokens nothing is asked of them."""
    p = norm_rope_valid(lib)
    for k, v in change.items():
        setattr(p, k, v)
    for f in TOKEN_POINTERS:
        setattr(p, f, None)
    p.tokens = 0
    assert lib.qsfm_norm_rope_store(ctypes.byref(p), None) == 0


@pytest.mark.parametrize("change,code", [(dict(dim=256), 2), (dict(in_type=3), 1), (dict(eps=-1.0), 1), (dict(heads=-1), 1),
                                         (dict(rope_dim=48), 2), (dict(rope_offset=480), 1)])
def test_no_tokens_with_bad_attributes(lib, change, code):  # noqa: F811
    p = norm_rope_valid(lib)
    p.tokens = 0
    for k, v in change.items():
        setattr(p, k, v)
    assert lib.qsfm_norm_rope_store(ctypes.byref(p), None) == code


# ------------------------------------------------------------------ the entry script
def test_the_entry_script_defines_all_before_it_runs():
    """Run as a script, the file calls smoke() in its last statement: what that
    calls has been defined by then."""
    body = ast.parse(open(os.path.join(ROOT, "__graft_entry__.py")).read()).body
    runs = [i for i, node in enumerate(body) if isinstance(node, ast.If) and "__main__" in ast.unparse(node.test)]
    assert runs == [len(body) - 1]
