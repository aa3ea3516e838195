"""fp64 CPU oracle of the operators around the cache: norm, rotation and
quantised store of rows, and block tables from request lengths.

TEST INFRASTRUCTURE, as the attention's oracle: only tests may import it, and
it shares no code with the library. Straight from the definitions in the C
header, with Python loops where an order is part of the definition.
"""

from __future__ import annotations

import numpy as np

DIM = 512
ROPE_DIM = 64
BLOCK = 128


def norm_rope(x, weight, eps, norm, cos, sin, offset, interleaved):
    """One row x [512] (fp64): x / sqrt(mean(x^2) + eps) * weight, then the
    elements from `offset` on rotated by cos / sin [rope_dim / 2]."""
    y = np.array(x, dtype=np.float64)
    if norm:
        y = y / np.sqrt(np.mean(y * y) + eps)
        if weight is not None:
            y = y * weight
    half = 0 if cos is None else len(cos)
    for i in range(half):
        a, b = (offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + half + i)
        ya, yb = y[a], y[b]
        y[a], y[b] = ya * cos[i] - yb * sin[i], yb * cos[i] + ya * sin[i]
    return y


def nearest(values, table):
    """Index of the table value nearest to each of `values`; on a tie the
    entry with the even index (the codes' last mantissa bit is the index's
    last bit)."""
    d = np.abs(np.asarray(values)[..., None] - table)
    best = d.min(axis=-1, keepdims=True)
    tied = d == best
    even = np.arange(len(table)) % 2 == 0
    first = np.argmax(tied, axis=-1)
    both = tied & even
    return np.where(both.any(axis=-1), np.argmax(both, axis=-1), first)


def pack384(y, e2m1, e4m3):
    """The 384 bytes of one finite row y [512] fp64 that fp32 holds exactly;
    e2m1 / e4m3: the formats' non-negative values by code."""
    out = np.zeros(384, dtype=np.uint8)
    out[:128] = bf16_bits(y[:64]).view(np.uint8)
    top = np.abs(y).max()
    e = int(np.clip(np.floor(np.log2(top)) - 10, -100, 100)) if top > 0 else -100
    codes = np.zeros(448, dtype=np.int64)
    for g in range(28):
        t = y[64 + 16 * g:80 + 16 * g]
        want = np.abs(t).max() / 6.0 * 2.0 ** -e
        c = int(nearest(min(want, 448.0), e4m3))
        out[352 + g] = c
        s = e4m3[c] * 2.0 ** e
        if s > 0:
            q = t / s
            codes[16 * g:16 * g + 16] = nearest(np.minimum(np.abs(q), 6.0), e2m1) + 8 * (np.signbit(q))
        # a group without a scale holds zeros
    out[128:352] = codes[0::2] + 16 * codes[1::2]
    out[380] = e + 127
    return out


def bf16_bits(x):
    """fp64 values to bf16 bit patterns (uint16), to nearest even."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def block_tables(table, prev_lens, lens, free_list, free_count, ratio, max_rows, num_blocks=None):
    """The state and the outputs after one step, request by request:
    (table, free_list, free_count, slot_map, positions, cu_rows, residual).
    What is not in [0, num_blocks) (default: the list's length) is no block: a
    column that holds such a thing gives nothing back, and what is taken from
    the list is then -1."""
    table, free_list = table.copy(), free_list.copy()
    blocks = len(free_list) if num_blocks is None else num_blocks
    before = [int(n) // ratio for n in prev_lens]
    after = [int(n) // ratio for n in lens]
    held = [-(-n // BLOCK) for n in before]
    need = [-(-n // BLOCK) for n in after]
    stack = [int(b) for b in free_list[:free_count]]
    for b in range(len(lens)):
        stack += [int(v) for v in table[b, need[b]:held[b]] if 0 <= v < blocks]
    for b in range(len(lens)):
        for c in range(held[b], need[b]):
            block = stack.pop() if stack else -1
            table[b, c] = block if 0 <= block < blocks else -1
    free_list[free_count:len(stack)] = stack[free_count:]
    slots, positions, cu = [], [], [0]
    for b in range(len(lens)):
        for row in range(before[b], after[b]):
            block = int(table[b, row // BLOCK])
            slots.append(block * BLOCK + row % BLOCK if 0 <= block < blocks else -1)
            positions.append(row * ratio)
        cu.append(len(slots))
    pad = max_rows - len(slots)
    i32 = lambda v: np.array(v, dtype=np.int32)  # noqa: E731
    return (table, free_list, len(stack), i32(slots + [-1] * pad), i32(positions + [-1] * pad), i32(cu),
            i32([int(n) % ratio for n in lens]))
