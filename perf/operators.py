"""The calls of a serving step around the attention's cache: block tables and slots from the
requests' lengths, normed and rotated queries and cache rows, and attention over 4-bit cache rows.

Each case is one call of one operator. `run` computes it with elementary torch operations in 32
bits (`own` false) or by this package's kernels (`own` true); `exact` computes it in 64 bits.

A packed384 cache row holds the 512 elements of one token: 64 bf16 (bytes 0..127), 448 e2m1 codes
(bytes 128..351, low nibble first), 28 e4m3 scales, one per 16 codes (bytes 352..379), the row's
e8m0 exponent (byte 380) and three zero bytes. An element of the second part is
code * scale * 2^(exponent - 127).
"""

import math
import random

import torch

own = False

BLOCK = 128
DIM = 512
ROPE = 64
WINDOW = 128


def listed():
    return [
        # the smallest decode step of the bench: two requests, one token each
        {"name": "attn_tiny", "op": "attn", "layout": "BSND", "batch": 2, "s1_lo": 1, "s1_hi": 1, "s2_lo": 4096,
         "s2_hi": 4096, "mode": "CSA", "ratio": 4, "k2": 512, "valid": 384, "heads": 64, "padded": False, "lens_seed": 0},
        # the bench's flagship: a decode batch of 128 requests, two tokens each
        {"name": "attn_decode", "op": "attn", "layout": "BSND", "batch": 128, "s1_lo": 2, "s1_hi": 2, "s2_lo": 4096,
         "s2_hi": 65536, "mode": "CSA", "ratio": 4, "k2": 512, "valid": 512, "heads": 64, "padded": False, "lens_seed": 2},
        # the long decode: every compressed row of 32K to 128K tokens, tokens split over the SMs
        {"name": "attn_long", "op": "attn", "layout": "BSND", "batch": 64, "s1_lo": 1, "s1_hi": 1, "s2_lo": 32768,
         "s2_hi": 131072, "mode": "HCA", "ratio": 128, "k2": 0, "valid": 0, "heads": 64, "padded": False, "lens_seed": 3},
        # prefill of four whole prompts with the window alone
        {"name": "attn_window", "op": "attn", "layout": "TND", "batch": 4, "s1_lo": 2048, "s1_hi": 2048, "s2_lo": 2048,
         "s2_hi": 2048, "mode": "SWA", "ratio": 1, "k2": 0, "valid": 0, "heads": 64, "padded": False, "lens_seed": 1},
        # ragged prefill chunks of requests with a history, 128 heads
        {"name": "attn_chunks", "op": "attn", "layout": "TND", "batch": 5, "s1_lo": 301, "s1_hi": 701, "s2_lo": 8192,
         "s2_hi": 32768, "mode": "CSA", "ratio": 4, "k2": 512, "valid": 512, "heads": 128, "padded": False, "lens_seed": 4},
        # one token: what a single stream waits for
        {"name": "rows_single", "op": "rows", "tokens": 1, "heads": 64, "format": "packed384", "pairs": "adjacent",
         "rope_at": 0, "dtype": "bfloat16", "fused": False, "weights": "float32", "padded": 0},
        # the decode batch's 256 tokens, q and kv in one projection's output
        {"name": "rows_decode", "op": "rows", "tokens": 256, "heads": 64, "format": "packed384", "pairs": "adjacent",
         "rope_at": 0, "dtype": "bfloat16", "fused": True, "weights": "bfloat16", "padded": 0},
        # a prefill step of 128-head queries into 8-bit rows, the last tokens of it padding
        {"name": "rows_prefill", "op": "rows", "tokens": 4099, "heads": 128, "format": "packed640", "pairs": "halves",
         "rope_at": 448, "dtype": "bfloat16", "fused": False, "weights": "float32", "padded": 37},
        # the compressed rows of a long prompt: rows only, no queries
        {"name": "rows_compressed", "op": "rows", "tokens": 8191, "heads": 0, "format": "fp8_fp32_scales",
         "pairs": "adjacent", "rope_at": 0, "dtype": "float32", "fused": False, "weights": "float32", "padded": 0},
        # tables of two requests that grow by one token
        {"name": "tables_tiny", "op": "tables", "batch": 2, "len_hi": 4096, "new_lo": 1, "new_hi": 1, "ratio": 1},
        # compressed rows of the decode batch: two tokens each, some requests end, some begin
        {"name": "tables_decode", "op": "tables", "batch": 128, "len_hi": 65536, "new_lo": 2, "new_hi": 2, "ratio": 4},
        # a large prefill step: chunks of half a million tokens
        {"name": "tables_prefill", "op": "tables", "batch": 500, "len_hi": 131072, "new_lo": 1, "new_hi": 2047, "ratio": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn", "attn", "rows", "rows", "tables"))
    if op == "attn":
        mode, heads = rng.choice(("CSA", "CSA", "HCA", "SWA")), rng.choice((64, 64, 128))
        ratio = 1 if mode == "SWA" else rng.choice((64, 128)) if mode == "HCA" else rng.choice((4, 8))
        k2 = rng.choice((512, 512, 100, 1024)) if mode == "CSA" else 0
        if rng.random() < 0.5:  # decode
            batch, s1 = _log(rng, 1, 200), rng.choice((1, 1, 2, 3))
            lo = _log(rng, 1, 30000)
            hi = _log(rng, lo, 65000)
            return {"op": "attn", "layout": "BSND", "batch": batch, "s1_lo": s1, "s1_hi": s1, "s2_lo": max(lo, s1),
                    "s2_hi": max(hi, s1), "mode": mode, "ratio": ratio, "k2": k2, "valid": k2, "heads": heads,
                    "padded": s1 > 1 and rng.random() < 0.3, "lens_seed": rng.randrange(1 << 20)}
        batch, hi = rng.randint(1, 6), _log(rng, 20, 350)  # chunks of requests, most with a history
        lo = rng.randint(1, hi)
        return {"op": "attn", "layout": "TND", "batch": batch, "s1_lo": lo, "s1_hi": hi, "s2_lo": hi,
                "s2_hi": _log(rng, hi, 20000), "mode": mode, "ratio": ratio, "k2": min(k2, 512), "valid": min(k2, 512),
                "heads": heads, "padded": False, "lens_seed": rng.randrange(1 << 20)}
    if op == "rows":
        heads = rng.choice((0, 64, 64, 128))
        tokens = _log(rng, 1, 4000)
        return {"op": "rows", "tokens": tokens, "heads": heads,
                "format": rng.choice(("packed384", "packed640", "fp8_fp32_scales", "bf16")),
                "pairs": rng.choice(("adjacent", "halves")), "rope_at": rng.choice((0, 448)),
                "dtype": rng.choice(("bfloat16", "bfloat16", "float16", "float32")) if heads < 128 else "bfloat16",
                "fused": heads > 0 and rng.random() < 0.5, "weights": rng.choice(("float32", "bfloat16")),
                "padded": rng.choice((0, tokens // 9))}
    ratio = rng.choice((1, 1, 4, 128))
    new = _log(rng, 1, 1500)
    return {"op": "tables", "batch": _log(rng, 1, 500), "len_hi": _log(rng, 2000, 131072), "new_lo": rng.randint(1, new),
            "new_hi": new, "ratio": ratio}


# ------------------------------------------------------------------ packed384 rows
def _e2m1(r):
    """The nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 to each |r|, ties to the even code: codes with the sign bit."""
    a = r.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * (r < 0).int()


def _pack384(y):
    """fp32 rows [n, 512] as packed384 bytes [n, 384]."""
    n = y.shape[0]
    amax = y.abs().amax(1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 11, -100).clamp(-100, 100)
    one = torch.ones_like(amax)
    t = y[:, ROPE:].reshape(n, 28, 16)
    s8 = (torch.ldexp(one, -e)[:, None] * (t.abs().amax(2) / 6)).to(torch.float8_e4m3fn)
    s = s8.float() * torch.ldexp(one, e)[:, None]
    r = torch.where(s[:, :, None] > 0, t / s[:, :, None], torch.zeros_like(t))
    c = _e2m1(r).reshape(n, 224, 2)
    out = torch.zeros(n, 384, dtype=torch.uint8, device=y.device)
    out[:, :128] = y[:, :ROPE].to(torch.bfloat16).contiguous().view(torch.uint8)
    out[:, 128:352] = (c[:, :, 0] + 16 * c[:, :, 1]).to(torch.uint8)
    out[:, 352:380] = s8.view(torch.uint8)
    out[:, 380] = (e + 127).to(torch.uint8)
    return out


def _unpack384(raw, dtype):
    """packed384 bytes [..., 384] as values [..., 512] of `dtype`."""
    c = raw[..., 128:352].to(torch.int32)
    c = torch.stack((c % 16, c // 16), -1).flatten(-2)
    m = c % 8
    v = torch.where(m < 2, 0.5 * m, torch.where(m % 2 == 0, 1.0, 1.5) * torch.exp2((m // 2 - 1).to(dtype))).to(dtype)
    v = torch.where(c >= 8, -v, v)
    s = raw[..., 352:380].contiguous().view(torch.float8_e4m3fn).to(dtype)
    s = s * torch.exp2(raw[..., 380:381].to(dtype) - 127)
    v = (v.unflatten(-1, (28, 16)) * s[..., None]).flatten(-2)
    return torch.cat((raw[..., :128].contiguous().view(torch.bfloat16).to(dtype), v), -1)


# ------------------------------------------------------------------ attention
def _lengths(case):
    """Query tokens and history (with them) of each request; every seed has the same lengths."""
    r = random.Random(case["lens_seed"])
    s1 = [r.randint(case["s1_lo"], case["s1_hi"]) for _ in range(case["batch"])]
    s2 = [max(n, r.randint(case["s2_lo"], case["s2_hi"])) for n in s1]
    return s1, s2


def _pool(bank, blocks, g):
    pick = torch.randint(0, bank.shape[0], (max(blocks, 1) * BLOCK,), generator=g, device="cuda")
    return bank[pick].view(max(blocks, 1), BLOCK, 1, 384)


def _prepare_attn(case, g):
    s1, s2 = _lengths(case)
    batch, r, heads, total = case["batch"], case["ratio"], case["heads"], sum(s1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"q": torch.randn(total, heads, DIM, generator=g, device="cuda").to(torch.bfloat16),
         "sinks": torch.randn(heads, generator=g, device="cuda"), "lens": i32(s2), "ratio": r,
         "cu": i32([sum(s1[:b]) for b in range(batch + 1)]), "mode": case["mode"], "tnd": case["layout"] == "TND",
         "used_q": i32([n - b % 2 for b, n in enumerate(s1)]) if case["padded"] else None,
         "idx": None, "cmp_kv": None, "cmp_table": None, "residual": None, "max_cmp": max(s2) // r}
    bank = _pack384(torch.randn(1 << 15, DIM, generator=g, device="cuda"))
    # blocks behind every window have been given back: -1 in the table
    first = [max(0, b2 - b1 - (WINDOW - 1)) // BLOCK for b1, b2 in zip(s1, s2)]
    ends = [-(-n // BLOCK) for n in s2]
    blocks = sum(e - f for f, e in zip(first, ends))
    perm = torch.randperm(blocks, generator=g, device="cuda").int()
    col = torch.arange(max(ends), device="cuda")[None]
    live = (col >= i32(first)[:, None]) & (col < i32(ends)[:, None])
    order = (live.flatten().cumsum(0) - 1).clamp(min=0).view(live.shape)
    s["ori_kv"], s["ori_table"] = _pool(bank, blocks, g), torch.where(live, perm[order], -1).int()
    if case["mode"] != "SWA":
        ends = [-(-(n // r) // BLOCK) for n in s2]
        blocks = sum(ends)
        perm = torch.randperm(max(blocks, 1), generator=g, device="cuda").int()
        col = torch.arange(max(max(ends), 1), device="cuda")[None]
        live = col < i32(ends)[:, None]
        order = (live.flatten().cumsum(0) - 1).clamp(min=0).view(live.shape)
        s["cmp_kv"], s["cmp_table"] = _pool(bank, blocks, g), torch.where(live, perm[order], -1).int()
        s["residual"] = i32([n % r for n in s2])
    if case["mode"] == "CSA":
        _, _, _, vis = _geometry(s)
        score = torch.rand(total, max(s["max_cmp"], case["k2"], 1), generator=g, device="cuda")
        score = torch.where(torch.arange(score.shape[1], device="cuda")[None] < vis[:, None], score, -1.0)
        top = score.topk(case["k2"], dim=1)
        idx = torch.where(top.values >= 0, top.indices, -1)
        idx[:, case["valid"]:] = -1
        s["idx"] = idx.int().view(total, 1, case["k2"]).contiguous()
    if own:  # the buffers and the parameter block that a serving loop keeps from step to step
        import compressed_mla_attention_gb300 as Q

        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(total, heads, device="cuda")
        s["plan"] = torch.empty(Q.METADATA_INTS, dtype=torch.int32, device="cuda")
        shaped = (lambda t: t) if s["tnd"] else (lambda t: t.view(batch, s1[0], heads, DIM))
        s["params"] = Q.make_params(
            q=shaped(s["q"]), attn_out=shaped(s["out"]), ori_kv=s["ori_kv"], ori_scale=None,
            ori_block_table=s["ori_table"], seqused_ori_kv=s["lens"], layout=case["layout"], cmp_kv=s["cmp_kv"],
            cmp_block_table=s["cmp_table"], cmp_sparse_indices=s["idx"], cu_seqlens_q=s["cu"] if s["tnd"] else None,
            seqused_q=s["used_q"], cmp_residual_kv=s["residual"], sinks=s["sinks"], metadata=s["plan"],
            softmax_lse=s["lse"], cmp_ratio=r, return_lse=True)
        size = Q.workspace_size(s["params"])
        s["work"] = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    return s


def _geometry(s):
    """Of each query token: its request, its position in the request, whether it is no padding, and how many
    compressed rows it sees."""
    t = torch.arange(s["q"].shape[0], device="cuda", dtype=torch.int32)
    b = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    i = t - s["cu"][b]
    n = s["cu"][b + 1] - s["cu"][b]
    pos = s["lens"][b] - n + i
    live = torch.ones_like(i, dtype=torch.bool) if s["used_q"] is None else i < s["used_q"][b]
    return b, pos, live, (pos + 1) // s["ratio"]


def _attn_rows(s):
    """The cache rows of each token, as bytes [T, R, 384], and which of them it attends [T, R]."""
    b, pos, live, vis = _geometry(s)
    row = pos[:, None] - (WINDOW - 1) + torch.arange(WINDOW, device="cuda")[None]
    ok = (row >= 0) & live[:, None]
    row = row.clamp(min=0)
    at = s["ori_table"][b[:, None], row // BLOCK] * BLOCK + row % BLOCK
    raw = s["ori_kv"].view(-1, 384)[torch.where(ok, at, 0)]
    if s["cmp_kv"] is not None and s["max_cmp"] > 0:
        row = s["idx"][:, 0].long() if s["idx"] is not None else torch.arange(s["max_cmp"], device="cuda")[None].expand(len(b), -1)
        good = (row >= 0) & (row < vis[:, None]) & live[:, None]
        row = torch.where(good, row, 0)
        at = s["cmp_table"][b[:, None], row // BLOCK] * BLOCK + row % BLOCK
        raw = torch.cat((raw, s["cmp_kv"].view(-1, 384)[torch.where(good, at, 0)]), 1)
        ok = torch.cat((ok, good), 1)
    return raw, ok


def _attend(q, k, ok, sinks):
    """softmax([q k^T / sqrt(512), sink]) k over the rows marked in ok; and the log of the sum without the sink."""
    x = torch.bmm(q, k.transpose(1, 2)) * DIM ** -0.5
    x = torch.where(ok[:, None, :], x, -math.inf)
    top = torch.maximum(x.amax(2), sinks[None])
    e = torch.exp(x - top[:, :, None])
    total = e.sum(2)
    any_row = ok.any(1)[:, None]
    out = torch.bmm(e / (total + torch.exp(sinks[None] - top))[:, :, None], k)
    return torch.where(any_row[:, :, None], out, 0.0), torch.where(any_row, torch.log(total) + top, -math.inf)


def _run_attn(s):
    if own:
        import compressed_mla_attention_gb300 as Q

        Q.metadata(s["params"], s["plan"])  # the lengths change from step to step: a step plans anew
        Q.forward(s["params"], s["work"])
        return {"out": s["out"], "lse": s["lse"]}
    raw, ok = _attn_rows(s)
    out, lse = _attend(s["q"].float(), _unpack384(raw, torch.float32), ok, s["sinks"])
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _exact_attn(case, g):
    """Request by request, from its rows in logical order."""
    s = _prepare_attn(case, g)
    s1, s2 = _lengths(case)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device="cuda")
    eight = torch.arange(256, device="cuda").to(torch.uint8).view(torch.float8_e4m3fn).double()

    def logical(kv, blocks, first, last):
        """The values of logical rows first .. last - 1 of the request with these blocks."""
        if last <= first:
            return torch.zeros(0, DIM, dtype=torch.float64, device="cuda")
        held = kv[blocks[first // BLOCK:(last - 1) // BLOCK + 1].long(), :, 0].flatten(0, 1)
        raw = held[first % BLOCK:first % BLOCK + last - first]
        code = raw[:, 128:352].int()
        value = table[torch.stack((code & 15, code >> 4), 2).long()].view(-1, 28, 16)
        value = value * eight[raw[:, 352:380].int().long()][:, :, None] * 2.0 ** (raw[:, 380].double() - 127)[:, None, None]
        return torch.cat((raw[:, :128].contiguous().view(torch.bfloat16).double(), value.flatten(1)), 1)

    sinks, r, out, lse, at = s["sinks"].double()[None], case["ratio"], [], [], 0
    for b, (n, m) in enumerate(zip(s1, s2)):
        far = logical(s["cmp_kv"], s["cmp_table"][b], 0, m // r) if case["mode"] != "SWA" else None
        for lo in range(0, n, 128):
            hi = min(lo + 128, n)
            i = torch.arange(lo, hi, device="cuda")[:, None]
            pos = m - n + i
            used = n - b % 2 if case["padded"] else n
            start = max(0, m - n + lo - WINDOW + 1)
            near = logical(s["ori_kv"], s["ori_table"][b], start, m - n + hi)
            q = s["q"][at + lo:at + hi].double() / math.sqrt(DIM)
            j = torch.arange(start, m - n + hi, device="cuda")[None]
            sees = (j <= pos) & (j > pos - WINDOW) & (i < used)
            x = [torch.einsum("thd,rd->thr", q, near).masked_fill(~sees[:, None], -math.inf)]
            if case["mode"] == "HCA" and len(far):
                sees = ((torch.arange(len(far), device="cuda")[None] + 1) * r - 1 <= pos) & (i < used)
                x.append(torch.einsum("thd,rd->thr", q, far).masked_fill(~sees[:, None], -math.inf))
            elif case["mode"] == "CSA" and len(far):
                pick = s["idx"][at + lo:at + hi, 0].long()
                sees = (pick >= 0) & ((pick + 1) * r - 1 <= pos) & (i < used)
                k = far[pick.clamp(0, len(far) - 1)]
                x.append(torch.bmm(q, k.transpose(1, 2)).masked_fill(~sees[:, None], -math.inf))
            total = torch.logsumexp(torch.cat(x, 2), 2)
            both = torch.logaddexp(total, sinks)[:, :, None]
            o = torch.einsum("thr,rd->thd", torch.exp(x[0] - both), near)
            if len(x) > 1:
                w = torch.exp(x[1] - both)
                o = o + (torch.bmm(w, k) if case["mode"] == "CSA" else torch.einsum("thr,rd->thd", w, far))
            out.append(o)
            lse.append(total)
        at += n
    return {"out": torch.cat(out), "lse": torch.cat(lse)}


def _work_attn(case):
    s1, s2 = _lengths(case)
    r, k2, heads, read, pairs, idx = case["ratio"], case["valid"], case["heads"], 0.0, 0, 0
    for n, m in zip(s1, s2):
        read += min(m, n + WINDOW - 1)
        seen = (m + 1) // r if case["mode"] != "SWA" else 0
        if case["mode"] == "HCA":
            read += m // r
        elif case["mode"] == "CSA" and seen:
            read += seen * (1 - (1 - min(k2, seen) / seen) ** n)
        for i in range(n):
            pos = m - n + i
            vis = 0 if case["mode"] == "SWA" else (pos + 1) // r
            pairs += min(pos + 1, WINDOW) + (min(vis, k2) if case["mode"] == "CSA" else vis)
            idx += case["k2"]
    return {"bytes": read * 384 + sum(s1) * heads * (4 * DIM + 4) + 4 * idx, "flops": 4.0 * heads * DIM * pairs}


# ------------------------------------------------------------------ rows
def _cache(fmt, rows):
    if fmt == "bf16":
        return torch.zeros(rows // BLOCK, BLOCK, 1, DIM, dtype=torch.bfloat16, device="cuda"), None
    width = {"packed384": 384, "packed640": 640, "fp8_fp32_scales": DIM}[fmt]
    scale = torch.zeros(rows // BLOCK, BLOCK, 1, 8, device="cuda") if width == DIM else None
    return torch.zeros(rows // BLOCK, BLOCK, 1, width, dtype=torch.uint8, device="cuda"), scale


def _prepare_rows(case, g):
    n, heads, dtype = case["tokens"], case["heads"], getattr(torch, case["dtype"])
    far = 1 << 16
    if case["fused"]:  # one projection's output, queries first
        x = torch.randn(n, heads + 1, DIM, generator=g, device="cuda").to(dtype)
        q, kv = x[:, :heads], x[:, heads]
    else:
        q = torch.randn(n, heads, DIM, generator=g, device="cuda").to(dtype) if heads else None
        kv = (1.5 * torch.randn(n, DIM, generator=g, device="cuda")).to(dtype)
    angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None]
    angle = angle * 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
    start = int(torch.randint(0, far - n, (1,), generator=g, device="cuda"))
    pos = torch.randint(0, far, (n,), generator=g, device="cuda") if n <= 512 else start + torch.arange(n, device="cuda")
    rows = -(-2 * n // BLOCK) * BLOCK + BLOCK
    slots = torch.randperm(rows - 1, generator=g, device="cuda")[:n]
    if case["padded"]:
        pos[-case["padded"]:] = -1
        slots[-case["padded"]:] = -1
    weight = lambda: (1 + 0.2 * torch.randn(DIM, generator=g, device="cuda")).to(getattr(torch, case["weights"]))  # noqa: E731
    cache, scale = _cache(case["format"], rows)
    s = {"q": q, "kv": kv, "pos": pos.int(), "slots": slots.int(), "table": torch.cat((angle.cos(), angle.sin()), 1).float(),
         "q_weight": weight() if heads else None, "kv_weight": weight(), "cache": cache, "scale": scale, "case": case,
         "q_out": torch.zeros(n, heads, DIM, dtype=torch.bfloat16, device="cuda") if heads else None,
         "rows": torch.zeros(n, DIM, dtype=torch.bfloat16, device="cuda")}
    if own:  # the parameter block that a serving loop keeps
        import compressed_mla_attention_gb300 as Q

        s["params"] = Q.make_norm_rope_params(
            q=q, q_out=s["q_out"], kv=kv, kv_cache=cache, kv_scale=scale, kv_out=s["rows"], slot_map=s["slots"],
            positions=s["pos"], cos_sin=s["table"], q_weight=s["q_weight"], kv_weight=s["kv_weight"], eps=1e-6,
            rope_offset=case["rope_at"], interleaved=case["pairs"] == "adjacent")
    return s


def _norm_rope(x, weight, pos, s):
    """Norm and rotation of rows x [n, heads, 512] in 32 bits."""
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(2, keepdim=True) + 1e-6) * weight.float()
    at = s["case"]["rope_at"]
    z, (cos, sin) = y[:, :, at:at + ROPE], s["table"][pos.clamp(min=0)][:, None].chunk(2, 2)
    if s["case"]["pairs"] == "adjacent":
        a, b = z[..., 0::2], z[..., 1::2]
        z = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
    else:
        a, b = z.chunk(2, 2)
        z = torch.cat((a * cos - b * sin, b * cos + a * sin), 2)
    return torch.cat((y[:, :, :at], z, y[:, :, at + ROPE:]), 2)


def _store(y, fmt):
    """fp32 rows [n, 512] as the format's bytes (bf16 rows: values), its scales, and the values that they stand for."""
    n = y.shape[0]
    if fmt == "bf16":
        return y.to(torch.bfloat16), None, y.to(torch.bfloat16)
    if fmt == "packed384":
        raw = _pack384(y)
        return raw, None, _unpack384(raw, torch.float32).to(torch.bfloat16)
    if fmt == "packed640":
        t = y[:, ROPE:].reshape(n, 7, 64)
        m, e = torch.frexp(t.abs().amax(2))  # the smallest power of two that keeps the tile within 448
        e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -100).clamp(-100, 100)
        power = torch.ldexp(torch.ones_like(m), e)[:, :, None]
        c = (t / power).to(torch.float8_e4m3fn)
        rope = y[:, :ROPE].to(torch.bfloat16)
        raw = torch.cat((rope.contiguous().view(torch.uint8), c.view(torch.uint8).reshape(n, 448),
                         (e + 127).to(torch.uint8), torch.zeros(n, 57, dtype=torch.uint8, device="cuda")), 1)
        return raw, None, torch.cat((rope.float(), (c.float() * power).reshape(n, 448)), 1).to(torch.bfloat16)
    t = y.reshape(n, 8, 64)
    scale = t.abs().amax(2).clamp(min=1e-12) / 448
    c = (t / scale[:, :, None]).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).reshape(n, DIM), scale, (c.float() * scale[:, :, None]).reshape(n, DIM).to(torch.bfloat16)


def _cache_parts(s):
    """The cache as the values that its bytes stand for (views)."""
    fmt = s["case"]["format"]
    if fmt == "bf16":
        return {"cache": s["cache"]}
    flat = s["cache"].view(-1, s["cache"].shape[-1])
    if fmt == "fp8_fp32_scales":
        return {"codes": flat.view(torch.float8_e4m3fn), "scales": s["scale"]}
    if fmt == "packed640":
        return {"rope": flat[:, :128].view(torch.bfloat16), "codes": flat[:, 128:576].view(torch.float8_e4m3fn),
                "scales": flat[:, 576:583].view(torch.float8_e8m0fnu)}
    return {"rope": flat[:, :128].view(torch.bfloat16), "scales": flat[:, 352:380].view(torch.float8_e4m3fn)}


def _run_rows(s):
    if own:
        import compressed_mla_attention_gb300 as Q

        Q.norm_rope(s["params"])
    else:
        live = s["pos"] >= 0
        if s["q"] is not None:
            q = _norm_rope(s["q"], s["q_weight"], s["pos"], s).to(torch.bfloat16)
            s["q_out"] = torch.where(live[:, None, None], q, s["q_out"])
        raw, scale, rows = _store(_norm_rope(s["kv"][:, None], s["kv_weight"], s["pos"], s)[:, 0], s["case"]["format"])
        s["rows"] = torch.where(live[:, None], rows, s["rows"])
        # a padded token writes the last row, which no token has, as it was
        for cache, new in ((s["cache"], raw), (s["scale"], scale)):
            if new is not None:
                flat = cache.view(-1, cache.shape[-1])
                at = torch.where(live, s["slots"], flat.shape[0] - 1).long()
                flat[at] = torch.where(live[:, None], new, flat[-1:])
    return {"q": s["q_out"], "rows": s["rows"], **_cache_parts(s)}


def _half_even(x, bits, lowest):
    """x to `bits` significant bits, none finer than `lowest`; ties to even."""
    unit = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=1e-300))) + 1 - bits).clamp(min=lowest)
    return torch.round(x / unit) * unit


def _exact_rows(case, g):
    s = _prepare_rows(case, g)
    at, fmt, n = case["rope_at"], case["format"], case["tokens"]
    turn = torch.complex(*s["table"][s["pos"].clamp(min=0)].double().chunk(2, 1))[:, None]

    def rows(x, w):
        y = x.double()
        y = y / torch.sqrt(y.square().sum(2, keepdim=True) / DIM + 1e-6) * w.double()
        z = y[:, :, at:at + ROPE].unflatten(2, (ROPE // 2, 2) if case["pairs"] == "adjacent" else (2, ROPE // 2))
        pair = 3 if case["pairs"] == "adjacent" else 2
        z = torch.complex(z.select(pair, 0), z.select(pair, 1)) * turn
        y[:, :, at:at + ROPE] = torch.stack((z.real, z.imag), pair).flatten(2)
        return y

    live = (s["pos"] >= 0)[:, None]
    y = rows(s["kv"][:, None], s["kv_weight"])[:, 0]
    far = s["cache"].shape[0] * BLOCK
    spread = lambda v: torch.zeros(far, v.shape[1], dtype=torch.float64, device="cuda").index_copy_(  # noqa: E731
        0, torch.where(live[:, 0], s["slots"], far - 1).long(), torch.where(live, v, 0.0))
    rope, parts = _half_even(y[:, :ROPE], 8, 1e-300), {}
    if fmt == "bf16":
        held = _half_even(y, 8, 1e-300)
        parts["cache"] = spread(held).view(s["cache"].shape)
    elif fmt == "fp8_fp32_scales":
        t = y.view(n, 8, 64)
        scale = t.abs().amax(2) / 448
        code = _half_even(t / scale[:, :, None], 4, 2.0 ** -9)
        held = (code * scale[:, :, None]).view(n, DIM)
        parts["codes"], parts["scales"] = spread(code.view(n, DIM)), spread(scale).view(s["scale"].shape)
    elif fmt == "packed640":
        t = y[:, ROPE:].reshape(n, 7, 64)
        scale = torch.exp2(torch.ceil(torch.log2(t.abs().amax(2) / 448)))
        code = _half_even(t / scale[:, :, None], 4, 2.0 ** -9)
        held = torch.cat((rope, (code * scale[:, :, None]).view(n, 448)), 1)
        none = 2.0 ** -127 * (torch.ones(far, 7, dtype=torch.float64, device="cuda") - spread(torch.ones_like(scale)))
        parts = {"rope": spread(rope), "codes": spread(code.view(n, 448)), "scales": spread(scale) + none}
    else:
        t = y[:, ROPE:].reshape(n, 28, 16)
        power = torch.exp2(torch.floor(torch.log2(y.abs().amax(1))) - 10)[:, None]
        scale = _half_even(t.abs().amax(2) / 6 / power, 4, 2.0 ** -9)
        step = (scale * power)[:, :, None]
        code = _half_even(torch.where(step > 0, t / step, 0.0), 2, 0.5).clamp(-6, 6)
        held = torch.cat((rope, (code * step).reshape(n, 448)), 1)
        parts = {"rope": spread(rope), "scales": spread(scale)}
    q = None
    if s["q"] is not None and s["q"].numel() <= 1 << 29:
        q = torch.where(live[:, :, None], rows(s["q"], s["q_weight"]), 0.0)
    return {"q": q, "rows": torch.where(live, held, 0.0), **parts}


def _work_rows(case):
    n, heads = case["tokens"] - case["padded"], case["heads"]
    size = 4 if case["dtype"] == "float32" else 2
    row = {"packed384": 384, "packed640": 640, "fp8_fp32_scales": 544, "bf16": 1024}[case["format"]]
    return {"bytes": n * (heads * DIM * (size + 2) + DIM * (size + 2) + row + 4 * ROPE + 8),
            "flops": 5.0 * n * (heads + 1) * DIM}


# ------------------------------------------------------------------ tables
def _prepare_tables(case, g):
    batch, r = case["batch"], case["ratio"]
    chance = torch.rand(batch, generator=g, device="cuda")
    prev = torch.randint(1, case["len_hi"], (batch,), generator=g, device="cuda")
    prev = torch.where(chance < 0.05, 0, prev)  # a request begins
    new = torch.randint(case["new_lo"], case["new_hi"] + 1, (batch,), generator=g, device="cuda")
    lens = torch.where(chance > 0.95, 0, prev + new)  # a request ends
    width = -(-((case["len_hi"] + case["new_hi"]) // r) // BLOCK) + 1
    held = (prev // r + BLOCK - 1) // BLOCK
    blocks = batch * width
    perm = torch.randperm(blocks, generator=g, device="cuda").int()
    live = torch.arange(width, device="cuda")[None] < held[:, None]
    order = (live.flatten().cumsum(0) - 1).clamp(min=0).view(live.shape)
    used = live.sum()
    s = {"table": torch.where(live, perm[order], -1).int(), "prev": prev.int(), "lens": lens.int(), "ratio": r,
         "free": perm.roll(-int(used)).contiguous(), "count": (blocks - used).int().view(1),
         "rows": batch * (case["new_hi"] // r + 1), "batch": batch}
    if own:  # the outputs and the parameter block that a serving loop keeps
        import compressed_mla_attention_gb300 as Q

        i32 = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        s |= {"slots": i32(s["rows"]), "pos": i32(s["rows"]), "cu": i32(batch + 1), "left": i32(1), "residual": i32(batch)}
        s["params"] = Q.make_block_table_params(
            block_table=s["table"], prev_lens=s["prev"], lens=s["lens"], free_list=s["free"], free_count=s["count"],
            free_count_out=s["left"], cmp_ratio=r, slot_map=s["slots"], positions=s["pos"], cu_rows=s["cu"],
            residual=s["residual"])
    return s


def _run_tables(s):
    if own:
        import compressed_mla_attention_gb300 as Q

        Q.block_tables(s["params"])
        return {"table": s["table"], "free": s["free"], "count": s["left"], "slots": s["slots"], "pos": s["pos"],
                "cu": s["cu"], "residual": s["residual"]}
    r, table, free, count = s["ratio"], s["table"], s["free"], s["count"]
    before, after = s["prev"] // r, s["lens"] // r
    held, need = (before + BLOCK - 1) // BLOCK, (after + BLOCK - 1) // BLOCK
    cu = torch.zeros(s["batch"] + 1, dtype=torch.int32, device="cuda")
    cu[1:] = (after - before).clamp(min=0).cumsum(0)
    col = torch.arange(table.shape[1], device="cuda")[None]
    give = ((col >= need[:, None]) & (col < held[:, None])).flatten()
    take = ((col >= held[:, None]) & (col < need[:, None])).flatten()
    given, taken = give.cumsum(0), take.cumsum(0)
    back = torch.zeros(give.numel() + 1, dtype=torch.int32, device="cuda")  # the blocks given back, in order
    back[torch.where(give, given - 1, give.numel())] = table.flatten()
    at = count + given[-1] - taken  # the taken blocks' places in the stack: free, then given back
    block = torch.where(at >= count, back[(at - count).clamp(0, give.numel())], free[at.clamp(0, free.numel() - 1)])
    table = torch.where(take, torch.where(at >= 0, block, -1), table.flatten()).view(table.shape)
    j = torch.arange(free.numel(), device="cuda") - count
    left = given[-1] - taken[-1]
    free = torch.where((j >= 0) & (j < left), back[j.clamp(0, give.numel())], free)
    t = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=s["batch"] - 1)
    row = before[b] + t - cu[b]
    block = table[b, (row // BLOCK).clamp(0, table.shape[1] - 1)]
    live = t < cu[-1]
    slots = torch.where(live & (block >= 0), block * BLOCK + row % BLOCK, -1).int()
    return {"table": table, "free": free, "count": (count + left).clamp(min=0).int(), "slots": slots,
            "pos": torch.where(live, row * r, -1).int(), "cu": cu, "residual": s["lens"] % r}


def _work_tables(case):
    rows = 0.95 * case["batch"] * (case["new_lo"] + case["new_hi"]) / 2 / case["ratio"]
    given = 0.05 * case["batch"] * case["len_hi"] / 2 / case["ratio"] / BLOCK
    return {"bytes": 16.0 * case["batch"] + 8 * rows + 4 * rows / BLOCK + 8 * given, "flops": 0.0}


# ------------------------------------------------------------------ the calls
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"attn": _prepare_attn, "rows": _prepare_rows, "tables": _prepare_tables}[case["op"]](case, g)
    return s | {"op": case["op"]}


def run(state):
    return {"attn": _run_attn, "rows": _run_rows, "tables": _run_tables}[state["op"]](state)


def work(case):
    return {"attn": _work_attn, "rows": _work_rows, "tables": _work_tables}[case["op"]](case)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers alone
    g = torch.Generator("cuda").manual_seed(seed)
    return {"attn": _exact_attn, "rows": _exact_rows}[case["op"]](case, g)
