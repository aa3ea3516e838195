"""The 8-bit products around the attention: rows quantised to e4m3 with a scale per 128 elements, the product of such rows
with a weight matrix, and the same product with one matrix per group of rows.

Each case is one call of one operator. `run` computes it with elementary torch operations (`own` false) or by this package's
kernels (`own` true); `exact` computes it in 64 bits.

A quantised row of K elements is K e4m3 codes and ceil(K / 128) fp32 scales: with A the largest magnitude of 128 elements (at
least 1e-12), scale = A / 448 and code = e4m3(448 y / A); with scales that are powers of two, the smallest power that keeps A
within 448 steps. A quantised matrix has one scale for each 128 x 128 elements.
"""

import math
import random

import torch

own = False

GROUP = 128
ROPE = 64
FAR = 1 << 16  # positions of the rotation's table


def listed():
    return [
        # one token's hidden state before a projection: what a single stream waits for
        {"name": "quant_single", "op": "quant", "tokens": 1, "source": 1, "heads": 1, "dim": 4096, "dtype": "bfloat16",
         "mode": "plain", "pairs": "adjacent", "rope_at": 0, "pow2": False},
        # the indexer's queries of the decode batch's 256 tokens: 64 heads of 128, the last 64 elements rotated
        {"name": "quant_indexer", "op": "quant", "tokens": 256, "source": 256, "heads": 64, "dim": 128, "dtype": "bfloat16",
         "mode": "rotate", "pairs": "adjacent", "rope_at": 64, "pow2": False},
        # a prefill step's attention output, rotated back before the output projection
        {"name": "quant_output", "op": "quant", "tokens": 4099, "source": 4099, "heads": 64, "dim": 512, "dtype": "bfloat16",
         "mode": "rotate_back", "pairs": "halves", "rope_at": 448, "pow2": False},
        # the hidden rows of experts: silu(gate) * up, both halves of one product's output
        {"name": "quant_gated", "op": "quant", "tokens": 16001, "source": 16001, "heads": 1, "dim": 2048, "dtype": "bfloat16",
         "mode": "gated", "pairs": "adjacent", "rope_at": 0, "pow2": True},
        # a prefill step's tokens in the order of their experts, eight for each
        {"name": "quant_gather", "op": "quant", "tokens": 16384, "source": 2048, "heads": 1, "dim": 5120, "dtype": "float32",
         "mode": "gather", "pairs": "adjacent", "rope_at": 0, "pow2": False},
        # one token through a square projection
        {"name": "product_single", "op": "product", "rows": 1, "n": 4096, "k": 4096, "out": "bfloat16"},
        # the output projection of the decode batch's 256 tokens: 64 heads of 512
        {"name": "product_decode", "op": "product", "rows": 256, "n": 4096, "k": 32768, "out": "bfloat16"},
        # a ragged product in fp32: no size is a multiple of the tiles
        {"name": "product_odd", "op": "product", "rows": 777, "n": 1000, "k": 2064, "out": "float32"},
        # the output projection of four whole prompts of 2048 tokens
        {"name": "product_prefill", "op": "product", "rows": 8192, "n": 4096, "k": 32768, "out": "bfloat16"},
        # two tokens, eight experts each
        {"name": "grouped_tiny", "op": "grouped", "rows": 16, "padded": 0, "groups": 64, "n": 1408, "k": 2048, "out": "bfloat16"},
        # the decode batch's 256 tokens, eight of 128 experts each, some rows without a group
        {"name": "grouped_decode", "op": "grouped", "rows": 2048, "padded": 31, "groups": 128, "n": 2048, "k": 4096,
         "out": "bfloat16"},
        # a prefill step of 8192 tokens, eight of 64 experts each
        {"name": "grouped_prefill", "op": "grouped", "rows": 65536, "padded": 0, "groups": 64, "n": 2048, "k": 4096,
         "out": "bfloat16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "product", "grouped"))
    if op == "quant":
        mode = rng.choice(("plain", "rotate", "rotate_back", "gated", "gather"))
        if mode in ("plain", "rotate", "rotate_back"):
            heads, dim = rng.choice(((1, 128), (64, 128), (64, 512), (128, 512), (8, 256)))
            if mode == "plain" and rng.random() < 0.5:
                heads, dim = 1, 16 * _log(rng, 1, 1024)
        else:
            heads, dim = 1, 16 * _log(rng, 4, 512)
        tokens = _log(rng, 1, min(30000, 40000000 // (heads * dim)))
        return {"op": "quant", "tokens": tokens, "source": max(1, tokens // rng.choice((1, 2, 8))) if mode == "gather" else tokens,
                "heads": heads, "dim": dim, "dtype": rng.choice(("bfloat16", "bfloat16", "float16", "float32")), "mode": mode,
                "pairs": rng.choice(("adjacent", "halves")), "rope_at": rng.choice((0, dim - ROPE)) if dim > ROPE else 0,
                "pow2": rng.random() < 0.3}
    out = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
    if op == "product":
        n, k = _log(rng, 40, 32768), 16 * _log(rng, 4, 2048)
        return {"op": "product", "rows": _log(rng, 1, max(2, min(10000, (1 << 39) // (n * k)))), "n": n, "k": k, "out": out}
    n, k = _log(rng, 100, 4096), 16 * _log(rng, 16, 400)
    rows = _log(rng, 1, 30000)
    return {"op": "grouped", "rows": rows, "padded": rng.choice((0, rows // 20)),
            "groups": _log(rng, 1, max(2, min(256, (1 << 30) // (n * k)))), "n": n, "k": k, "out": out}


# ------------------------------------------------------------------ quantised rows
def _prepare_quant(case, g):
    t, src, heads, dim = case["tokens"], case["source"], case["heads"], case["dim"]
    dtype, mode = getattr(torch, case["dtype"]), case["mode"]
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # rows of different size, a few elements of each far larger than the others
    size = torch.exp(0.7 * rand(src, 1, 1))
    s = {"case": case, "gate": None, "index": None, "pos": None, "table": None}
    s["powers"] = torch.tensor([2.0 ** k for k in range(-160, 161)], dtype=torch.float64).cuda()  # of two, exactly
    if mode == "gated":  # gate and up projection side by side in one product's output
        both = (2 * rand(src, 2, dim) * size).to(dtype)
        s["gate"], s["x"] = both[:, :1], both[:, 1:]
    else:
        x = rand(src, heads, dim) * size
        s["x"] = torch.where(torch.rand(src, heads, dim, generator=g, device="cuda") < 1e-3, 20 * x, x).to(dtype)
    if mode in ("rotate", "rotate_back"):
        angle = torch.arange(FAR, device="cuda", dtype=torch.float64)[:, None]
        angle = angle * 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)
        s["table"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["pos"] = torch.randint(0, FAR, (t,), generator=g, device="cuda").int()
    if mode == "gather":
        s["index"] = torch.randint(0, src, (t,), generator=g, device="cuda").int()
    if own:  # the outputs and the parameter block that a serving loop keeps
        import compressed_mla_attention_gb300 as Q

        s["codes"] = torch.empty(t, heads * dim, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(t, -(-heads * dim // GROUP), device="cuda")
        s["params"] = Q.make_quantize_params(
            x=s["x"], gate=s["gate"], row_index=s["index"], positions=s["pos"], cos_sin=s["table"], rope_offset=case["rope_at"],
            interleaved=case["pairs"] == "adjacent", inverse=mode == "rotate_back", pow2_scale=case["pow2"],
            codes=s["codes"], scale=s["scales"])
    return s


def _run_quant(s):
    case = s["case"]
    if own:
        import compressed_mla_attention_gb300 as Q

        Q.quantize(s["params"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    mode, at, n = case["mode"], case["rope_at"], case["heads"] * case["dim"]
    # values that 16-bit inputs hold are quantised right in 32 bits; computed ones, and fp32's own, lie next to a border
    wide = mode in ("rotate", "rotate_back", "gated") or s["x"].dtype == torch.float32
    y = s["x"].to(torch.float64 if wide else torch.float32)
    if mode == "gated":
        gate = s["gate"].double()
        y = y * gate / (1 + torch.exp(-gate))
    if s["index"] is not None:
        y = y[s["index"].long()]
    if s["pos"] is not None:
        z, (cos, sin) = y[:, :, at:at + ROPE], s["table"][s["pos"]].to(y.dtype)[:, None].chunk(2, 2)
        sin = -sin if mode == "rotate_back" else sin
        if case["pairs"] == "adjacent":
            a, b = z[..., 0::2], z[..., 1::2]
            z = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
        else:
            a, b = z.chunk(2, 2)
            z = torch.cat((a * cos - b * sin, b * cos + a * sin), 2)
        y = torch.cat((y[:, :, :at], z, y[:, :, at + ROPE:]), 2)
    y = y.flatten(1)
    if n % GROUP:
        y = torch.nn.functional.pad(y, (0, GROUP - n % GROUP))
    y = y.view(y.shape[0], -1, GROUP)
    amax = y.abs().amax(2, keepdim=True)
    if case["pow2"]:
        m, e = torch.frexp(amax)
        e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -100).clamp(-100, 100)
        scale = s["powers"][(e + 160).long()].to(y.dtype)
        q = y / scale
    else:
        amax = amax.clamp(min=1e-12)
        scale = amax / 448
        q = y * 448 / amax
    # to the nearest of the codes' values, ties to even: 4 significant bits, none finer than 2^-9
    unit = s["powers"][((torch.frexp(q).exponent - 4).clamp(min=-9) + 160).long()].to(q.dtype)
    q = (torch.round(q / unit) * unit).flatten(1)[:, :n]
    return {"codes": q.float().to(torch.float8_e4m3fn), "scales": scale[:, :, 0].float()}


def _exact_quant(case, g):
    s = _prepare_quant(case, g)
    y, mode = s["x"].double(), case["mode"]
    if mode == "gated":
        y = y * s["gate"].double() * torch.sigmoid(s["gate"].double())
    if mode == "gather":
        y = torch.index_select(y, 0, s["index"].long())
    if s["pos"] is not None:
        turn = torch.complex(*s["table"][s["pos"].long()].double().chunk(2, 1))[:, None]
        turn = turn.conj() if mode == "rotate_back" else turn
        part = y.narrow(2, case["rope_at"], ROPE)
        z = part.unflatten(2, (ROPE // 2, 2) if case["pairs"] == "adjacent" else (2, ROPE // 2))
        axis = 3 if case["pairs"] == "adjacent" else 2
        z = torch.complex(z.select(axis, 0), z.select(axis, 1)) * turn
        part.copy_(torch.stack((z.real, z.imag), axis).flatten(2))
    n = y.shape[1] * y.shape[2]
    groups = -(-n // GROUP)
    full = torch.zeros(y.shape[0], groups * GROUP, dtype=torch.float64, device="cuda")
    full[:, :n] = y.reshape(y.shape[0], n)
    top = full.view(-1, groups, GROUP).abs().max(2).values
    if case["pow2"]:
        m, e = torch.frexp(top / 448)
        scale = torch.tensor([2.0 ** k for k in range(-100, 101)], dtype=torch.float64, device="cuda")
        step = scale = scale[torch.where(top > 0, e - (m == 0.5).int(), -100).clamp(-100, 100).long() + 100]
    else:
        scale = top.clamp(min=1e-12) / 448
        step = scale
    # the codes' values and the borders between them; a value on a border goes to the even code
    values = torch.tensor([(k % 8 / 8 + (k >= 8)) * 2.0 ** (max(k // 8, 1) - 7) for k in range(127)], dtype=torch.float64,
                          device="cuda")
    border = (values[1:] + values[:-1]) / 2
    codes = torch.empty(full.shape, dtype=torch.float32, device="cuda")
    for lo in range(0, full.shape[0], 1024):
        f = full[lo:lo + 1024].view(-1, groups, GROUP)
        q = f / step[lo:lo + 1024, :, None] if case["pow2"] else f * 448 / top[lo:lo + 1024, :, None].clamp(min=1e-12)
        a = q.abs().contiguous()
        up, down = torch.searchsorted(border, a, right=True), torch.searchsorted(border, a)
        k = torch.where(up % 2 == 0, up, down)
        codes[lo:lo + 1024] = (values[k] * q.sign()).float().flatten(1)
    return {"codes": codes[:, :n].double(), "scales": scale}


def _work_quant(case):
    t, src, k = case["tokens"], case["source"], case["heads"] * case["dim"]
    size = 4 if case["dtype"] == "float32" else 2
    read = src * k * size * (2 if case["mode"] == "gated" else 1)
    read += 4 * t * (1 + ROPE) if case["mode"].startswith("rotate") else 4 * t if case["mode"] == "gather" else 0
    return {"bytes": read + t * k + 4 * t * -(-k // GROUP), "flops": 4.0 * t * k}


# ------------------------------------------------------------------ products
def _quantised(x):
    """x [..., rows, K] as codes with a scale for each 128 elements of a row."""
    n = x.shape[-1]
    t = torch.nn.functional.pad(x, (0, -n % GROUP)).unflatten(-1, (-1, GROUP))
    scale = t.abs().amax(-1, keepdim=True).clamp(min=1e-12) / 448
    return (t / scale).to(torch.float8_e4m3fn).flatten(-2)[..., :n].contiguous(), scale[..., 0].contiguous()


def _quantised_matrix(x):
    """x [N, K] as codes with a scale for each 128 x 128 elements."""
    n, k = x.shape
    t = torch.nn.functional.pad(x, (0, -k % GROUP, 0, -n % GROUP)).unflatten(1, (-1, GROUP)).unflatten(0, (-1, GROUP))
    scale = t.abs().amax((1, 3), keepdim=True).clamp(min=1e-12) / 448
    codes = (t / scale).to(torch.float8_e4m3fn).flatten(2).flatten(0, 1)
    return codes[:n, :k].contiguous(), scale[:, 0, :, 0].contiguous()


def _activations(rows, k, g):
    x = torch.randn(rows, k, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    return _quantised(torch.where(torch.rand(rows, k, generator=g, device="cuda") < 1e-3, 20 * x, x))


def _prepare_product(case, g):
    rows, n, k = case["rows"], case["n"], case["k"]
    a, a_scale = _activations(rows, k, g)
    w, w_scale = _quantised_matrix(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k))
    s = {"case": case, "a": a, "a_scale": a_scale, "w": w, "w_scale": w_scale}
    if own:  # the output and the parameter block that a serving loop keeps
        import compressed_mla_attention_gb300 as Q

        s["out"] = torch.empty(rows, n, dtype=getattr(torch, case["out"]), device="cuda")
        s["params"] = Q.make_matmul_params(a=a, a_scale=a_scale, w=w, w_scale=w_scale, out=s["out"])
    return s


def _values(codes, scale, dtype):
    """The values of quantised rows."""
    n = codes.shape[-1]
    return codes.to(dtype) * scale.to(dtype).repeat_interleave(GROUP, -1)[..., :n]


def _matrix_values(codes, scale, dtype):
    n, k = codes.shape
    scale = scale.to(dtype).repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]
    return codes.to(dtype) * scale


def _run_product(s):
    if own:
        import compressed_mla_attention_gb300 as Q

        Q.matmul(s["params"])
        return s["out"]
    a, w = _values(s["a"], s["a_scale"], torch.float32), _matrix_values(s["w"], s["w_scale"], torch.float32)
    return (a @ w.t()).to(getattr(torch, s["case"]["out"]))


def _wide_product(a, a_scale, w, w_scale):
    """The sum over blocks of 128 of the codes' products times both scales, in 64 bits."""
    n, k = w.shape
    out = torch.zeros(a.shape[0], n, dtype=torch.float64, device="cuda")
    step = 32 * GROUP
    for lo in range(0, k, step):  # the scales go to the codes, block by block
        hi, b = min(k, lo + step), slice(lo // GROUP, -(-min(k, lo + step) // GROUP))
        at = torch.arange(lo, hi, device="cuda") // GROUP - lo // GROUP
        left = a[:, lo:hi].double() * a_scale[:, b].double()[:, at]
        right = w[:, lo:hi].double() * w_scale[:, b].double()[torch.arange(n, device="cuda") // GROUP][:, at]
        out.addmm_(left, right.t())
    return out


def _exact_product(case, g):
    s = _prepare_product(case, g)
    return _wide_product(s["a"], s["a_scale"], s["w"], s["w_scale"])


def _work_product(case):
    m, n, k = case["rows"], case["n"], case["k"]
    kb, size = -(-k // GROUP), 4 if case["out"] == "float32" else 2
    return {"bytes": m * k + n * k + 4 * m * kb + 4 * -(-n // GROUP) * kb + m * n * size, "flops": 2.0 * m * n * k}


# ------------------------------------------------------------------ products by group
def _prepare_grouped(case, g):
    rows, groups, n, k = case["rows"], case["groups"], case["n"], case["k"]
    host = torch.Generator().manual_seed(g.initial_seed())
    share = torch.softmax(0.6 * torch.randn(groups, generator=host), 0)  # some experts are chosen more often
    picks = torch.multinomial(share, rows - case["padded"], replacement=True, generator=host)
    bounds = [0] + torch.bincount(picks, minlength=groups).cumsum(0).tolist()
    a, a_scale = _activations(rows, k, g)
    w = torch.empty(groups, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    w_scale = torch.empty(groups, -(-n // GROUP), -(-k // GROUP), device="cuda")
    for e in range(groups):
        w[e], w_scale[e] = _quantised_matrix(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k))
    s = {"case": case, "a": a, "a_scale": a_scale, "w": w, "w_scale": w_scale, "bounds": bounds,
         "cu": torch.tensor(bounds, dtype=torch.int32).cuda(),
         "out": torch.zeros(rows, n, dtype=getattr(torch, case["out"]), device="cuda")}
    if own:  # the parameter block that a serving loop keeps
        import compressed_mla_attention_gb300 as Q

        s["params"] = Q.make_matmul_params(a=a, a_scale=a_scale, w=w, w_scale=w_scale, cu_rows=s["cu"], out=s["out"])
    return s


def _run_grouped(s):
    if own:
        import compressed_mla_attention_gb300 as Q

        Q.matmul(s["params"])
        return s["out"]
    a = _values(s["a"], s["a_scale"], torch.float32)
    for e, (lo, hi) in enumerate(zip(s["bounds"][:-1], s["bounds"][1:])):
        if hi > lo:  # rows behind the last group stay as they are
            s["out"][lo:hi] = (a[lo:hi] @ _matrix_values(s["w"][e], s["w_scale"][e], torch.float32).t()).to(s["out"].dtype)
    return s["out"]


def _exact_grouped(case, g):
    s = _prepare_grouped(case, g)
    out = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda")
    for e in range(case["groups"]):
        at = slice(s["bounds"][e], s["bounds"][e + 1])
        if at.stop > at.start:
            out[at] = _wide_product(s["a"][at], s["a_scale"][at], s["w"][e], s["w_scale"][e])
    return out


def _work_grouped(case):
    m, n, k, e = case["rows"] - case["padded"], case["n"], case["k"], case["groups"]
    kb, size = -(-k // GROUP), 4 if case["out"] == "float32" else 2
    live = sum(1 - (1 - p) ** m for p in _shares(e))  # groups with a row, on average
    return {"bytes": m * k + 4 * m * kb + live * (n * k + 4 * -(-n // GROUP) * kb) + m * n * size, "flops": 2.0 * m * n * k}


def _shares(groups):
    """The groups' shares at the middle of their distribution."""
    draws = random.Random(1)
    e = [math.exp(0.6 * draws.gauss(0, 1)) for _ in range(groups)]
    return [v / sum(e) for v in e]


# ------------------------------------------------------------------ the calls
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"quant": _prepare_quant, "product": _prepare_product, "grouped": _prepare_grouped}[case["op"]](case, g)
    return s | {"op": case["op"]}


def run(state):
    return {"quant": _run_quant, "product": _run_product, "grouped": _run_grouped}[state["op"]](state)


def work(case):
    return {"quant": _work_quant, "product": _work_product, "grouped": _work_grouped}[case["op"]](case)


def exact(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return {"quant": _exact_quant, "product": _exact_product, "grouped": _exact_grouped}[case["op"]](case, g)
