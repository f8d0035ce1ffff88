"""The measured cases of an expert layer's routing and of its products in 8-bit
integers: tokens sorted by expert (``dispatch``), the experts' rows added up again
with the router's weights (``combine``) and the gradient of that (``combine_grad``);
rows quantised to 8 bits (``quantize``) and products of 8-bit integers with a scale
for each token and each output channel (``i8``).

``run(state)`` is one call of one operator: with ``own`` false in plain torch
operations, with ``own`` true through ``dense_gemm_bf16_gb300``.  ``exact`` evaluates
the definition in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "i8": torch.int8,
       "i32": torch.int32, "i64": torch.int64}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1, "i32": 4, "i64": 8}


def listed():
    return [
        # A decoding batch's tokens, quantised before they are copied to their experts'
        # rows (a byte an element to move), ids as a top-k call leaves them.
        dict(name="dispatch_decode", op="dispatch", dtype="i8", ids="i64", T=48, top=4, E=64,
             K=2048, skew=0.8, drop=0.0),
        # A training step's tokens.
        dict(name="dispatch_train", op="dispatch", dtype="bf16", ids="i32", T=16384, top=4, E=64,
             K=2048, skew=0.5, drop=0.0),
        # The decoding batch's expert outputs, added up per token.
        dict(name="combine_decode", op="combine", dtype="f16", weights="f32", out="f16", T=48,
             top=4, E=64, K=2048, skew=0.8, drop=0.0),
        # The training step's.
        dict(name="combine_train", op="combine", dtype="bf16", weights="f32", out="bf16", T=16384,
             top=4, E=64, K=2048, skew=0.5, drop=0.0),
        # A small step with rows that are no multiple of 16 bytes, and some tokens that
        # a capacity limit kept from an expert.
        dict(name="combine_grad_odd", op="combine_grad", dtype="f16", weights="f32", T=3001, top=6,
             E=160, K=1001, skew=1.0, drop=0.1),
        # The training step's gradient: of the experts' outputs and of the weights.
        dict(name="combine_grad_train", op="combine_grad", dtype="bf16", weights="f32", T=16384,
             top=4, E=64, K=2048, skew=0.5, drop=0.0),
        # A prompt's activations, token by token.
        dict(name="quantize_prompt", op="quantize", dtype="bf16", T=4096, K=4096),
        # An fp32 weight matrix, output channel by output channel, odd sizes.
        dict(name="quantize_weights_odd", op="quantize", dtype="f32", T=1001, K=7001),
        # One token, as 16-bit activations, times one matrix: bound by its 67 MB.
        dict(name="i8_one_token", op="i8", dtype="bf16", out="bf16", T=1, E=0, K=8192, N=8192,
             skew=0.0, epilogue="none"),
        # A decoding batch of 48 tokens x 4 experts, unevenly spread.
        dict(name="i8_decode_batch", op="i8", dtype="i8", out="bf16", T=192, E=64, K=2048, N=2048,
             skew=0.8, epilogue="none"),
        # A prompt through one matrix, its activations quantised on the way.
        dict(name="i8_prompt", op="i8", dtype="bf16", out="bf16", T=1500, E=0, K=4096, N=4096,
             skew=0.0, epilogue="bias"),
        # A batch of prompts through an expert layer's first product, the largest work here.
        dict(name="i8_experts_prompt", op="i8", dtype="i8", out="f16", T=16384, E=16, K=2048,
             N=4096, skew=0.5, epilogue="bias_gelu_tanh"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _width(rng, lo, hi):
    """A feature count: a multiple of 16 three times in four, any number else."""
    n = _log_int(rng, lo, hi)
    return max(16, n // 16 * 16) if rng.random() < 0.75 else n


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine_grad", "quantize", "i8", "i8"])
    if op == "quantize":
        c = dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), T=_log_int(rng, 1, 16384),
                 K=_width(rng, 16, 16384))
        while c["T"] * c["K"] > 1 << 26:
            c["T"] = c["T"] * 3 // 4
        return c
    if op == "i8":
        c = dict(op=op, dtype=rng.choice(["i8", "i8", "bf16", "f16"]),
                 out=rng.choice(["bf16", "f16", "f32"]), T=_log_int(rng, 1, 16384),
                 E=rng.choice([0, 0, _log_int(rng, 1, 64)]), K=_width(rng, 64, 8192),
                 N=_width(rng, 64, 8192), skew=rng.choice([0.0, 0.5, 1.0]),
                 epilogue=rng.choice(["none", "none", "bias", "bias_gelu_tanh"]))
        while max(c["E"], 1) * c["K"] * c["N"] > 1 << 28:
            c["E"], c["N"] = c["E"] // 2, c["N"] if c["E"] > 1 else c["N"] // 2
        while 2 * c["T"] * c["K"] * c["N"] > 2.7e11:
            c["T"] = c["T"] * 3 // 4
        return c
    E = _log_int(rng, 2, 256)
    c = dict(op=op, T=_log_int(rng, 1, 16384), top=min(E, rng.choice([1, 2, 3, 4, 6, 8])), E=E,
             K=_width(rng, 64, 4096), skew=rng.choice([0.0, 0.5, 1.0]),
             drop=rng.choice([0.0, 0.0, 0.1]))
    if op == "dispatch":
        c["dtype"] = rng.choice(["bf16", "f16", "f32", "i8"])
        c["ids"] = rng.choice(["i32", "i64"])
    else:
        c["dtype"] = rng.choice(["bf16", "f16", "f32"])
        c["weights"] = rng.choice(["f32", "f32", c["dtype"]])
        if op == "combine":
            c["out"] = rng.choice([c["dtype"], "f32"])
    while c["T"] * c["top"] * c["K"] * _BYTES[c["dtype"]] > 1 << 28:
        c["T"] = c["T"] * 3 // 4
    return c


def _counts(c):
    """Rows of each group of a product, largest first: T rows spread in proportion to
    1 / rank^skew, every rest to the largest remainders."""
    T, E = c["T"], c["E"]
    w = [1.0 / (i + 1) ** c["skew"] for i in range(E)]
    share = [T * v / sum(w) for v in w]
    n = [int(s) for s in share]
    order = sorted(range(E), key=lambda i: (n[i] - share[i], i))
    for i in order[:T - sum(n)]:
        n[i] += 1
    return n


def work(case):
    c = case
    T, K, ab = c["T"], c["K"], _BYTES[c["dtype"]]
    if c["op"] == "quantize":
        return {"bytes": float(T * K * (ab + 1) + T * 4), "flops": 2.0 * T * K}
    if c["op"] == "i8":
        N = c["N"]
        active = sum(1 for v in _counts(c) if v > 0) if c["E"] else 1
        n = T * K * ab + active * N * (K + 4) + T * N * _BYTES[c["out"]]
        n += T * 4 if c["dtype"] == "i8" else 0
        n += (c["E"] + 1) * 4 if c["E"] else 0
        n += active * N * 4 if c["epilogue"] != "none" else 0
        return {"bytes": float(n), "flops": 2.0 * T * K * N}
    pairs = T * c["top"] * (1.0 - c["drop"])  # (token, expert) pairs that have a row
    slots = T * c["top"] * 4
    if c["op"] == "dispatch":
        n = T * c["top"] * _BYTES[c["ids"]] + T * K * ab + pairs * K * ab + slots + (c["E"] + 1) * 4
        if c["dtype"] == "i8":
            n += T * 4 + pairs * 4
        return {"bytes": float(n), "flops": 0.0}
    weights = T * c["top"] * _BYTES[c["weights"]]
    if c["op"] == "combine":
        return {"bytes": float(pairs * K * ab + slots + weights + T * K * _BYTES[c["out"]]),
                "flops": 2.0 * pairs * K}
    return {"bytes": float(T * K * ab + 2 * pairs * K * ab + slots + 2 * weights),
            "flops": 3.0 * pairs * K}


def _route(c, g):
    """[T, top] expert ids, distinct per token, experts drawn unevenly; -1 where a pair
    was dropped."""
    rank = torch.randperm(c["E"], generator=g, device="cuda")
    popular = -c["skew"] * torch.log(rank.float() + 1.0)
    noise = -torch.log(-torch.log(torch.rand((c["T"], c["E"]), generator=g, device="cuda")
                                  .clamp(1e-9, 1.0 - 1e-7)))
    ids = torch.topk(popular + noise, c["top"], dim=1).indices
    if c["drop"]:
        gone = torch.rand(ids.shape, generator=g, device="cuda") < c["drop"]
        ids = ids.masked_fill(gone, -1)
    return ids


def _places(ids, E):
    """Offsets of the experts' rows, and every pair's row, -1 without one: rows stand in
    the order of expert, then token, then choice."""
    flat = ids.reshape(-1).to(torch.int32)
    hit = torch.arange(E, device=flat.device, dtype=torch.int32)[:, None] == flat
    seen = torch.cumsum(hit, dim=1, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.cumsum(seen[:, -1], dim=0)
    e = flat.clamp(min=0).long()
    slot = offsets[e] + seen.gather(0, e[None])[0] - 1
    return offsets, torch.where(flat >= 0, slot, -1).reshape(ids.shape)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]
    T, K = c["T"], c["K"]

    def normal(shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    def integers(shape):
        return normal(shape, 40.0).round_().clamp_(-127, 127).to(torch.int8)

    def positive(shape, scale):
        return (torch.rand(shape, generator=g, device="cuda") + 0.5) * scale

    s = dict(case=dict(c))
    if c["op"] == "quantize":
        # tokens (or channels) of different sizes, some entries far out
        s["x"] = (normal((T, K)) * torch.exp(normal((T, 1))) *
                  (1.0 + 20.0 * (torch.rand((1, K), generator=g, device="cuda") < 0.01))).to(dt)
        return s
    if c["op"] == "i8":
        N = c["N"]
        lead = (c["E"],) if c["E"] else ()
        if c["E"]:
            counts = _counts(c)
            random.Random(seed).shuffle(counts)
            bounds = [0]
            for v in counts:
                bounds.append(bounds[-1] + v)
            s["bounds"] = bounds
            s["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        if c["dtype"] == "i8":
            s["x"] = integers((T, K))
            s["x_scales"] = positive((T,), 0.02)
        else:
            s["x"] = (normal((T, K)) * torch.exp(0.5 * normal((T, 1)))).to(dt)
        s["q"] = integers(lead + (N, K))
        s["scales"] = positive(lead + (N,), 0.03 * K ** -0.5)
        if c["epilogue"] != "none":
            s["bias"] = normal(lead + (N,), 0.5)
        return s
    ids = _route(c, g)
    if c["op"] == "dispatch":
        s["ids"] = ids.to(_DT[c["ids"]])
        rows = (T * c["top"], K)
        if c["dtype"] == "i8":
            s["x"] = integers((T, K))
            s["scales"] = positive((T,), 0.02)
            s["rows_scales"] = torch.zeros(rows[0], device="cuda")
        else:
            s["x"] = normal((T, K)).to(dt)
        # the program's buffers: rows past the last expert's keep what they held
        s["rows"] = torch.zeros(rows, dtype=dt, device="cuda")
        return s
    _, s["slots"] = _places(ids, c["E"])
    w = torch.rand(ids.shape, generator=g, device="cuda") + 0.05
    s["weights"] = (w / w.sum(dim=1, keepdim=True)).to(_DT[c["weights"]])
    s["ys"] = normal((T * c["top"], K)).to(dt)
    if c["op"] == "combine_grad":
        s["dy"] = normal((T, K), 1e-2).to(dt)
        s["d_rows"] = torch.zeros_like(s["ys"])
    return s


def _quantize(x, dtype=torch.float32):
    """Row by row: scale = max |x| / 127, q = x / scale to the nearest integer.  The
    quotient decides between two integers, so it is taken in 64 bits."""
    wide = x.to(torch.float64)
    top = wide.abs().amax(dim=-1, keepdim=True)
    q = torch.where(top > 0, torch.round(127.0 * wide / top), 0.0)
    return q, (top[..., 0] / 127.0).to(dtype)


def _gelu_tanh(x):
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _plain_i8(s):
    c = s["case"]
    f32 = torch.float32
    if c["dtype"] == "i8":
        x, sx = s["x"].to(f32), s["x_scales"]
    else:
        x, sx = _quantize(s["x"])
        x = x.to(f32)
    y = torch.empty((c["T"], c["N"]), dtype=f32, device=x.device)
    bounds = s.get("bounds", [0, c["T"]])
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi == lo:
            continue
        q, sw = (s["q"][e], s["scales"][e]) if c["E"] else (s["q"], s["scales"])
        v = (x[lo:hi] @ q.to(f32).transpose(0, 1)) * sx[lo:hi, None] * sw
        if c["epilogue"] != "none":
            v = v + (s["bias"][e] if c["E"] else s["bias"])
        y[lo:hi] = _gelu_tanh(v) if c["epilogue"].endswith("gelu_tanh") else v
    return y.to(_DT[c["out"]])


def _plain(s):
    c = s["case"]
    f32 = torch.float32
    if c["op"] == "quantize":
        q, scales = _quantize(s["x"])
        return q.to(torch.int8), scales
    if c["op"] == "i8":
        return _plain_i8(s)
    if c["op"] == "dispatch":
        offsets, slots = _places(s["ids"], c["E"])
        flat = slots.reshape(-1).long()
        pair = torch.nonzero(flat >= 0)[:, 0]
        s["rows"][flat[pair]] = s["x"][pair // c["top"]]
        if "scales" not in s:
            return s["rows"], offsets, slots
        s["rows_scales"][flat[pair]] = s["scales"][pair // c["top"]]
        return s["rows"], offsets, slots, s["rows_scales"]
    slots = s["slots"].long()
    has = (slots >= 0)[..., None]
    at = slots.clamp(min=0)
    w = torch.where(has, s["weights"].to(f32)[..., None], 0.0)
    if c["op"] == "combine":
        y = torch.zeros((c["T"], c["K"]), dtype=f32, device=at.device)
        for j in range(c["top"]):
            y += torch.where(has[:, j], w[:, j] * s["ys"][at[:, j]].to(f32), 0.0)
        return y.to(_DT[c["out"]])
    dy = s["dy"].to(f32)
    d_weights = torch.zeros(slots.shape, dtype=f32, device=at.device)
    for j in range(c["top"]):
        t = torch.nonzero(has[:, j, 0])[:, 0]
        s["d_rows"][at[t, j]] = (w[t, j] * dy[t]).to(s["d_rows"].dtype)
        d_weights[t, j] = (dy[t] * s["ys"][at[t, j]].to(f32)).sum(dim=1)
    return s["d_rows"], d_weights.to(s["weights"].dtype)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain(s)
    import dense_gemm_bf16_gb300 as dg

    if c["op"] == "quantize":
        return dg.i8_quantize(s["x"])
    if c["op"] == "i8":
        return dg.i8_gemm(s["x"], s["q"], s["scales"], x_scales=s.get("x_scales"),
                          offsets=s.get("offsets"), bias=s.get("bias"), epilogue=c["epilogue"],
                          out_dtype=_DT[c["out"]])
    if c["op"] == "dispatch":
        return dg.expert_dispatch(s["x"], s["ids"], c["E"], scales=s.get("scales"), out=s["rows"],
                                  out_scales=s.get("rows_scales"))
    if c["op"] == "combine":
        return dg.expert_combine(s["ys"], s["slots"], s["weights"], out_dtype=_DT[c["out"]])
    return dg.expert_combine_grad(s["dy"], s["slots"], s["weights"], rows=s["ys"],
                                  out=s["d_rows"])


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    f64 = torch.float64
    T, K = c["T"], c["K"]

    def integers_of(x):
        # 127 x is exact in 64 bits, so a quotient halfway between two integers is found
        # as such (with x / scale the scale's own rounding would decide it)
        x = x.to(f64)
        top = torch.linalg.vector_norm(x, ord=math.inf, dim=1)
        return torch.round((x * 127.0) / torch.where(top > 0, top, 1.0)[:, None]), top / 127.0

    if c["op"] == "quantize":
        q, scales = integers_of(s["x"])
        return q.to(torch.int8), scales
    if c["op"] == "i8":
        N = c["N"]
        if c["dtype"] == "i8":
            x, sx = s["x"].to(f64), s["x_scales"].to(f64)
        else:
            x, sx = integers_of(s["x"])
        bounds = s["bounds"] if c["E"] else [0, T]
        q = s["q"] if c["E"] else s["q"][None]
        sw = s["scales"].to(f64).reshape(-1, N)
        parts = []
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            if hi == lo:
                continue
            y = torch.einsum("tk,nk->tn", x[lo:hi] * sx[lo:hi, None], q[e].to(f64) * sw[e][:, None])
            if c["epilogue"] != "none":
                y = y + s["bias"].to(f64).reshape(-1, N)[e]
            if c["epilogue"].endswith("gelu_tanh"):
                y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
            parts.append(y)
        return torch.cat(parts)
    if c["op"] == "dispatch":
        flat = s["ids"].reshape(-1).cpu().tolist()
        order = sorted((e, i) for i, e in enumerate(flat) if e >= 0)
        slots, offsets = [-1] * len(flat), [0] * (c["E"] + 1)
        for row, (e, i) in enumerate(order):
            slots[i] = row
            offsets[e + 1] = row + 1
        for e in range(c["E"]):
            offsets[e + 1] = max(offsets[e + 1], offsets[e])
        token = torch.tensor([i // c["top"] for _, i in order], dtype=torch.long, device="cuda")
        rows = s["rows"].clone()
        rows[:len(order)] = s["x"][token]
        ints = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (offsets, slots)]
        out = (rows if c["dtype"] == "i8" else rows.to(f64), ints[0], ints[1].reshape(T, c["top"]))
        if c["dtype"] != "i8":
            return out
        scales = torch.zeros(len(flat), dtype=f64, device="cuda")
        scales[:len(order)] = s["scales"].to(f64)[token]
        return out + (scales,)
    # by sorted row: its pair, its token
    flat = s["slots"].reshape(-1).long()
    pair = torch.nonzero(flat >= 0)[:, 0]
    token, row = pair // c["top"], flat[pair]
    w = s["weights"].to(f64).reshape(-1)[pair][:, None]
    if c["op"] == "combine":
        y = torch.zeros((T, K), dtype=f64, device="cuda")
        return y.index_add_(0, token, s["ys"][row].to(f64) * w)
    dy = s["dy"].to(f64)[token]
    d_rows = torch.zeros(s["ys"].shape, dtype=f64, device="cuda")
    d_rows[row] = dy * w
    d_weights = torch.zeros(flat.shape, dtype=f64, device="cuda")
    d_weights[pair] = torch.einsum("pk,pk->p", dy, s["ys"][row].to(f64))
    return d_rows, d_weights.reshape(T, c["top"])
