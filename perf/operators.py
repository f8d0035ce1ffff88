"""The measured cases of the expert-layer operators: products grouped by expert
with ragged row counts, their weight gradient, the orthogonalised update
(Newton-Schulz products) and the products with 4-bit weights.

``run(state)`` is one call of one operator: with ``own`` false in plain fp32
torch operations, with ``own`` true through ``dense_gemm_bf16_gb300``.
``exact`` evaluates the definition in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}

# The quintic's coefficients and the step count that matrix-orthogonalising
# optimisers use, and their guard of the norm.
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # One token routed to 8 of 64 experts: the smallest serving step, bound
        # by the 8 weight matrices that have to be read.
        dict(name="rows_one_token", op="rows", dtype="bf16", out="bf16", T=8, E=64, K=2048,
             N=1024, layout="col", skew=0.0, epilogue="none"),
        # A decoding batch of 48 tokens x 4 experts, unevenly spread.
        dict(name="rows_decode_batch", op="rows", dtype="bf16", out="bf16", T=192, E=64, K=2048,
             N=2048, layout="row", skew=0.8, epilogue="none"),
        # A training step's first product, bias and GELU fused.
        dict(name="rows_train", op="rows", dtype="bf16", out="bf16", T=16384, E=16, K=2048,
             N=4096, layout="col", skew=0.5, epilogue="bias_gelu_tanh"),
        # The gradient of a layer's input (the other weight layout), odd sizes.
        dict(name="rows_input_grad_odd", op="rows", dtype="f16", out="f16", T=7001, E=24, K=1496,
             N=1000, layout="row", skew=1.0, epilogue="none"),
        # The weights' gradient of the training step, kept in fp32.
        dict(name="wgrad_train", op="wgrad", dtype="bf16", out="f32", T=16384, E=16, K=2048,
             N=4096, skew=0.5),
        # Many small experts with few tokens each, some with none.
        dict(name="wgrad_small_experts", op="wgrad", dtype="f16", out="f16", T=3001, E=64, K=520,
             N=1000, skew=1.2),
        # The update of one small matrix: latency of the chain of products.
        dict(name="orth_small", op="orth", dtype="f32", out="bf16", B=1, M=256, N=256),
        # The updates of a layer's experts, one batch.
        dict(name="orth_experts", op="orth", dtype="f32", out="bf16", B=16, M=1024, N=2048),
        # The update of one large matrix, the largest amount of work here.
        dict(name="orth_large", op="orth", dtype="bf16", out="bf16", B=1, M=4096, N=4096),
        # One token times one 4-bit matrix.
        dict(name="w4_one_token", op="w4", dtype="bf16", out="bf16", T=1, E=0, K=8192, N=8192,
             group=128, zeros=False, skew=0.0),
        # Tokens routed to 4-bit experts, small groups, zero points.
        dict(name="w4_experts", op="w4", dtype="f16", out="f16", T=32, E=32, K=2048, N=4096,
             group=32, zeros=True, skew=0.8),
        # A prompt through a 4-bit matrix.
        dict(name="w4_prompt", op="w4", dtype="bf16", out="bf16", T=1500, E=0, K=4096, N=4096,
             group=64, zeros=True, skew=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _width(rng, lo, hi, step=8):
    """A feature count: a multiple of `step` three times in four, any number else."""
    n = _log_int(rng, lo, hi)
    if step > 8 or rng.random() < 0.75:
        n = max(step, n // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["rows", "rows", "wgrad", "orth", "w4", "w4"])
    if op in ("rows", "wgrad"):
        c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), T=_log_int(rng, 1, 16384),
                 E=_log_int(rng, 1, 64), K=_width(rng, 128, 4096), N=_width(rng, 128, 4096),
                 skew=rng.choice([0.0, 0.5, 1.0, 1.5]))
        c["out"] = rng.choice([c["dtype"], "f32"])
        while c["E"] * c["K"] * c["N"] > 1 << 28:
            c["E"] = max(1, c["E"] // 2)
        while 2 * c["T"] * c["K"] * c["N"] > 2.7e11:
            c["T"] = c["T"] * 3 // 4
        if op == "rows":
            c["layout"] = rng.choice(["row", "col"])
            c["epilogue"] = rng.choice(["none", "none", "bias", "bias_gelu_tanh"])
    elif op == "orth":
        c = dict(op=op, dtype=rng.choice(["f32", "bf16"]), out="bf16", B=_log_int(rng, 1, 32),
                 M=_width(rng, 64, 4096), N=_width(rng, 64, 4096))
        while c["B"] > 1 and _orth_flops(c) > 1.0e12:
            c["B"] //= 2
    else:
        c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), T=_log_int(rng, 1, 1500),
                 E=rng.choice([0, 0, 8, 32]), K=_width(rng, 512, 8192, 128),
                 N=_width(rng, 512, 8192), group=rng.choice([32, 64, 128]),
                 zeros=rng.choice([False, True]), skew=rng.choice([0.0, 0.8]))
        c["out"] = c["dtype"]
        while max(c["E"], 1) * c["K"] * c["N"] > 1 << 28:
            c["N"] = c["N"] // 2
    return c


def _orth_flops(c):
    """Five steps of A = X X^T, B = b A + c A A, X = a X + B X on the smaller
    side m, where both symmetric products need half of their entries."""
    m, n = min(c["M"], c["N"]), max(c["M"], c["N"])
    return c["B"] * 5.0 * (m * (m + 1.0) * n + m * (m + 1.0) * m + 2.0 * m * m * n)


def _counts(c):
    """Rows of each group, largest first: T rows spread in proportion to
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
    if c["op"] == "orth":
        e = c["B"] * c["M"] * c["N"]
        return {"bytes": float(e * (_BYTES[c["dtype"]] + _BYTES[c["out"]])),
                "flops": _orth_flops(c)}
    T, K, N = c["T"], c["K"], c["N"]
    ab, out = _BYTES[c["dtype"]], _BYTES[c["out"]]
    flops = 2.0 * T * K * N
    if c["op"] == "wgrad":
        nbytes = T * (K + N) * ab + c["E"] * K * N * out + (c["E"] + 1) * 4
    else:
        active = sum(1 for v in _counts(c) if v > 0) if c["E"] else 1
        nbytes = T * K * ab + T * N * out
        if c["op"] == "rows":
            nbytes += active * K * N * ab + (c["E"] + 1) * 4
            if c["epilogue"] != "none":
                nbytes += active * N * 4
        else:
            nbytes += active * (K * N // 2 + N * (K // c["group"]) * (ab + (1 if c["zeros"] else 0)))
            if c["E"]:
                nbytes += (c["E"] + 1) * 4
    return {"bytes": float(nbytes), "flops": flops}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case=dict(c), out=_DT[c["out"]])
    if c["op"] == "orth":
        # a momentum: noise, and a few directions in which the gradients agree
        b, m, n = c["B"], c["M"], c["N"]
        u = torch.randn((b, m, 4), generator=g, device="cuda")
        v = torch.randn((b, 4, n), generator=g, device="cuda")
        x = torch.randn((b, m, n), generator=g, device="cuda")
        s["G"] = (1e-3 * (x + u @ v)).to(dt)
        return s
    T, K, N = c["T"], c["K"], c["N"]
    if c.get("E"):
        counts = _counts(c)
        random.Random(seed).shuffle(counts)
        bounds = [0]
        for v in counts:
            bounds.append(bounds[-1] + v)
        s["bounds"] = bounds
        s["offsets"] = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    E = max(c["E"], 1)
    s["x"] = normal((T, K))
    if c["op"] == "rows":
        if c["layout"] == "row":
            s["w"] = normal((E, K, N), K ** -0.5)
        else:
            s["w"] = normal((E, N, K), K ** -0.5).transpose(1, 2)
        if c["epilogue"] != "none":
            s["bias"] = normal((E, N), 0.5, torch.float32)
    elif c["op"] == "wgrad":
        s["d"] = normal((T, N), T ** -0.5)
    else:
        lead = (E,) if c["E"] else ()
        s["q"] = torch.randint(0, 256, lead + (N, K // 2), generator=g, device="cuda",
                               dtype=torch.uint8)
        groups = lead + (N, K // c["group"])
        s["scales"] = (torch.rand(groups, generator=g, device="cuda") * 0.5 + 0.5).mul(
            0.25 * K ** -0.5).to(dt)
        if c["zeros"]:
            s["zeros"] = torch.randint(4, 12, groups, generator=g, device="cuda",
                                       dtype=torch.uint8)
    return s


def _gelu_tanh(x):
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _activate(y, s, e):
    epilogue = s["case"]["epilogue"]
    if epilogue != "none":
        y = y + s["bias"][e].to(y.dtype)
    return _gelu_tanh(y) if epilogue.endswith("gelu_tanh") else y


def _dequantise(s, e, dtype):
    """w[n, k] = (q[n, k] - z[n, k / group]) * scale[n, k / group]; k even in
    the low half of byte k / 2; z = 8 without zero points."""
    c = s["case"]
    pick = (lambda t: t[e]) if c["E"] else (lambda t: t)
    q = pick(s["q"])
    w = torch.stack((q & 15, q >> 4), dim=-1).reshape(c["N"], c["K"] // c["group"], c["group"])
    w = w.to(dtype)
    w = w - (pick(s["zeros"]).to(dtype).unsqueeze(-1) if c["zeros"] else 8.0)
    return (w * pick(s["scales"]).to(dtype).unsqueeze(-1)).reshape(c["N"], c["K"])


def _orthogonalise(x):
    a, b, c = COEFFICIENTS
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2)
    x = x / ((x * x).sum(dim=(-1, -2), keepdim=True).sqrt() + EPS)
    for _ in range(5):
        p = x @ x.transpose(-1, -2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(-1, -2) if tall else x


def _plain(s, dtype):
    """The operator in elementary operations of the given precision."""
    c = s["case"]
    if c["op"] == "orth":
        return _orthogonalise(s["G"].to(dtype))
    x = s["x"].to(dtype)
    if c["op"] == "wgrad":
        d = s["d"].to(dtype)
        y = torch.zeros((c["E"], c["K"], c["N"]), dtype=dtype, device=x.device)
        for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            if hi > lo:
                y[e] = x[lo:hi].transpose(0, 1) @ d[lo:hi]
        return y
    if not c["E"]:
        return x @ _dequantise(s, 0, dtype).transpose(0, 1)
    y = torch.empty((c["T"], c["N"]), dtype=dtype, device=x.device)
    for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        if hi > lo:
            if c["op"] == "rows":
                y[lo:hi] = _activate(x[lo:hi] @ s["w"][e].to(dtype), s, e)
            else:
                y[lo:hi] = x[lo:hi] @ _dequantise(s, e, dtype).transpose(0, 1)
    return y


def run(state):
    s = state
    c = s["case"]
    if not own:
        return _plain(s, torch.float32).to(s["out"])
    import dense_gemm_bf16_gb300 as dg

    if c["op"] == "rows":
        return dg.grouped_gemm(s["x"], s["w"], s["offsets"], bias=s.get("bias"),
                               epilogue=c["epilogue"], out_dtype=s["out"])
    if c["op"] == "wgrad":
        return dg.grouped_gemm_wgrad(s["x"], s["d"], s["offsets"], out_dtype=s["out"])
    if c["op"] == "orth":
        return dg.newton_schulz(s["G"], out_dtype=s["out"], steps=5, coefficients=COEFFICIENTS,
                                eps=EPS)
    return dg.w4_gemm(s["x"], s["q"], s["scales"], zeros=s.get("zeros"), offsets=s.get("offsets"),
                      out_dtype=s["out"])


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    f64 = torch.float64
    if c["op"] == "orth":
        a, b, cc = COEFFICIENTS
        x = s["G"].to(f64)
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
        for _ in range(5):
            if c["M"] <= c["N"]:
                p = torch.bmm(x, x.mT)
                x = a * x + b * torch.bmm(p, x) + cc * torch.bmm(p, torch.bmm(p, x))
            else:
                p = torch.bmm(x.mT, x)
                x = a * x + b * torch.bmm(x, p) + cc * torch.bmm(torch.bmm(x, p), p)
        return x
    x = s["x"].to(f64)
    T, K, N = c["T"], c["K"], c["N"]
    bounds = s["bounds"] if c["E"] else [0, T]
    if c["op"] == "wgrad":
        d = s["d"].to(f64)
        return torch.stack([torch.einsum("tk,tn->kn", x[lo:hi], d[lo:hi])
                            for lo, hi in zip(bounds, bounds[1:])])
    rows = []
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi == lo:
            continue
        if c["op"] == "rows":
            y = torch.einsum("tk,kn->tn", x[lo:hi], s["w"][e].to(f64))
            if c["epilogue"] != "none":
                y = y + s["bias"][e].to(f64)
            if c["epilogue"].endswith("gelu_tanh"):
                y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
        else:
            q = (s["q"][e] if c["E"] else s["q"]).to(torch.int64)
            scale = (s["scales"][e] if c["E"] else s["scales"]).to(f64)
            w = torch.empty((N, K), dtype=f64, device="cuda")
            w[:, 0::2] = (q % 16).to(f64)
            w[:, 1::2] = (q // 16).to(f64)
            if c["zeros"]:
                z = (s["zeros"][e] if c["E"] else s["zeros"]).to(f64)
                w -= z.repeat_interleave(c["group"], dim=1)
            else:
                w -= 8.0
            y = torch.einsum("tk,nk->tn", x[lo:hi], w * scale.repeat_interleave(c["group"], dim=1))
        rows.append(y)
    return torch.cat(rows)
