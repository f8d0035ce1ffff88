"""Plain 64-bit references of the expert-layer operators, on the CPU in numpy,
written from their definitions; and inputs whose results are exact.

Small integers (times powers of two) make every product and partial sum exactly
representable in fp32, so an fp32 output has to equal the reference bit for bit,
and a 16-bit output the reference rounded once.
"""
import numpy as np
import torch


def ints(rng, shape, lo=-4, hi=4, dtype=torch.bfloat16):
    return torch.from_numpy(rng.integers(lo, hi + 1, size=shape).astype(np.float32)).to(dtype)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def gelu_tanh(x):
    return 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)))


def gelu_erf(x):
    from math import erf
    return 0.5 * x * (1 + np.vectorize(erf)(x / np.sqrt(2)))


ACT = {"none": lambda x: x, "gelu_tanh": gelu_tanh, "gelu_erf": gelu_erf,
       "relu": lambda x: np.where(x > 0, x, 0.0)}


def activation(epilogue):
    name = epilogue[5:] if epilogue.startswith("bias_") else epilogue
    return ACT["none" if name in ("bias", "none") else name]


def grouped(A, B, offsets, C0=None, alpha=1.0, beta=0.0, bias=None, epilogue="none"):
    """Rows of no group keep C0 (or NaN)."""
    A, B = f64(A), f64(B)
    out = np.full((A.shape[0], B.shape[2]), np.nan) if C0 is None else f64(C0).copy()
    for e in range(B.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        if hi <= lo:
            continue
        y = alpha * (A[lo:hi] @ B[e])
        if beta:
            y = y + beta * out[lo:hi]
        if bias is not None:
            b = f64(bias)
            y = y + (b if b.ndim == 1 else b[e])
        out[lo:hi] = activation(epilogue)(y)
    return out


def wgrad(A, D, offsets, C0=None, alpha=1.0, beta=0.0):
    A, D = f64(A), f64(D)
    E = len(offsets) - 1
    out = np.zeros((E, A.shape[1], D.shape[1]))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        out[e] = alpha * (A[lo:hi].T @ D[lo:hi])
    if beta:
        out += beta * f64(C0)
    return out


def newton_schulz(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    a, b, c = coefficients
    X = f64(G)
    single = X.ndim == 2
    X = X[None] if single else X
    X = np.stack([x / (np.sqrt((x * x).sum()) + eps) for x in X])
    for _ in range(steps):
        S = X @ X.transpose(0, 2, 1)
        X = a * X + (b * S + c * (S @ S)) @ X
    return X[0] if single else X


def newton_schulz_fp16(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7):
    """The same with what the kernels hold between products rounded to fp16: X times
    2^13, Y = S + b / (2 c) and P = c Y Y + a - b b / (4 c) times 2^12, the result as it
    is; all products in 64 bits, S on the smaller side.  What Y's diagonal loses, r_i, comes
    back in P's as 2 c r_i Y_ii."""
    a, b, c = coefficients

    def fp16(x, scale=1.0):
        return (x * scale).astype(np.float16).astype(np.float64) / scale

    def one(x):
        X = fp16(x / (np.sqrt((x * x).sum()) + eps), 2.0 ** 13)
        wide = X.shape[0] <= X.shape[1]
        eye = np.eye(min(X.shape))
        for step in range(steps):
            exact = (X @ X.T if wide else X.T @ X) + b / (2 * c) * eye
            Y = fp16(exact, 2.0 ** 12)
            lost = np.diag(2 * c * np.diag(exact - Y) * np.diag(Y))
            P = fp16(c * (Y @ Y) + (a - b * b / (4 * c)) * eye + lost, 2.0 ** 12)
            X = P @ X if wide else X @ P
            X = fp16(X, 1.0 if step == steps - 1 else 2.0 ** 13)
        return X

    G = f64(G)
    return one(G) if G.ndim == 2 else np.stack([one(x) for x in G])


def w4_weights(q, scales, zeros):
    """[..., N, K] weights of packed q [..., N, K / 2]."""
    q = q.cpu().numpy().astype(np.int64)
    s = f64(scales)
    w = np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], q.shape[-1] * 2).astype(float)
    group = w.shape[-1] // s.shape[-1]
    z = 8.0 if zeros is None else np.repeat(zeros.cpu().numpy().astype(float), group, axis=-1)
    return (w - z) * np.repeat(s, group, axis=-1)


def w4(x, q, scales, zeros=None, offsets=None, bias=None, epilogue="none"):
    W = w4_weights(q, scales, zeros)
    if offsets is None:
        W = W[None]
        offsets = [0, x.shape[0]]
    return grouped(x, torch.from_numpy(W.transpose(0, 2, 1)), offsets, bias=bias,
                   epilogue=epilogue)


def rounded(ref, dtype):
    """The 64-bit reference rounded once to `dtype`, as 64 bits.  (The exact cases
    fit fp32, so going through it rounds nothing twice.)"""
    return torch.from_numpy(ref.astype(np.float32)).to(dtype).to(torch.float64).numpy()
