"""Plain 64-bit references of the routing operators and of the 8-bit products, on the CPU
in numpy, written from their definitions."""
import numpy as np
import torch

from experts_ref import activation, f64

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINIEST = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def places(ids, experts):
    """(offsets, slots) by sorting the pairs (expert, t, j)."""
    ids = np.asarray(ids)
    T, top = ids.shape
    pairs = sorted((int(ids[t, j]), t, j) for t in range(T) for j in range(top)
                   if 0 <= ids[t, j] < experts)
    slots = np.full((T, top), -1, dtype=np.int64)
    offsets = np.zeros(experts + 1, dtype=np.int64)
    for row, (e, t, j) in enumerate(pairs):
        slots[t, j] = row
        offsets[e + 1:] += 1
    return offsets, slots


def combine(rows, slots, weights=None):
    """(y, the same sum over magnitudes)."""
    rows, slots = f64(rows), np.asarray(slots)
    T, top = slots.shape
    w = np.ones((T, top)) if weights is None else f64(weights)
    y, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(top):
            if slots[t, j] >= 0:
                y[t] += w[t, j] * rows[slots[t, j]]
                size[t] += np.abs(w[t, j] * rows[slots[t, j]])
    return y, size


def combine_grad(dy, slots, weights, rows, like):
    """(d_rows with `like` where no pair writes, d_weights, sums of magnitudes of those)."""
    dy, slots = f64(dy), np.asarray(slots)
    T, top = slots.shape
    w = np.ones((T, top)) if weights is None else f64(weights)
    d_rows = f64(like).copy()
    d_w, size = np.zeros((T, top)), np.zeros((T, top))
    for t in range(T):
        for j in range(top):
            s = slots[t, j]
            if s < 0:
                continue
            d_rows[s] = w[t, j] * dy[t]
            if rows is not None:
                r = f64(rows[s])
                d_w[t, j] = dy[t] @ r
                size[t, j] = np.abs(dy[t]) @ np.abs(r)
    return d_rows, d_w, size


def quantize(x):
    """(q, scales in 64 bits) row by row; rows of zeros or with a NaN or infinity as
    documented."""
    x = f64(x)
    top = np.abs(x).max(axis=-1, initial=0.0)
    fine = np.isfinite(x).all(axis=-1)
    q = np.zeros(x.shape)
    some = fine & (top > 0)
    q[some] = np.rint(127.0 * x[some] / top[some][..., None])  # 127 x is exact, ties show as such
    return q.astype(np.int8), np.where(fine, top / 127.0, np.nan)


def integer_sums(x, q, offsets=None):
    """Exact sums [T, N]; rows of no group are None-filled with 0."""
    x, q = np.asarray(x).astype(np.int64), np.asarray(q).astype(np.int64)
    if offsets is None:
        return x @ q.T
    out = np.zeros((x.shape[0], q.shape[1]), dtype=np.int64)
    for e in range(q.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        out[lo:hi] = x[lo:hi] @ q[e].T
    return out


def i8_bits(sums, x_scales, scales, dtype, offsets=None):
    """The result without bias and activation, bit for bit: the sum rounded to fp32, times
    the token's scale, rounded, times the channel's, rounded, then to `dtype`.  (A product
    of two fp32 numbers is exact in 64 bits.)"""
    f32 = np.float32
    v = sums.astype(f32).astype(np.float64) * np.asarray(x_scales, dtype=f32)[:, None]
    v = v.astype(f32).astype(np.float64)
    s = np.asarray(scales, dtype=f32).astype(np.float64)
    if offsets is None:
        v = v * s
    else:
        for e in range(s.shape[0]):
            v[offsets[e]:offsets[e + 1]] *= s[e]
    return torch.from_numpy(v.astype(f32)).to(dtype)


def i8(sums, x_scales, scales, offsets=None, bias=None, epilogue="none"):
    """In 64 bits; with the size of the value before the activation."""
    v = sums.astype(np.float64) * np.asarray(x_scales, dtype=np.float64)[:, None]
    s = np.asarray(scales, dtype=np.float64)
    b = None if bias is None else np.asarray(bias, dtype=np.float64)
    size = np.zeros_like(v)
    bounds = [0, v.shape[0]] if offsets is None else offsets
    for e in range(len(bounds) - 1):
        lo, hi = bounds[e], bounds[e + 1]
        v[lo:hi] *= s if s.ndim == 1 else s[e]
        size[lo:hi] = np.abs(v[lo:hi])
        if b is not None:
            v[lo:hi] += b if b.ndim == 1 else b[e]
            size[lo:hi] += np.abs(b if b.ndim == 1 else b[e])
    return activation(epilogue)(v), size
