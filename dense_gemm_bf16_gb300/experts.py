"""Tensor-level calls of the expert-layer operators (include/gemm_experts.h):
reads pointers, leading dimensions and strides off torch tensors and calls the
C entry points.  PyTorch only provides device memory and the current stream.

A decoding step calls these with kernels of ten microseconds, so the checks are
written to cost little: plain dictionaries and integers, no work for arguments
that are not given.
"""
from __future__ import annotations

import torch

from . import _abi
from .api import _DT, _EPI, check
from ._abi import Epi

_CODE = {dt: int(v) for dt, v in _DT.items()}
_CODE16 = {dt: v for dt, v in _CODE.items() if dt != torch.float32}
_EPI_CODE = {name: int(v) for name, v in _EPI.items()}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _fn(name):
    """The library's function itself (loaded once)."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_abi.lib(), name)
    return fn


_fns: dict = {}


def _wrong_device(dev, **tensors):
    """Every buffer has to be on one CUDA device: the kernels read device pointers."""
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.get_device() != dev):
            where = f"cuda:{dev}" if dev >= 0 else "one CUDA device"
            raise ValueError(f"{name} must be a CUDA tensor on {where} (it is on {t.device})")


def _require_current(dev):
    """The library launches on the current device, with that device's error word; the
    stream is the tensors' device's.  On another device both would meet foreign pointers."""
    if dev != _current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, but cuda:{_current_device()} is the "
                         "current device: make theirs current (torch.cuda.device)")


def _ld(name, t):
    """Leading dimension of a row-major matrix (the last two dimensions of t)
    with unit inner stride and rows that do not overlap."""
    r, c = t.shape[-2:]
    s = t.stride()
    if (s[-1] == 1 or c <= 1) and (r <= 1 or s[-2] >= c):
        return s[-2] if r > 1 and s[-2] > 0 else max(c, 1)
    raise ValueError(f"{name} must be row-major with unit inner stride "
                     f"(shape {tuple(t.shape)}, strides {tuple(s)})")


def _offsets(offsets, groups):
    if offsets.dtype is not torch.int32 or offsets.shape != (groups + 1,) or \
            not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 vector of groups + 1 = {groups + 1} "
                         f"values (it is {offsets.dtype} of shape {tuple(offsets.shape)})")
    return offsets.data_ptr()


def _epilogue(epilogue, bias, groups, N):
    """(epilogue, bias pointer, bias stride): bias [N] or [groups, N]."""
    if bias is None and (epilogue is None or epilogue == "none"):
        return 0, 0, 0
    if epilogue is None:
        epilogue = "bias"
    epi = _EPI_CODE.get(epilogue) if isinstance(epilogue, str) else int(epilogue)
    if epi is None and isinstance(epilogue, str):
        epi = _EPI_CODE.get(epilogue.lower())
    if epi is None:
        raise ValueError(f"unknown epilogue {epilogue!r}; one of {sorted(_EPI)}")
    if bool(epi & 1) != (bias is not None):
        raise ValueError(f"epilogue {Epi(epi).name.lower()} " +
                         ("needs a bias" if bias is None else "takes no bias"))
    if bias is None:
        return epi, 0, 0
    if bias.dtype != torch.float32 or tuple(bias.shape) not in ((N,), (groups, N)) or \
            (N > 1 and bias.stride(-1) != 1):
        raise ValueError(f"bias must be fp32 of shape ({N},) or ({groups}, {N}) with unit inner "
                         "stride")
    return epi, bias.data_ptr(), bias.stride(0) if bias.dim() == 2 and groups > 1 else 0


def _empty(shape, dtype, like, stream):
    """New memory that belongs to the stream the kernels run on: a block of another
    stream's pool may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device)):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _out(name, out, shape, dtype, like, types, stream):
    if out is None:
        if dtype is None:
            dtype = types[0]
        elif dtype not in types:
            raise TypeError(f"{name} must be one of {', '.join(str(t) for t in types)}")
        return _empty(shape, dtype, like, stream)
    if out.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (it has {tuple(out.shape)})")
    if out.dtype not in types or (dtype is not None and out.dtype != dtype):
        raise TypeError(f"{name} must be one of {', '.join(str(t) for t in types)}")
    return out


def _code16(A, B, names="A and B"):
    code = _CODE16.get(A.dtype)
    if code is None or A.dtype != B.dtype:
        raise TypeError(f"{names} must share one dtype, bfloat16 or float16")
    return code


def _scratch(workspace, need, like, stream):
    """(workspace kept alive, pointer, bytes)."""
    if workspace is None:
        if need == 0:
            return None, 0, 0
        workspace = _empty(need, torch.uint8, like, stream)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


if _raw_stream is None:
    def _raw_stream(dev):
        return torch.cuda.current_stream(dev).cuda_stream


def grouped_gemm(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor,
                 C: torch.Tensor | None = None, *, alpha=1.0, beta=0.0, bias=None, epilogue=None,
                 out_dtype=None, workspace=None, stream=None) -> torch.Tensor:
    """C[t] <- act(alpha * A[t] @ B[e] + beta * C[t] + bias[e]) for the rows t
    of every group e, rows offsets[e] .. offsets[e + 1] - 1, on the current CUDA device.

    A: [T, K] row-major; B: [groups, K, N], row- or column-major matrices (a
    ``transpose(1, 2)`` gives the gradient of A); offsets: int32 [groups + 1] on
    the device; C: [T, N] row-major (allocated when None, in ``out_dtype`` or
    A's dtype; rows of no group are not written); bias: fp32 [N] or [groups, N].
    ``epilogue`` is a name as in ``gemm``.

    Calls repeat bit for bit.  T and the number of groups choose the kernel, and with
    it the order of a row's sum; at equal ones a group's results do not depend on the
    other groups.
    """
    dt = _code16(A, B)
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)}")
    dev = A.get_device()
    if not dev == B.get_device() == offsets.get_device() or dev < 0 or C is not None or \
            bias is not None or workspace is not None:
        _wrong_device(dev, A=A, B=B, offsets=offsets, C=C, bias=bias, workspace=workspace)
    _require_current(dev)
    T, K = A.shape
    groups, _, N = B.shape
    if C is None and beta != 0.0:
        raise ValueError("beta != 0 needs an input C")
    C = _out("C", C, (T, N), out_dtype, A, (A.dtype, torch.float32), stream)
    epi, bias_ptr, stride_bias = _epilogue(epilogue, bias, groups, N)
    lda, ldc = _ld("A", A), _ld("C", C)
    sb, s1, s2 = B.stride()
    if groups <= 1:
        sb = 0
    if (s2 == 1 or N <= 1) and (K <= 1 or s1 >= N):
        lb, ldb = 0, (s1 if K > 1 else max(N, 1))
    elif (s1 == 1 or K <= 1) and (N <= 1 or s2 >= K):
        lb, ldb = 1, (s2 if N > 1 else max(K, 1))
    else:
        raise ValueError("B must hold row- or column-major matrices with unit inner stride "
                         f"(shape {tuple(B.shape)}, strides {tuple(B.stride())})")
    off = _offsets(offsets, groups)
    pa, pb = A.data_ptr(), B.data_ptr()
    need = 0
    if workspace is None and ((pa | pb | (lda | ldb | sb) * 2) & 15 or 0 < sb < ldb):
        need = _abi.gemm_grouped_workspace_size(dt, groups, T, N, K, pa, lda, pb, ldb, lb, sb)
    workspace, ws, ws_bytes = _scratch(workspace, need, A, stream)
    st = _fn("gemm_grouped")(dt, groups, T, N, K, pa, lda, pb, ldb, lb, sb, C.data_ptr(), ldc,
                             _CODE[C.dtype], off, alpha, beta, bias_ptr, stride_bias, epi, ws,
                             ws_bytes, _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return C


def grouped_gemm_wgrad(A: torch.Tensor, D: torch.Tensor, offsets: torch.Tensor,
                       C: torch.Tensor | None = None, *, alpha=1.0, beta=0.0, out_dtype=None,
                       workspace=None, stream=None) -> torch.Tensor:
    """C[e] <- alpha * A_e^T @ D_e + beta * C[e], the weights' gradient of
    ``grouped_gemm``, on the current CUDA device: A [T, M] and D [T, N] row-major,
    C [groups, M, N] (a group without rows gives beta * C[e])."""
    dt = _code16(A, D, "A and D")
    if A.dim() != 2 or D.dim() != 2 or A.shape[0] != D.shape[0]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} D{tuple(D.shape)}")
    dev = A.get_device()
    _wrong_device(dev, A=A, D=D, offsets=offsets, C=C, workspace=workspace)
    _require_current(dev)
    T, M = A.shape
    N = D.shape[1]
    groups = offsets.numel() - 1
    if groups < 0:
        raise ValueError("offsets must hold groups + 1 values")
    if C is None and beta != 0.0:
        raise ValueError("beta != 0 needs an input C")
    C = _out("C", C, (groups, M, N), out_dtype, A, (A.dtype, torch.float32), stream)
    lda, ldd, ldc = _ld("A", A), _ld("D", D), _ld("C", C)
    off = _offsets(offsets, groups)
    pa, pd = A.data_ptr(), D.data_ptr()
    need = 0
    if workspace is None and (pa | pd | (lda | ldd) * 2) & 15:
        need = _abi.gemm_grouped_wgrad_workspace_size(dt, groups, T, M, N, pa, lda, pd, ldd)
    workspace, ws, ws_bytes = _scratch(workspace, need, A, stream)
    st = _fn("gemm_grouped_wgrad")(dt, groups, T, M, N, pa, lda, pd, ldd, C.data_ptr(), ldc,
                                   C.stride(0) if groups > 1 else 0, _CODE[C.dtype], off, alpha,
                                   beta, ws, ws_bytes, _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return C


def newton_schulz(G: torch.Tensor, out: torch.Tensor | None = None, *, steps=5,
                  coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out_dtype=None,
                  workspace=None, stream=None) -> torch.Tensor:
    """The orthogonalised form of G ([M, N], or [batch, M, N] matrix by matrix):
    X = G / (||G||_F + eps), then ``steps`` times X = a X + (b S + c S S) X with
    S = X X^T.  G is fp32, bf16 or fp16; the result bf16 (default) or fp16.  Runs on
    the current CUDA device."""
    if G.dtype not in _CODE:
        raise TypeError("G must be bfloat16, float16 or float32")
    if G.dim() not in (2, 3):
        raise ValueError("G must be a 2-D or 3-D tensor")
    if len(coefficients) != 3:
        raise ValueError("coefficients must be three numbers")
    dev = G.get_device()
    _wrong_device(dev, G=G, out=out, workspace=workspace)
    _require_current(dev)
    out = _out("out", out, G.shape, out_dtype, G, (torch.bfloat16, torch.float16), stream)
    batch = G.shape[0] if G.dim() == 3 else 1
    M, N = G.shape[-2:]
    ldg, ldo = _ld("G", G), _ld("out", out)
    sg, so = (G.stride(0), out.stride(0)) if batch > 1 else (0, 0)
    need = _abi.gemm_newton_schulz_workspace_size(batch, M, N) if workspace is None else 0
    workspace, ws, ws_bytes = _scratch(workspace, need, G, stream)
    a, b, c = coefficients
    st = _fn("gemm_newton_schulz")(_CODE[G.dtype], batch, M, N, G.data_ptr(), ldg, sg,
                                   out.data_ptr(), ldo, so, _CODE[out.dtype], steps, a, b, c, eps,
                                   ws, ws_bytes, _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return out


def w4_gemm(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, *, zeros=None, offsets=None,
            out=None, bias=None, epilogue=None, out_dtype=None, workspace=None,
            stream=None) -> torch.Tensor:
    """act(x @ W^T + bias) with 4-bit weights W[n, k] = (q[n, k] - z) * s, one
    scale (and zero point, 8 without ``zeros``) per group of K // scales.shape[-1]
    neighbours along k, on the current CUDA device.

    x: [T, K] row-major; q: uint8 [N, K // 2], the low half of byte j holding
    k = 2 j; scales: [N, K // group] in x's dtype; zeros: uint8 of that shape.
    With ``offsets`` (int32 [experts + 1]) q, scales and zeros carry a leading
    expert dimension and rows offsets[e] .. offsets[e + 1] - 1 use expert e
    (rows of no expert are not written).

    An fp32 result (``out_dtype``, ``out``) and 16-bit results of up to 64 rows, or of
    40 rows an expert on average, round nothing before the output; more rows multiply
    weights that were rounded to x's dtype (unless ``Option.W4_EXACT`` is set), so a
    row's last bits may depend on how many rows the call has.
    """
    dt = _code16(x, scales, "x and scales")
    lead = 3 if offsets is not None else 2
    if x.dim() != 2 or q.dim() != lead or scales.dim() != lead:
        raise ValueError(f"x must be 2-D, q and scales {lead}-D "
                         f"({'with' if lead == 3 else 'without'} offsets)")
    dev = x.get_device()
    if not dev == q.get_device() == scales.get_device() or dev < 0 or zeros is not None or \
            offsets is not None or out is not None or bias is not None or workspace is not None:
        _wrong_device(dev, x=x, q=q, scales=scales, zeros=zeros, offsets=offsets, out=out,
                      bias=bias, workspace=workspace)
    _require_current(dev)
    T, K = x.shape
    groups = q.shape[0] if lead == 3 else 1
    N = q.shape[-2]
    if q.dtype != torch.uint8 or q.shape[-1] * 2 != K:
        raise ValueError(f"q must be uint8 of shape (..., N, {K // 2}) (it is {q.dtype} of shape "
                         f"{tuple(q.shape)})")
    n_groups = scales.shape[-1]
    if scales.shape[:-1] != q.shape[:-1] or n_groups == 0 or K % n_groups:
        raise ValueError(f"scales {tuple(scales.shape)} do not fit q {tuple(q.shape)}")
    if zeros is not None and (zeros.dtype != torch.uint8 or zeros.shape != scales.shape):
        raise ValueError("zeros must be uint8 of the shape of scales")
    if not (q.is_contiguous() and scales.is_contiguous() and
            (zeros is None or zeros.is_contiguous())):
        raise ValueError("q, scales and zeros must be contiguous")
    out = _out("out", out, (T, N), out_dtype, x, (x.dtype, torch.float32), stream)
    epi, bias_ptr, stride_bias = _epilogue(epilogue, bias, groups, N)
    ldx, ldo = _ld("x", x), _ld("out", out)
    off = _offsets(offsets, groups) if offsets is not None else 0
    px, odt = x.data_ptr(), _CODE[out.dtype]
    need = 0
    if workspace is None and ((px | ldx * 2) & 15 or T > groups):
        need = _abi.gemm_w4_workspace_size(dt, groups, T, N, K, px, ldx, odt)
    workspace, ws, ws_bytes = _scratch(workspace, need, x, stream)
    st = _fn("gemm_w4")(dt, groups, T, N, K, px, ldx, q.data_ptr(), scales.data_ptr(),
                        0 if zeros is None else zeros.data_ptr(), K // n_groups, out.data_ptr(),
                        ldo, odt, off, bias_ptr, stride_bias, epi, ws, ws_bytes,
                        _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return out


def _rows(name, t):
    """_ld of a matrix that is usually contiguous or has padded rows."""
    s0, s1 = t.stride()
    r, c = t.shape
    return s0 if s1 == 1 and s0 >= c and r > 1 else _ld(name, t)


def _elsewhere(dev, *tensors):
    """Is one of them not on CUDA device `dev`?  (_wrong_device then says which.)"""
    if dev < 0:
        return True
    for t in tensors:
        if t is not None and t.get_device() != dev:
            return True
    return False


def _slots(slots, T):
    if slots.dtype is not torch.int32 or slots.shape[0] != T or not slots.is_contiguous():
        raise ValueError(f"slots must be a contiguous int32 matrix of {T} rows (it is {slots.dtype} "
                         f"of shape {tuple(slots.shape)})")
    return slots.data_ptr()


def _pair_weights(weights, slots):
    """(pointer, dtype code, row pitch) of the weights of all pairs."""
    if weights is None:
        return 0, 0, 0
    if weights.dtype not in _CODE:
        raise TypeError("weights must be bfloat16, float16 or float32")
    if weights.shape != slots.shape:
        raise ValueError(f"weights must have the shape of slots, {tuple(slots.shape)} (they have "
                         f"{tuple(weights.shape)})")
    return weights.data_ptr(), _CODE[weights.dtype], _rows("weights", weights)


_COPIED = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4, torch.int8: 1}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
# Pairs up to which a dispatch needs no workspace (the library refuses a call that does).
_ONE_PASS = 4096


def expert_dispatch(x: torch.Tensor, ids: torch.Tensor, experts: int, *, scales=None, out=None,
                    out_scales=None, workspace=None, stream=None):
    """Tokens to the rows of their experts, on the current CUDA device: the pairs (t, j)
    that have an expert get the rows 0, 1, ... in the order of (expert, t, j).  Returns
    (rows, offsets, slots): rows[slots[t, j]] = x[t], expert e owns the rows offsets[e] ..
    offsets[e + 1] - 1, and slots[t, j] is -1 for a pair without a row.  With ``scales``
    (fp32 [T], of int8 rows) the rows' scales come fourth.

    x: [T, K] row-major, bf16, fp16, fp32 or int8; ids: int32 or int64 [T, top], the experts
    that each token chose, negative for none (ids past the last expert are reported by
    ``gemm_check_device_status`` and get no row).  ``out`` [T * top, K] and ``out_scales``
    [T * top] are allocated when None; rows past the last expert's are not written.

    The gradient of x is ``expert_combine(d_rows, slots)``.
    """
    elem_bytes, id_bytes = _COPIED.get(x.dtype), _ID_BYTES.get(ids.dtype)
    if elem_bytes is None or id_bytes is None:
        raise TypeError("x must be bfloat16, float16, float32 or int8, ids int32 or int64")
    if x.dim() != 2 or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError(f"shape mismatch: x{tuple(x.shape)} ids{tuple(ids.shape)}")
    if experts < 0:
        raise ValueError("the number of experts must not be negative")
    dev = x.get_device()
    if _elsewhere(dev, ids, scales, out, out_scales, workspace):
        _wrong_device(dev, x=x, ids=ids, scales=scales, out=out, out_scales=out_scales,
                      workspace=workspace)
    _require_current(dev)
    T, K = x.shape
    top = ids.shape[1]
    ps = po = 0
    if scales is not None:
        if scales.dtype != torch.float32 or scales.shape != (T,) or not scales.is_contiguous():
            raise ValueError(f"scales must be a contiguous fp32 vector of {T} values")
        ps = scales.data_ptr()
        out_scales = _out("out_scales", out_scales, (T * top,), None, x, (torch.float32,), stream)
        if not out_scales.is_contiguous():
            raise ValueError("out_scales must be contiguous")
        po = out_scales.data_ptr()
    elif out_scales is not None:
        raise ValueError("out_scales needs scales")
    if out is None:
        out, ldo = _empty((T * top, K), x.dtype, x, stream), max(K, 1)
    else:
        out = _out("out", out, (T * top, K), None, x, (x.dtype,), stream)
        ldo = _rows("out", out)
    offsets = _empty((experts + 1,), torch.int32, x, stream)
    slots = _empty((T, top), torch.int32, x, stream)
    need = 0
    if workspace is None and T * top > _ONE_PASS:
        need = _fn("gemm_expert_dispatch_workspace_size")(T, top, experts)
    workspace, ws, ws_bytes = _scratch(workspace, need, x, stream)
    st = _fn("gemm_expert_dispatch")(elem_bytes, T, K, x.data_ptr(), _rows("x", x), ps, id_bytes,
                                     ids.data_ptr(), _rows("ids", ids), top, experts,
                                     out.data_ptr(), ldo, po, offsets.data_ptr(), slots.data_ptr(), ws,
                                     ws_bytes, _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return (out, offsets, slots) if scales is None else (out, offsets, slots, out_scales)


def expert_combine(rows: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None, *,
                   out=None, out_dtype=None, stream=None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] * rows[slots[t, j]], the experts' rows added up per token
    (in fp32, j ascending, rounded once), on the current CUDA device.

    rows: [R, K] row-major, bf16, fp16 or fp32; slots: int32 [T, top] of ``expert_dispatch``
    (negative: no row, adds nothing); weights: [T, top] of any of the three types, or None:
    ones.  The result is [T, K] in rows' dtype or fp32."""
    code = _CODE.get(rows.dtype)
    if code is None:
        raise TypeError("rows must be bfloat16, float16 or float32")
    if rows.dim() != 2 or slots.dim() != 2:
        raise ValueError(f"shape mismatch: rows{tuple(rows.shape)} slots{tuple(slots.shape)}")
    dev = rows.get_device()
    if _elsewhere(dev, slots, weights, out):
        _wrong_device(dev, rows=rows, slots=slots, weights=weights, out=out)
    _require_current(dev)
    R, K = rows.shape
    T, top = slots.shape
    psl = _slots(slots, T)
    pw, w_dt, ldw = _pair_weights(weights, slots)
    if out is None and (out_dtype is None or out_dtype is rows.dtype):
        out, ldo = _empty((T, K), rows.dtype, rows, stream), max(K, 1)
    else:
        out = _out("out", out, (T, K), out_dtype, rows, (rows.dtype, torch.float32), stream)
        ldo = _rows("out", out)
    st = _fn("gemm_expert_combine")(code, T, K, top, rows.data_ptr(), R, _rows("rows", rows), psl,
                                    pw, w_dt, ldw, out.data_ptr(), ldo, _CODE[out.dtype],
                                    _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return out


def expert_combine_grad(dy: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor | None = None,
                        *, rows=None, out=None, stream=None):
    """The gradient of ``expert_combine``, in one pass over dy, on the current CUDA device:
    (d_rows, d_weights) with d_rows[slots[t, j]] = weights[t, j] * dy[t] and d_weights[t, j] =
    <dy[t], rows[slots[t, j]]>.

    dy: [T, K] row-major, bf16, fp16 or fp32; slots and weights as in the forward call;
    rows: the forward call's rows, or None: no gradient of the weights (None is returned for
    it).  ``out`` is [R, K] in dy's dtype (allocated with T * top rows, or as many as
    ``rows`` has, when None); rows that no pair names are not written.  d_weights has weights'
    dtype (fp32 without weights)."""
    code = _CODE.get(dy.dtype)
    if code is None:
        raise TypeError("dy must be bfloat16, float16 or float32")
    if dy.dim() != 2 or slots.dim() != 2:
        raise ValueError(f"shape mismatch: dy{tuple(dy.shape)} slots{tuple(slots.shape)}")
    dev = dy.get_device()
    if _elsewhere(dev, slots, weights, rows, out):
        _wrong_device(dev, dy=dy, slots=slots, weights=weights, rows=rows, out=out)
    _require_current(dev)
    T, K = dy.shape
    psl = _slots(slots, T)
    top = slots.shape[1]
    pw, w_dt, ldw = _pair_weights(weights, slots)
    if rows is not None:
        if rows.dtype != dy.dtype:
            raise TypeError("rows and dy must share one dtype")
        if rows.dim() != 2 or rows.shape[1] != K:
            raise ValueError(f"shape mismatch: dy{tuple(dy.shape)} rows{tuple(rows.shape)}")
    R = rows.shape[0] if rows is not None else (T * top if out is None else out.shape[0])
    out = _out("out", out, (R, K), None, dy, (dy.dtype,), stream)
    d_weights, pr, ldr, pdw, dw_dt = None, 0, 0, 0, 0
    if rows is not None:
        d_weights = _empty((T, top), torch.float32 if weights is None else weights.dtype, dy, stream)
        pr, ldr, pdw, dw_dt = rows.data_ptr(), _rows("rows", rows), d_weights.data_ptr(), \
            _CODE[d_weights.dtype]
    st = _fn("gemm_expert_combine_grad")(code, T, K, top, dy.data_ptr(), _rows("dy", dy), psl, pw,
                                         w_dt, ldw, pr, R, ldr, out.data_ptr(), _rows("out", out),
                                         pdw, dw_dt, max(top, 1),
                                         _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return out, d_weights


def i8_quantize(x: torch.Tensor, *, out=None, out_scales=None, stream=None):
    """(q, scales) with q = 127 x / max|x| to the nearest integer (ties to even) and scales =
    max|x| / 127, row by row over the last dimension, on the current CUDA device: tokens
    [T, K] over their features, weights [..., N, K] over the inputs of an output channel.

    x: bf16, fp16 or fp32, its rows one after another at one distance.  A row of zeros has the
    scale 0; a row with an infinity or a NaN has a NaN scale."""
    code = _CODE.get(x.dtype)
    if code is None:
        raise TypeError("x must be bfloat16, float16 or float32")
    if x.dim() < 2:
        raise ValueError("x must have at least two dimensions")
    dev = x.get_device()
    if _elsewhere(dev, out, out_scales):
        _wrong_device(dev, x=x, out=out, out_scales=out_scales)
    _require_current(dev)
    shape = x.shape
    if out is None:
        out, ldo = _empty(shape, torch.int8, x, stream), max(shape[-1], 1)
    else:
        out = _out("out", out, shape, None, x, (torch.int8,), stream)
        ldo = _row_pitch("out", out)
    if out_scales is None:
        out_scales = _empty(shape[:-1], torch.float32, x, stream)
    else:
        out_scales = _out("out_scales", out_scales, shape[:-1], None, x, (torch.float32,), stream)
        if not out_scales.is_contiguous():
            raise ValueError("out_scales must be contiguous")
    st = _fn("gemm_i8_quantize")(code, out_scales.numel(), shape[-1], x.data_ptr(),
                                 _row_pitch("x", x), out.data_ptr(), ldo, out_scales.data_ptr(),
                                 _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return out, out_scales


def _row_pitch(name, t):
    """Distance of neighbouring rows over all leading dimensions."""
    if t.dim() == 2:
        return _rows(name, t)
    ld = _ld(name, t)
    if t.is_contiguous():
        return ld
    step = None                             # the rows' distance, times those seen so far
    for n, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            ld = step = stride
        if stride != step or stride < t.shape[-1]:
            raise ValueError(f"{name}'s rows must lie at one distance (shape {tuple(t.shape)}, "
                             f"strides {tuple(t.stride())})")
        step *= n
    return ld


_RESULTS = (torch.bfloat16, torch.float16, torch.float32)


def i8_gemm(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, *, x_scales=None, offsets=None,
            out=None, bias=None, epilogue=None, out_dtype=None, workspace=None,
            stream=None) -> torch.Tensor:
    """act((x @ q^T) * x_scales[:, None] * scales + bias) with 8-bit integers x and q and a
    scale for each token and each output channel, on the current CUDA device.

    x: [T, K] row-major, int8 with x_scales (fp32 [T]), or bf16, fp16 or fp32, which is
    quantised row by row on the way as by ``i8_quantize``; q: int8 [N, K]; scales: fp32 [N].
    With ``offsets`` (int32 [experts + 1]) q and scales carry a leading expert dimension and
    rows offsets[e] .. offsets[e + 1] - 1 use expert e (rows of no expert are not written).
    The result is bf16 (default for int8 x, else x's dtype), fp16 or fp32.

    Sums are exact integers and the result is rounded once: a row's bits do not depend on the
    call's other rows.  NaN scales give NaN, through ReLU too.  Rows of q on 16-byte boundaries are used in place, others copied."""
    given = x.dtype is torch.int8
    if not given and x.dtype not in _CODE:
        raise TypeError("x must be int8, bfloat16, float16 or float32")
    if given != (x_scales is not None):
        raise ValueError("int8 x needs x_scales" if given else "x_scales belong to int8 x")
    if q.dtype is not torch.int8 or scales.dtype is not torch.float32:
        raise TypeError("q must be int8 and scales float32")
    lead = 3 if offsets is not None else 2
    shape = q.shape
    if x.dim() != 2 or len(shape) != lead or shape[-1] != x.shape[1] or scales.shape != shape[:-1]:
        raise ValueError(f"shape mismatch: x{tuple(x.shape)} q{tuple(shape)} "
                         f"scales{tuple(scales.shape)} "
                         f"({'with' if lead == 3 else 'without'} offsets)")
    dev = x.get_device()
    if _elsewhere(dev, q, scales, x_scales, offsets, out, bias, workspace):
        _wrong_device(dev, x=x, q=q, scales=scales, x_scales=x_scales, offsets=offsets, out=out,
                      bias=bias, workspace=workspace)
    _require_current(dev)
    T, K = x.shape
    groups = shape[0] if lead == 3 else 1
    N = shape[-2]
    if given and (x_scales.dtype is not torch.float32 or x_scales.shape != (T,) or
                  not x_scales.is_contiguous()):
        raise ValueError(f"x_scales must be a contiguous fp32 vector of {T} values")
    if N > 1 and scales.stride(-1) != 1:
        raise ValueError("scales must have unit inner stride")
    if out is None:
        if out_dtype is None:
            out_dtype = torch.bfloat16 if given else x.dtype
        code = _CODE.get(out_dtype)
        if code is None:
            raise TypeError("out must be bfloat16, float16 or float32")
        out, ldo = _empty((T, N), out_dtype, x, stream), max(N, 1)
    else:
        out = _out("out", out, (T, N), out_dtype, x, _RESULTS, stream)
        code, ldo = _CODE[out.dtype], _rows("out", out)
    epi, bias_ptr, stride_bias = _epilogue(epilogue, bias, groups, N)
    off = _offsets(offsets, groups) if offsets is not None else 0
    ldq = _rows("q", q) if lead == 2 else _ld("q", q)
    stride_q, stride_s = (q.stride(0), scales.stride(0)) if groups > 1 else (0, 0)
    dt = 3 if given else _CODE[x.dtype]
    pq = q.data_ptr()
    need = 0
    if workspace is None:
        if (pq | ldq | stride_q) & 15 or 0 < stride_q < ldq:  # (the weights are copied)
            need = _fn("gemm_i8_workspace_size")(dt, groups, T, N, K, pq, ldq, stride_q)
        else:                               # tokens as 16-bit integers, and their scales
            need = (T * (K + 63 & -64) * 2 + 255 & -256) + (0 if given else T * 4 + 255 & -256)
    workspace, ws, ws_bytes = _scratch(workspace, need, x, stream)
    st = _fn("gemm_i8")(dt, groups, T, N, K, x.data_ptr(), _rows("x", x),
                        x_scales.data_ptr() if given else 0, pq, ldq, stride_q, scales.data_ptr(),
                        stride_s, out.data_ptr(), ldo, code, off, bias_ptr, stride_bias, epi, ws,
                        ws_bytes, _raw_stream(dev) if stream is None else stream)
    if st:
        check(st)
    return out
