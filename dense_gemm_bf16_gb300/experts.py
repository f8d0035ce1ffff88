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
