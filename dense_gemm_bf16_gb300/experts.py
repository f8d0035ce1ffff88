"""Tensor-level calls of the expert-layer operators (include/gemm_experts.h):
reads pointers, leading dimensions and strides off torch tensors and calls the
C entry points.  PyTorch only provides device memory and the current stream.
"""
from __future__ import annotations

import torch

from . import _abi
from .api import _DT, _EPI, check, matrix_desc
from ._abi import Epi, Layout


def _cuda(**tensors):
    """Every buffer on one CUDA device: the kernels read device pointers."""
    dev = next(t.device for t in tensors.values() if t is not None)
    for name, t in tensors.items():
        if t is not None and (not t.is_cuda or t.device != dev):
            where = dev if dev.type == "cuda" else "one CUDA device"
            raise ValueError(f"{name} must be a CUDA tensor on {where} (it is on {t.device})")
    return dev


def _rows(name, t, what="a 2-D tensor"):
    """(pointer, leading dimension) of a row-major matrix with unit inner stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be {what}")
    try:
        ptr, ld, layout, _, _ = matrix_desc(t)
    except ValueError:
        layout = None
    if layout != Layout.ROW_MAJOR:
        raise ValueError(f"{name} must be row-major with unit inner stride "
                         f"(shape {tuple(t.shape)}, strides {tuple(t.stride())})")
    return ptr, ld


def _offsets(offsets, groups):
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 vector")
    if offsets.numel() != groups + 1:
        raise ValueError(f"offsets must hold groups + 1 = {groups + 1} values "
                         f"(it holds {offsets.numel()})")
    return offsets.data_ptr()


def _epilogue(epilogue, bias, groups, N):
    """(epilogue, bias pointer, bias stride): bias [N] or [groups, N]."""
    if epilogue is None:
        epilogue = "bias" if bias is not None else "none"
    epi = epilogue if isinstance(epilogue, Epi) else _EPI.get(str(epilogue).lower())
    if epi is None:
        raise ValueError(f"unknown epilogue {epilogue!r}; one of {sorted(_EPI)}")
    if bool(epi & Epi.BIAS) != (bias is not None):
        raise ValueError(f"epilogue {epi.name.lower()} " +
                         ("needs a bias" if bias is None else "takes no bias"))
    if bias is None:
        return epi, 0, 0
    if bias.dtype != torch.float32 or tuple(bias.shape) not in ((N,), (groups, N)) or \
            (N > 1 and bias.stride(-1) != 1):
        raise ValueError(f"bias must be fp32 of shape ({N},) or ({groups}, {N}) with unit inner "
                         "stride")
    return epi, bias.data_ptr(), bias.stride(0) if bias.dim() == 2 and groups > 1 else 0


def _out(name, out, shape, dtype, device, types):
    if dtype is not None and dtype not in types:
        raise TypeError(f"{name} must be one of {', '.join(str(t) for t in types)}")
    if out is None:
        return torch.empty(shape, dtype=dtype or types[0], device=device)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (it has {tuple(out.shape)})")
    if out.dtype not in types or (dtype is not None and out.dtype != dtype):
        raise TypeError(f"{name} must be one of {', '.join(str(t) for t in types)}")
    return out


def _pair(A, B, names="A and B"):
    if A.dtype != B.dtype or A.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{names} must share one dtype, bfloat16 or float16")
    return A.dtype


def _scratch(workspace, need, device):
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is None:
        return None, 0, 0
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream(stream, device):
    return torch.cuda.current_stream(device).cuda_stream if stream is None else stream


def grouped_gemm(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor,
                 C: torch.Tensor | None = None, *, alpha=1.0, beta=0.0, bias=None, epilogue=None,
                 out_dtype=None, workspace=None, stream=None) -> torch.Tensor:
    """C[t] <- act(alpha * A[t] @ B[e] + beta * C[t] + bias[e]) for the rows t
    of every group e, rows offsets[e] .. offsets[e + 1] - 1.

    A: [T, K] row-major; B: [groups, K, N], row- or column-major matrices (a
    ``transpose(1, 2)`` gives the gradient of A); offsets: int32 [groups + 1] on
    the device; C: [T, N] row-major (allocated when None, in ``out_dtype`` or
    A's dtype; rows of no group are not written); bias: fp32 [N] or [groups, N].
    ``epilogue`` is a name as in ``gemm``.
    """
    dtype = _pair(A, B)
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[1]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} B{tuple(B.shape)}")
    dev = _cuda(A=A, B=B, offsets=offsets, C=C, bias=bias, workspace=workspace)
    T, K = A.shape
    groups, _, N = B.shape
    if C is None and beta != 0.0:
        raise ValueError("beta != 0 needs an input C")
    C = _out("C", C, (T, N), out_dtype, dev, (dtype, torch.float32))
    epi, bias_ptr, stride_bias = _epilogue(epilogue, bias, groups, N)
    pa, lda = _rows("A", A)
    pb, ldb, lb, _, sb = matrix_desc(B)
    pc, ldc = _rows("C", C)
    off = _offsets(offsets, groups)
    dt = int(_DT[dtype])
    need = 0
    if workspace is None:
        need = _abi.gemm_grouped_workspace_size(dt, groups, T, N, K, pa, lda, pb, ldb, int(lb), sb)
    workspace, ws, ws_bytes = _scratch(workspace, need, dev)
    check(_abi.gemm_grouped(dt, groups, T, N, K, pa, lda, pb, ldb, int(lb), sb, pc, ldc,
                            int(_DT[C.dtype]), off, float(alpha), float(beta), bias_ptr,
                            stride_bias, int(epi), ws, ws_bytes, _stream(stream, dev)))
    return C


def grouped_gemm_wgrad(A: torch.Tensor, D: torch.Tensor, offsets: torch.Tensor,
                       C: torch.Tensor | None = None, *, alpha=1.0, beta=0.0, out_dtype=None,
                       workspace=None, stream=None) -> torch.Tensor:
    """C[e] <- alpha * A_e^T @ D_e + beta * C[e], the weights' gradient of
    ``grouped_gemm``: A [T, M] and D [T, N] row-major, C [groups, M, N] (a group
    without rows gives beta * C[e])."""
    dtype = _pair(A, D, "A and D")
    if A.dim() != 2 or D.dim() != 2 or A.shape[0] != D.shape[0]:
        raise ValueError(f"shape mismatch: A{tuple(A.shape)} D{tuple(D.shape)}")
    dev = _cuda(A=A, D=D, offsets=offsets, C=C, workspace=workspace)
    T, M = A.shape
    N = D.shape[1]
    groups = offsets.numel() - 1
    if groups < 0:
        raise ValueError("offsets must hold groups + 1 values")
    if C is None and beta != 0.0:
        raise ValueError("beta != 0 needs an input C")
    C = _out("C", C, (groups, M, N), out_dtype, dev, (dtype, torch.float32))
    pa, lda = _rows("A", A)
    pd, ldd = _rows("D", D)
    pc, ldc, lc, _, sc = matrix_desc(C)
    if lc != Layout.ROW_MAJOR:
        raise ValueError("C must hold row-major matrices")
    off = _offsets(offsets, groups)
    dt = int(_DT[dtype])
    need = 0
    if workspace is None:
        need = _abi.gemm_grouped_wgrad_workspace_size(dt, groups, T, M, N, pa, lda, pd, ldd)
    workspace, ws, ws_bytes = _scratch(workspace, need, dev)
    check(_abi.gemm_grouped_wgrad(dt, groups, T, M, N, pa, lda, pd, ldd, pc, ldc, sc,
                                  int(_DT[C.dtype]), off, float(alpha), float(beta), ws, ws_bytes,
                                  _stream(stream, dev)))
    return C


def newton_schulz(G: torch.Tensor, out: torch.Tensor | None = None, *, steps=5,
                  coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out_dtype=None,
                  workspace=None, stream=None) -> torch.Tensor:
    """The orthogonalised form of G ([M, N], or [batch, M, N] matrix by matrix):
    X = G / (||G||_F + eps), then ``steps`` times X = a X + (b S + c S S) X with
    S = X X^T.  G is fp32, bf16 or fp16; the result bf16 (default) or fp16."""
    if G.dtype not in _DT:
        raise TypeError("G must be bfloat16, float16 or float32")
    if G.dim() not in (2, 3):
        raise ValueError("G must be a 2-D or 3-D tensor")
    if len(coefficients) != 3:
        raise ValueError("coefficients must be three numbers")
    dev = _cuda(G=G, out=out, workspace=workspace)
    out = _out("out", out, G.shape, out_dtype, dev, (torch.bfloat16, torch.float16))
    batch = G.shape[0] if G.dim() == 3 else 1
    M, N = G.shape[-2:]
    pg, ldg, lg, _, sg = matrix_desc(G)
    po, ldo, lo, _, so = matrix_desc(out)
    if lg != Layout.ROW_MAJOR or lo != Layout.ROW_MAJOR:
        raise ValueError("G and out must hold row-major matrices")
    need = _abi.gemm_newton_schulz_workspace_size(batch, M, N) if workspace is None else 0
    workspace, ws, ws_bytes = _scratch(workspace, need, dev)
    a, b, c = (float(v) for v in coefficients)
    check(_abi.gemm_newton_schulz(int(_DT[G.dtype]), batch, M, N, pg, ldg, sg, po, ldo, so,
                                  int(_DT[out.dtype]), int(steps), a, b, c, float(eps), ws,
                                  ws_bytes, _stream(stream, dev)))
    return out


def w4_gemm(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, *, zeros=None, offsets=None,
            out=None, bias=None, epilogue=None, out_dtype=None, workspace=None,
            stream=None) -> torch.Tensor:
    """act(x @ W^T + bias) with 4-bit weights W[n, k] = (q[n, k] - z) * s, one
    scale (and zero point, 8 without ``zeros``) per group of K // scales.shape[-1]
    neighbours along k.

    x: [T, K] row-major; q: uint8 [N, K // 2], the low half of byte j holding
    k = 2 j; scales: [N, K // group] in x's dtype; zeros: uint8 of that shape.
    With ``offsets`` (int32 [experts + 1]) q, scales and zeros carry a leading
    expert dimension and rows offsets[e] .. offsets[e + 1] - 1 use expert e.
    """
    dtype = _pair(x, scales, "x and scales")
    lead = 3 if offsets is not None else 2
    if x.dim() != 2 or q.dim() != lead or scales.dim() != lead:
        raise ValueError(f"x must be 2-D, q and scales {lead}-D "
                         f"({'with' if lead == 3 else 'without'} offsets)")
    dev = _cuda(x=x, q=q, scales=scales, zeros=zeros, offsets=offsets, out=out, bias=bias,
                workspace=workspace)
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
    for name, t in (("q", q), ("scales", scales), ("zeros", zeros)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    out = _out("out", out, (T, N), out_dtype, dev, (dtype, torch.float32))
    epi, bias_ptr, stride_bias = _epilogue(epilogue, bias, groups, N)
    px, ldx = _rows("x", x)
    po, ldo = _rows("out", out)
    off = _offsets(offsets, groups) if offsets is not None else 0
    dt, odt = int(_DT[dtype]), int(_DT[out.dtype])
    need = _abi.gemm_w4_workspace_size(dt, groups, T, N, K, px, ldx, odt) if workspace is None else 0
    workspace, ws, ws_bytes = _scratch(workspace, need, dev)
    check(_abi.gemm_w4(dt, groups, T, N, K, px, ldx, q.data_ptr(), scales.data_ptr(),
                       0 if zeros is None else zeros.data_ptr(), K // n_groups, po, ldo, odt, off,
                       bias_ptr, stride_bias, int(epi), ws, ws_bytes, _stream(stream, dev)))
    return out
