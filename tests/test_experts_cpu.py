"""The expert-layer entry points without a GPU: refusals before anything is
enqueued, workspace sizes, and the tensor-level checks."""
import numpy as np
import pytest
import torch

import dense_gemm_bf16_gb300 as dg
import experts_ref as ref
from dense_gemm_bf16_gb300 import DType, Epi, Status

NO_GPU = not torch.cuda.is_available()
BAD, UNSUP, NODEV = Status.ERR_INVALID_ARG, Status.ERR_UNSUPPORTED, Status.ERR_NO_DEVICE


@pytest.fixture(scope="module", autouse=True)
def lib():
    dg.build()
    return dg.lib()


def grouped(**kw):
    a = dict(ab_dtype=DType.BF16, groups=3, T=10, N=16, K=8, A=64, lda=8, B=64, ldb=16, lb=0,
             stride_b=128, C=64, ldc=16, c_dtype=DType.BF16, offsets=64, alpha=1.0, beta=0.0,
             bias=None, stride_bias=0, epi=Epi.NONE, workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    return dg.gemm_grouped(**a)


def wgrad(**kw):
    a = dict(ab_dtype=DType.BF16, groups=3, T=10, M=8, N=16, A=64, lda=8, D=64, ldd=16, C=64,
             ldc=16, stride_c=128, c_dtype=DType.F32, offsets=64, alpha=1.0, beta=0.0,
             workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    return dg.gemm_grouped_wgrad(**a)


def ns(**kw):
    a = dict(g_dtype=DType.F32, batch=1, M=8, N=16, G=64, ldg=16, stride_g=0, O=64, ldo=16,
             stride_o=0, o_dtype=DType.BF16, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7,
             workspace=256, workspace_bytes=1 << 20, stream=None)
    a.update(kw)
    return dg.gemm_newton_schulz(**a)


def w4(**kw):
    a = dict(ab_dtype=DType.BF16, groups=1, T=2, N=16, K=64, A=64, lda=64, Q=64, scales=64,
             zeros=None, group=32, C=64, ldc=16, c_dtype=DType.BF16, offsets=None, bias=None,
             stride_bias=0, epi=Epi.NONE, workspace=None, workspace_bytes=0, stream=None)
    a.update(kw)
    return dg.gemm_w4(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(groups=-1), BAD), (dict(T=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD),
    (dict(T=1 << 31), BAD), (dict(lda=7), BAD), (dict(ldb=15), BAD), (dict(ldb=7, lb=1), BAD),
    (dict(ldc=15), BAD), (dict(lb=2), BAD), (dict(stride_b=-8), BAD), (dict(stride_b=100), BAD),
    (dict(A=None), BAD), (dict(B=None), BAD), (dict(C=None), BAD), (dict(offsets=None), BAD),
    (dict(offsets=66), BAD), (dict(A=65), BAD), (dict(C=65), BAD),
    (dict(c_dtype=DType.F32, C=66), BAD), (dict(epi=16), BAD), (dict(epi=Epi.BIAS), BAD),
    (dict(epi=Epi.BIAS, bias=66), BAD), (dict(epi=Epi.BIAS, bias=64, stride_bias=-1), BAD),
    (dict(epi=Epi.ROW_BIAS, bias=64), UNSUP), (dict(ab_dtype=5), BAD), (dict(c_dtype=5), BAD),
    (dict(ab_dtype=DType.F32), UNSUP), (dict(c_dtype=DType.F16), UNSUP),
    (dict(lda=1 << 60), BAD), (dict(stride_b=1 << 50), BAD),
])
def test_grouped_refusals(kw, want):
    assert grouped(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(groups=-1), BAD), (dict(T=-1), BAD), (dict(M=-1), BAD), (dict(N=1 << 31), BAD),
    (dict(lda=7), BAD), (dict(ldd=15), BAD), (dict(ldc=15), BAD), (dict(stride_c=127), BAD),
    (dict(A=None), BAD), (dict(D=65), BAD), (dict(C=66), BAD), (dict(offsets=None), BAD),
    (dict(ab_dtype=DType.F32), UNSUP), (dict(c_dtype=DType.F16), UNSUP), (dict(c_dtype=9), BAD),
])
def test_wgrad_refusals(kw, want):
    assert wgrad(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(batch=-1), BAD), (dict(M=-1), BAD), (dict(ldg=15), BAD), (dict(ldo=15), BAD),
    (dict(G=None), BAD), (dict(G=66), BAD), (dict(O=65), BAD), (dict(steps=0), BAD),
    (dict(steps=65), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(g_dtype=7), BAD), (dict(o_dtype=DType.F32), UNSUP), (dict(batch=2, stride_o=127), BAD),
    (dict(workspace=None), Status.ERR_WORKSPACE), (dict(workspace_bytes=16), Status.ERR_WORKSPACE),
    (dict(workspace=128), BAD),
])
def test_newton_schulz_refusals(kw, want):
    assert ns(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), BAD), (dict(groups=2), BAD), (dict(group=16), BAD), (dict(group=256), BAD),
    (dict(K=80, lda=80), BAD), (dict(lda=63), BAD), (dict(ldc=15), BAD), (dict(A=None), BAD),
    (dict(Q=None), BAD), (dict(Q=72), BAD), (dict(scales=None), BAD), (dict(scales=65), BAD),
    (dict(C=None), BAD), (dict(offsets=62), BAD), (dict(ab_dtype=DType.F32), UNSUP),
    (dict(c_dtype=DType.F16), UNSUP), (dict(epi=Epi.ROW_BIAS, bias=64), UNSUP),
    (dict(epi=Epi.BIAS), BAD), (dict(T=100), Status.ERR_WORKSPACE),
    (dict(lda=65), Status.ERR_WORKSPACE),
])
def test_w4_refusals(kw, want):
    assert w4(**kw) == want


@pytest.mark.parametrize("call,dims", [
    (grouped, dict(groups="stride_b", T="", N="ldb ldc", K="lda")),
    (wgrad, dict(groups="stride_c", T="", M="lda", N="ldd ldc")),
    (ns, dict(batch="", M="", N="ldg ldo")),
    (w4, dict(groups="", T="", N="ldc", K="lda")),
])
def test_extents_that_would_wrap_in_32_bits_are_refused(call, dims):
    """The kernels step past an extent by up to 2048 and round it up to a tile."""
    big = (1 << 31) - 32                     # (a multiple of the 4-bit weights' group)
    for dim, pitches in dims.items():
        kw = {p: big if p[0] == "l" else 0 for p in pitches.split()}
        if dim == "N" and call is grouped:
            kw["stride_b"] = 0
        assert call(**{dim: big, **kw}) == UNSUP, dim


WIDE = (1 << 31) - 4096


@pytest.mark.parametrize("kw", [
    # more than 2^31 tiles of at least 64 outputs each, with an operand to be copied first
    dict(call=grouped, groups=64, T=64, N=WIDE, K=1, lda=1, ldb=WIDE, stride_b=0, ldc=WIDE),
    dict(call=grouped, groups=1 << 17, T=1 << 17, N=1 << 30, K=1, lda=1, ldb=1 << 30, stride_b=0,
         ldc=1 << 30),
    dict(call=wgrad, groups=1 << 30, T=1, M=129, N=129, lda=129, ldd=129, ldc=129,
         stride_c=129 * 129),
    dict(call=w4, groups=64, T=64, N=WIDE, K=32, lda=33, ldc=WIDE, offsets=64),
    dict(call=w4, groups=1, T=1 << 28, N=1 << 20, K=32, lda=32, ldc=1 << 20),
])
def test_more_tiles_than_32_bits_are_refused_before_anything_else(kw):
    """Before a device is looked for, so before a copy or a pass over the weights is
    enqueued."""
    kw = dict(kw, workspace=256, workspace_bytes=1 << 50)
    assert kw.pop("call")(**kw) == UNSUP


def test_empty_calls_are_noops():
    assert grouped(T=0, A=None, C=None, offsets=None) == 0
    assert grouped(groups=0, offsets=None) == 0 and grouped(N=0, C=None) == 0
    assert wgrad(M=0, A=None, C=None) == 0 and wgrad(groups=0, offsets=None) == 0
    assert ns(batch=0, G=None) == 0 and ns(N=0, O=None) == 0
    assert w4(T=0, A=None) == 0 and w4(N=0, Q=None) == 0


@pytest.mark.skipif(not NO_GPU, reason="host has a GPU")
def test_valid_calls_report_no_device():
    assert grouped() == NODEV and wgrad() == NODEV and ns() == NODEV and w4() == NODEV


def test_workspace_sizes():
    # operands in place need none; copies are padded to 8 elements a row and 256 bytes
    assert dg.gemm_grouped_workspace_size(0, 3, 10, 16, 8, 64, 8, 64, 16, 0, 128) == 0
    assert dg.gemm_grouped_workspace_size(0, 3, 10, 16, 8, 66, 8, 64, 16, 0, 128) == 256
    assert dg.gemm_grouped_workspace_size(0, 3, 10, 16, 8, 64, 8, 64, 17, 0, 136) == 768
    assert dg.gemm_grouped_workspace_size(0, 3, 10, 16, 8, 64, 8, 64, 17, 0, 0) == 256
    assert dg.gemm_grouped_workspace_size(2, 3, 10, 16, 8, 64, 8, 64, 16, 0, 128) == 0
    assert dg.gemm_grouped_wgrad_workspace_size(0, 3, 10, 9, 16, 64, 9, 64, 16) == 512
    assert dg.gemm_newton_schulz_workspace_size(0, 8, 8) == 0
    assert dg.gemm_newton_schulz_workspace_size(-1, 8, 8) == 0
    # two states of 9 x 24, two symmetric matrices of 9 x 16, partial sums, a counter
    assert dg.gemm_newton_schulz_workspace_size(1, 9, 20) == 2 * 512 + 2 * 512 + 256 + 256
    assert dg.gemm_w4_workspace_size(0, 1, 64, 16, 64, 64, 64, 0) == 0
    assert dg.gemm_w4_workspace_size(0, 1, 65, 16, 64, 64, 64, 0) == 2048
    assert dg.gemm_w4_workspace_size(0, 1, 65, 16, 64, 64, 64, 2) == 0
    assert dg.gemm_w4_workspace_size(0, 1, 2, 16, 64, 64, 65, 0) == 256


def test_exact_4_bit_products_need_no_weights_in_the_workspace():
    opt = dg.Option.W4_EXACT
    assert dg.gemm_get_option(opt) == 0
    assert dg.gemm_set_option(opt, 2) == BAD and dg.gemm_set_option(opt, -1) == BAD
    assert dg.gemm_set_option(opt, 1) == 0 and dg.gemm_get_option(opt) == 1
    try:
        assert dg.gemm_w4_workspace_size(0, 1, 300, 16, 64, 64, 64, 0) == 0
        assert dg.gemm_w4_workspace_size(0, 3, 300, 16, 64, 64, 65, 0) == \
            dg.gemm_w4_workspace_size(0, 3, 300, 16, 64, 64, 65, 2) > 0
    finally:
        assert dg.gemm_set_option(opt, 0) == 0
    assert dg.gemm_w4_workspace_size(0, 1, 300, 16, 64, 64, 64, 0) == 2048


def test_matrices_side_by_side_are_no_overlap():
    """Column blocks of one wide matrix stay clear of each other; blocks that are not as wide
    as their stride says do not."""
    ok = NODEV if NO_GPU else None
    assert dg.gemm_grouped_workspace_size(0, 3, 10, 16, 8, 64, 8, 64, 48, 0, 16) == 512 + 256
    assert grouped(ldb=40, stride_b=16) == BAD and grouped(ldb=48, stride_b=8) == BAD
    assert wgrad(ldc=40, stride_c=16) == BAD and wgrad(ldc=48, stride_c=8) == BAD
    assert ns(batch=3, stride_g=16, ldg=48, ldo=40, stride_o=16) == BAD
    if ok is not None:
        assert grouped(ldb=48, stride_b=16, workspace=256, workspace_bytes=768) == ok
        assert wgrad(ldc=48, stride_c=16) == ok
        assert ns(batch=3, stride_g=16, ldg=48, ldo=48, stride_o=16) == ok


def test_tensor_level_refusals():
    A, B = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((2, 8, 16), dtype=torch.bfloat16)
    o = torch.tensor([0, 1, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dg.grouped_gemm(A, B, o)
    with pytest.raises(TypeError):
        dg.grouped_gemm(A.float(), B.float(), o)
    with pytest.raises(TypeError):
        dg.grouped_gemm(A, B.half(), o)
    with pytest.raises(ValueError, match="shape"):
        dg.grouped_gemm(A[:, :7], B, o)
    with pytest.raises(ValueError, match="shape"):
        dg.grouped_gemm_wgrad(A, A[:3], o)
    with pytest.raises(ValueError, match="CUDA"):
        dg.grouped_gemm_wgrad(A, A, o)
    with pytest.raises(TypeError):
        dg.newton_schulz(A.to(torch.int32))
    with pytest.raises(ValueError):
        dg.newton_schulz(A[0])
    with pytest.raises(ValueError, match="three"):
        dg.newton_schulz(A, coefficients=(1.0, 2.0))
    with pytest.raises(ValueError, match="CUDA"):
        dg.newton_schulz(A)
    q, s = torch.zeros((6, 32), dtype=torch.uint8), torch.ones((6, 2), dtype=torch.bfloat16)
    x = torch.zeros((1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dg.w4_gemm(x, q, s)
    with pytest.raises(TypeError):
        dg.w4_gemm(x.half(), q, s)
    with pytest.raises(ValueError):
        dg.w4_gemm(x, q[None], s)


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    """The library launches on the current device, so tensors of another one would be
    foreign pointers there: refused before the library is called."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    from dense_gemm_bf16_gb300 import experts
    called = []
    monkeypatch.setattr(experts, "_fn", lambda name: called.append(name))
    monkeypatch.setattr(experts, "_current_device", lambda: 0, raising=False)
    with FakeTensorMode():
        A = torch.empty((4, 64), dtype=torch.bfloat16, device="cuda:1")
        B = torch.empty((2, 64, 16), dtype=torch.bfloat16, device="cuda:1")
        o = torch.empty(3, dtype=torch.int32, device="cuda:1")
        q = torch.empty((6, 32), dtype=torch.uint8, device="cuda:1")
        s = torch.empty((6, 2), dtype=torch.bfloat16, device="cuda:1")
        for call in (lambda: dg.grouped_gemm(A, B, o, stream=0),
                     lambda: dg.grouped_gemm_wgrad(A, A, o, stream=0),
                     lambda: dg.newton_schulz(A, stream=0),
                     lambda: dg.w4_gemm(A, q, s, stream=0)):
            with pytest.raises(ValueError, match="current"):
                call()
    assert called == []


def test_references_agree_with_closed_forms():
    """The references themselves: identity weights, a transposed product, an orthogonal
    matrix's fixed scaling, and packed weights written out by hand."""
    rng = np.random.default_rng(1)
    A = ref.ints(rng, (6, 5))
    eye = torch.eye(5).expand(2, 5, 5)
    assert np.array_equal(ref.grouped(A, eye, [0, 2, 6]), ref.f64(A))
    W = ref.wgrad(A, A, [0, 6])
    assert np.array_equal(W[0], ref.f64(A).T @ ref.f64(A))
    Q, _ = np.linalg.qr(rng.standard_normal((4, 4)))
    a, b, c = 3.4445, -4.7750, 2.0315
    x = 0.5                                       # singular values of Q / ||Q||
    for _ in range(5):
        x = a * x + b * x ** 3 + c * x ** 5
    assert np.allclose(ref.newton_schulz(torch.from_numpy(Q), eps=0.0), x * Q, atol=1e-12)
    q = torch.tensor([[0x21, 0x43]], dtype=torch.uint8)
    s = torch.tensor([[2.0, 0.5]])
    z = torch.tensor([[1, 4]], dtype=torch.uint8)
    assert np.array_equal(ref.w4_weights(q, s, z), [[0.0, 2.0, -0.5, 0.0]])
    assert np.array_equal(ref.w4_weights(q, s, None), [[-14.0, -12.0, -2.5, -2.0]])
