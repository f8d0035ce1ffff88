"""The routing operators and the 8-bit products without a GPU: refusals before anything is
enqueued, workspace sizes, the tensor-level checks and the references' own."""
import numpy as np
import pytest
import torch

import dense_gemm_bf16_gb300 as dg
import routing_ref as ref
from dense_gemm_bf16_gb300 import DType, Epi, Status

NO_GPU = not torch.cuda.is_available()
BAD, UNSUP, SMALL = Status.ERR_INVALID_ARG, Status.ERR_UNSUPPORTED, Status.ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def lib():
    dg.build()
    return dg.lib()


def dispatch(**kw):
    a = dict(elem_bytes=2, T=10, K=8, X=64, ldx=8, scales=None, id_bytes=4, ids=64, ld_ids=2, top=2,
             groups=5, rows=64, ld_rows=8, row_scales=None, offsets=64, slots=64, workspace=None,
             workspace_bytes=0, stream=None)
    a.update(kw)
    return dg.gemm_expert_dispatch(**a)


def combine(**kw):
    a = dict(dtype=DType.BF16, T=10, K=8, top=2, rows=64, R=20, ld_rows=8, slots=64, weights=64,
             w_dtype=DType.F32, ld_weights=2, Y=64, ldy=8, y_dtype=DType.BF16, stream=None)
    a.update(kw)
    return dg.gemm_expert_combine(**a)


def grad(**kw):
    a = dict(dtype=DType.BF16, T=10, K=8, top=2, DY=64, lddy=8, slots=64, weights=64,
             w_dtype=DType.F32, ld_weights=2, rows=64, R=20, ld_rows=8, d_rows=64, ld_drows=8,
             d_weights=64, dw_dtype=DType.F32, ld_dweights=2, stream=None)
    a.update(kw)
    return dg.gemm_expert_combine_grad(**a)


def quantize(**kw):
    a = dict(dtype=DType.BF16, T=10, K=8, X=64, ldx=8, Q=64, ldq=8, scales=64, stream=None)
    a.update(kw)
    return dg.gemm_i8_quantize(**a)


def i8(**kw):
    a = dict(x_dtype=DType.I8, groups=1, T=10, N=16, K=32, X=64, ldx=32, x_scales=64, Q=64, ldq=32,
             stride_q=0, w_scales=64, stride_ws=0, C=64, ldc=16, c_dtype=DType.BF16, offsets=None,
             bias=None, stride_bias=0, epi=Epi.NONE, workspace=256, workspace_bytes=1 << 20,
             stream=None)
    a.update(kw)
    return dg.gemm_i8(**a)


BIG = (1 << 31) - 32


@pytest.mark.parametrize("kw,want", [
    (dict(elem_bytes=3), BAD), (dict(elem_bytes=8), BAD), (dict(id_bytes=2), BAD), (dict(T=-1), BAD),
    (dict(K=-1), BAD), (dict(top=-1), BAD), (dict(groups=-1), BAD), (dict(T=1 << 31), BAD),
    (dict(X=None), BAD), (dict(X=65), BAD), (dict(ldx=7), BAD), (dict(ids=None), BAD),
    (dict(ids=66), BAD), (dict(id_bytes=8, ids=68), BAD), (dict(ld_ids=1), BAD), (dict(rows=None), BAD),
    (dict(rows=65), BAD), (dict(ld_rows=7), BAD), (dict(offsets=None), BAD), (dict(offsets=66), BAD),
    (dict(slots=None), BAD), (dict(slots=66), BAD), (dict(scales=64), BAD), (dict(scales=66, row_scales=64), BAD),
    (dict(scales=64, row_scales=66), BAD), (dict(groups=4097), UNSUP), (dict(T=1 << 20, top=1 << 12), UNSUP),
    (dict(T=BIG, top=1), UNSUP), (dict(ldx=1 << 60), BAD), (dict(ld_ids=1 << 60), BAD),
    (dict(T=5000), SMALL), (dict(T=5000, workspace=128, workspace_bytes=1 << 20), BAD),
    (dict(T=5000, workspace=256, workspace_bytes=100), SMALL),
])
def test_dispatch_refusals(kw, want):
    assert dispatch(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=DType.I8), BAD), (dict(dtype=9), BAD), (dict(y_dtype=9), BAD), (dict(w_dtype=9), BAD),
    (dict(y_dtype=DType.F16), UNSUP), (dict(T=-1), BAD), (dict(R=-1), BAD), (dict(K=BIG), UNSUP),
    (dict(rows=None), BAD), (dict(rows=65), BAD), (dict(ld_rows=7), BAD), (dict(slots=None), BAD),
    (dict(slots=66), BAD), (dict(weights=66), BAD), (dict(ld_weights=1), BAD), (dict(Y=None), BAD),
    (dict(Y=65), BAD), (dict(ldy=7), BAD), (dict(Y=66, y_dtype=DType.F32), BAD), (dict(ldy=1 << 60), BAD),
    (dict(top=513, ld_weights=513), UNSUP),
])
def test_combine_refusals(kw, want):
    assert combine(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=DType.I8), BAD), (dict(w_dtype=9), BAD), (dict(dw_dtype=9), BAD), (dict(top=-1), BAD),
    (dict(R=BIG), UNSUP), (dict(DY=None), BAD), (dict(DY=65), BAD), (dict(lddy=7), BAD),
    (dict(slots=None), BAD), (dict(weights=66), BAD), (dict(ld_weights=1), BAD), (dict(rows=None), BAD),
    (dict(ld_rows=7), BAD), (dict(d_rows=None), BAD), (dict(d_rows=65), BAD), (dict(ld_drows=7), BAD),
    (dict(d_weights=66), BAD), (dict(ld_dweights=1), BAD), (dict(top=513, ld_weights=513, ld_dweights=513), UNSUP),
])
def test_combine_grad_refusals(kw, want):
    assert grad(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=DType.I8), BAD), (dict(T=-1), BAD), (dict(K=BIG, ldx=BIG, ldq=BIG), UNSUP), (dict(X=None), BAD),
    (dict(X=65), BAD), (dict(ldx=7), BAD), (dict(Q=None), BAD), (dict(ldq=7), BAD), (dict(scales=None), BAD),
    (dict(scales=66), BAD), (dict(ldx=1 << 60), BAD),
])
def test_quantize_refusals(kw, want):
    assert quantize(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x_dtype=9), BAD), (dict(groups=-1), BAD), (dict(T=-1), BAD), (dict(N=-1), BAD), (dict(K=-1), BAD),
    (dict(T=BIG), UNSUP), (dict(K=131072, ldx=131072, ldq=131072), UNSUP), (dict(X=None), BAD),
    (dict(ldx=31), BAD), (dict(x_scales=None), BAD), (dict(x_scales=66), BAD),
    (dict(x_dtype=DType.BF16), BAD), (dict(x_dtype=DType.BF16, x_scales=None, X=65), BAD),
    (dict(Q=None), BAD), (dict(ldq=31), BAD), (dict(stride_q=-16), BAD), (dict(w_scales=None), BAD),
    (dict(w_scales=66), BAD), (dict(stride_ws=-1), BAD), (dict(C=None), BAD), (dict(C=65), BAD),
    (dict(ldc=15), BAD), (dict(c_dtype=DType.I8), BAD), (dict(offsets=66), BAD), (dict(groups=2), BAD),
    (dict(epi=16), BAD), (dict(epi=Epi.BIAS), BAD), (dict(epi=Epi.ROW_BIAS, bias=64), UNSUP),
    (dict(workspace=None), SMALL), (dict(workspace_bytes=255), SMALL), (dict(workspace=128), BAD),
    (dict(ldq=1 << 60), BAD), (dict(groups=1 << 17, T=1 << 17, N=1 << 30, K=16, ldc=1 << 30, offsets=64), UNSUP),
])
def test_i8_refusals(kw, want):
    assert i8(**kw) == want


def test_other_products_refuse_8_bit_operands():
    assert dg.gemm_grouped(DType.I8, 1, 4, 16, 16, 64, 16, 64, 16, 0, 0, 64, 16, DType.F32, 64, 1.0, 0.0,
                           None, 0, 0, None, 0, None) == BAD
    assert dg.gemm_batched(DType.I8, 1, 4, 4, 4, 16, 4, 0, 0, 16, 4, 0, 0, 16, 4, 0, 0, DType.F32, 1.0,
                           0.0, None, 0, 0, None, 0, None) == BAD
    assert dg.gemm_w4(DType.I8, 1, 2, 16, 64, 64, 64, 64, 64, None, 32, 64, 16, DType.BF16, None, None,
                      0, 0, None, 0, None) == BAD


def test_workspace_sizes():
    assert dg.gemm_expert_dispatch_workspace_size(2048, 2, 64) == 0
    assert dg.gemm_expert_dispatch_workspace_size(2049, 2, 64) == 304 * 64 * 4
    assert dg.gemm_expert_dispatch_workspace_size(100, 100, 3) == 100 * 3 * 4
    assert dg.gemm_expert_dispatch_workspace_size(100, 100, 5000) == 0
    size = dg.gemm_i8_workspace_size
    assert size(DType.I8, 1, 10, 16, 100, 256, 112, 0) == 2560                # 10 x 128 fp16
    assert size(DType.BF16, 1, 10, 16, 100, 256, 112, 0) == 2560 + 256        # and 10 scales
    assert size(DType.I8, 3, 10, 16, 100, 256, 100, 1600) == 2560 + 5376      # 48 rows of 112 bytes
    assert size(DType.I8, 3, 10, 16, 100, 264, 112, 1792) == 2560 + 5376      # an odd base
    assert size(DType.I8, 3, 10, 16, 100, 256, 100, 0) == 2560 + 1792         # one matrix for all
    assert size(DType.I8, 3, 10, 16, 100, 256, 336, 112) == 2560 + 5376       # matrices side by side
    assert size(DType.I8, 1, 0, 16, 100, 256, 112, 0) == 0
    assert size(DType.I8, 1, 10, 16, 1 << 20, 256, 1 << 20, 0) == 0


@pytest.mark.skipif(not NO_GPU, reason="the calls would run")
def test_valid_calls_get_as_far_as_the_device():
    for call in (dispatch, combine, grad, quantize, i8):
        assert call() == Status.ERR_NO_DEVICE
    assert dispatch(T=0, ids=None, X=None, rows=None, slots=None) == Status.ERR_NO_DEVICE  # (writes offsets)
    assert combine(T=0) == grad(top=0) == quantize(T=0) == i8(N=0) == Status.OK
    assert combine(weights=None) == combine(top=0, slots=None, rows=None) == Status.ERR_NO_DEVICE
    assert grad(d_weights=None, rows=None) == i8(K=0, X=None, Q=None) == Status.ERR_NO_DEVICE


def test_tensor_level_refusals():
    x, ids = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int64)
    slots = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dg.expert_dispatch(x, ids, 3)
    with pytest.raises(TypeError):
        dg.expert_dispatch(x.double(), ids, 3)
    with pytest.raises(ValueError, match="shape"):
        dg.expert_dispatch(x, ids[:3], 3)
    with pytest.raises(ValueError, match="negative"):
        dg.expert_dispatch(x, ids, -1)
    with pytest.raises(ValueError, match="CUDA"):
        dg.expert_combine(x, slots)
    with pytest.raises(TypeError):
        dg.expert_combine(x.to(torch.int8), slots)
    with pytest.raises(ValueError, match="shape"):
        dg.expert_combine(x, slots[0])
    with pytest.raises(ValueError, match="CUDA"):
        dg.expert_combine_grad(x, slots)
    with pytest.raises(TypeError):
        dg.i8_quantize(ids)
    with pytest.raises(ValueError, match="two dimensions"):
        dg.i8_quantize(x[0])
    with pytest.raises(ValueError, match="CUDA"):
        dg.i8_quantize(x)
    q, s = torch.zeros((6, 8), dtype=torch.int8), torch.ones(6)
    with pytest.raises(ValueError, match="CUDA"):
        dg.i8_gemm(x, q, s)
    with pytest.raises(ValueError, match="x_scales"):
        dg.i8_gemm(x, q, s, x_scales=torch.ones(4))
    with pytest.raises(ValueError, match="x_scales"):
        dg.i8_gemm(x.to(torch.int8), q, s)
    with pytest.raises(TypeError):
        dg.i8_gemm(x, q.to(torch.uint8), s)
    with pytest.raises(TypeError):
        dg.i8_gemm(x, q, s.half())
    with pytest.raises(ValueError, match="shape"):
        dg.i8_gemm(x, q[:, :7], s)
    with pytest.raises(ValueError, match="offsets"):
        dg.i8_gemm(x, q[None], s[None])


def test_tensors_of_another_device_than_the_current_one_are_refused(monkeypatch):
    from torch._subclasses.fake_tensor import FakeTensorMode

    from dense_gemm_bf16_gb300 import experts
    called = []
    monkeypatch.setattr(experts, "_fn", lambda name: called.append(name))
    monkeypatch.setattr(experts, "_current_device", lambda: 0, raising=False)
    with FakeTensorMode():
        x = torch.empty((4, 8), dtype=torch.bfloat16, device="cuda:1")
        ids = torch.empty((4, 2), dtype=torch.int32, device="cuda:1")
        q, s = torch.empty((6, 8), dtype=torch.int8, device="cuda:1"), torch.empty(6, device="cuda:1")
        for call in (lambda: dg.expert_dispatch(x, ids, 3, stream=0),
                     lambda: dg.expert_combine(x, ids, stream=0),
                     lambda: dg.expert_combine_grad(x, ids, stream=0),
                     lambda: dg.i8_quantize(x, stream=0), lambda: dg.i8_gemm(x, q, s, stream=0)):
            with pytest.raises(ValueError, match="current"):
                call()
    assert called == []


def test_references():
    """By hand: places, sums, gradients, integers at ties, exact products."""
    offsets, slots = ref.places([[2, 0], [0, -1], [7, 2]], 3)
    assert offsets.tolist() == [0, 2, 2, 4] and slots.tolist() == [[2, 0], [1, -1], [-1, 3]]
    rows = torch.arange(8.0).reshape(4, 2)
    y, size = ref.combine(rows, slots, torch.tensor([[1.0, -2.0], [3.0, 9.0], [9.0, 0.5]]))
    assert y.tolist() == [[4.0, 3.0], [6.0, 9.0], [3.0, 3.5]] and size[0].tolist() == [4.0, 7.0]
    d_rows, d_w, _ = ref.combine_grad(torch.ones(3, 2), slots, None, rows, torch.zeros(4, 2))
    assert d_rows.tolist() == [[1.0, 1.0]] * 4 and d_w.tolist() == [[9.0, 1.0], [5.0, 0.0], [0.0, 13.0]]
    q, s = ref.quantize(torch.tensor([[127.0, 0.5, 1.5, -2.5], [0.0, 0.0, 0.0, 0.0]]))
    assert q.tolist() == [[127, 0, 2, -2], [0, 0, 0, 0]] and s.tolist() == [1.0, 0.0]
    sums = ref.integer_sums([[1, 2], [3, 4]], [[[1, 1]], [[10, 0]]], [0, 1, 2])
    assert sums.tolist() == [[3], [30]]
    bits = ref.i8_bits(sums, [2.0, 0.5], [[4.0], [1.0]], torch.float32, [0, 1, 2])
    assert bits.tolist() == [[24.0], [15.0]]


def test_rows_at_one_distance_over_any_leading_dimensions():
    """i8_quantize takes rows that lie at one distance, whichever leading dimensions are one."""
    from dense_gemm_bf16_gb300 import experts
    for lead in ((5,), (4, 1), (1, 4), (4, 1, 1), (1, 4, 1), (4, 3, 1), (2, 1, 3), (4, 1, 3, 1), (1, 1, 1)):
        for pad in (0, 3):
            t = torch.empty(lead + (8 + pad,))[..., :8]
            assert experts._row_pitch("x", t) == 8 + pad or t[..., 0].numel() == 1, (lead, pad)
    for t in (torch.empty((4, 2, 8))[::2, :, :5], torch.empty((4, 1, 3, 8))[:, :, :2],
              torch.empty((3, 8)).expand(2, 3, 8), torch.empty((1, 1, 8)).expand(4, 1, 8), torch.empty((4, 1, 1, 8))[..., ::2]):
        with pytest.raises(ValueError):
            experts._row_pitch("x", t)
