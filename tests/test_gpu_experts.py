"""The expert-layer operators on the GPU against plain 64-bit references: exact
small-integer cases at the sizes where groups, tiles, stages and alignments end,
bounds for the others, and what has to stay untouched or unaffected."""
import numpy as np
import pytest
import torch

import dense_gemm_bf16_gb300 as dg
import experts_ref as ref
from experts_ref import ints

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda:0"


def offs(bounds):
    return torch.tensor(bounds, dtype=torch.int32, device=DEV)


def status():
    return dg.gemm_check_device_status(torch.cuda.current_stream().cuda_stream)


def bounds_of(counts, start=0):
    return [start + int(v) for v in np.concatenate(([0], np.cumsum(counts)))]


def equal(got, want, dtype):
    assert np.array_equal(got.to(torch.float64).cpu().numpy(), ref.rounded(want, dtype),
                          equal_nan=True)


# ---------------------------------------------------------------- grouped products

GROUPS = {
    "one_row": [1],
    "single_tokens": [1, 0, 1, 1, 0, 0, 1],
    "few": [3, 0, 31, 32, 33, 1],
    "middle": [0, 100, 129, 64, 127, 128, 0],
    "large": [255, 256, 257, 0, 513, 40],
    "many_groups": [(7 * i) % 5 for i in range(100)],
    "empty": [0, 0, 0],
}


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("case", sorted(GROUPS))
def test_grouped_exact(case, layout, dtype, out):
    rng = np.random.default_rng(sorted(GROUPS).index(case) * 8 + (layout == "row") * 4)
    counts = GROUPS[case]
    E, (K, N) = len(counts), (200, 264) if layout == "row" else (320, 136)
    lead, trail = 2, 3                      # rows of no group, before and after
    b = bounds_of(counts, lead)
    T = b[-1] + trail
    A = ints(rng, (T, K), dtype=dtype)
    B = ints(rng, (E, K, N) if layout == "row" else (E, N, K), dtype=dtype)
    B = B if layout == "row" else B.transpose(1, 2)
    C = torch.full((T, N), float("nan"), dtype=out, device=DEV)
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), C)
    assert got is C
    equal(got, ref.grouped(A, B, b), out)
    assert status() == 0


@pytest.mark.parametrize("K,N", [(1, 1), (7, 9), (8, 8), (63, 65), (64, 128), (65, 129),
                                 (127, 130), (128, 257), (129, 31), (1000, 24)])
@pytest.mark.parametrize("layout", ["row", "col"])
def test_grouped_odd_sizes(K, N, layout):
    """Operands that TMA cannot address are copied; outputs end anywhere."""
    rng = np.random.default_rng(K * 1000 + N)
    counts = [5, 0, 140, 17]
    b = bounds_of(counts)
    A = ints(rng, (b[-1], K))
    B = ints(rng, (4, K, N) if layout == "row" else (4, N, K))
    B = B if layout == "row" else B.transpose(1, 2)
    for out in (BF, F32):
        equal(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=out),
              ref.grouped(A, B, b), out)


def test_grouped_padded_strided_and_broadcast_operands():
    rng = np.random.default_rng(5)
    b = bounds_of([30, 90, 0, 7])
    T, K, N = b[-1], 96, 80
    A = ints(rng, (T, K + 9)).to(DEV)[:, 4:4 + K]            # odd pitch and base
    W = ints(rng, (K, N)).to(DEV)
    B = W.expand(4, K, N)                                    # one matrix for all groups
    C = torch.full((T, N + 5), 3.0, dtype=F32, device=DEV)
    dg.grouped_gemm(A, B, offs(b), C[:, 2:2 + N])
    equal(C[:, 2:2 + N], ref.grouped(A, B, b), F32)
    assert bool((C[:, :2] == 3).all()) and bool((C[:, 2 + N:] == 3).all())
    B2 = ints(rng, (4, K, N + 3)).to(DEV)[:, :, 1:1 + N]     # odd leading dimension
    equal(dg.grouped_gemm(A, B2, offs(b), out_dtype=F32), ref.grouped(A, B2, b), F32)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("per_group", [False, True])
@pytest.mark.parametrize("counts", [[2, 1, 0, 5], [100, 3, 0, 300]])
def test_grouped_alpha_beta_bias_relu(counts, per_group, out):
    rng = np.random.default_rng(11)
    b = bounds_of(counts, 1)
    T, K, N, E = b[-1] + 1, 72, 104, len(counts)
    A, B = ints(rng, (T, K)), ints(rng, (E, K, N))
    bias = ints(rng, (E, N) if per_group else (N,), dtype=F32)
    C0 = ints(rng, (T, N), dtype=out)
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), C0.to(DEV), alpha=2.0, beta=-0.5,
                          bias=bias.to(DEV), epilogue="bias_relu")
    equal(got, ref.grouped(A, B, b, C0, 2.0, -0.5, bias, "bias_relu"), out)


def test_grouped_alpha_zero_and_empty_contraction_read_no_operand():
    rng = np.random.default_rng(12)
    b = bounds_of([3, 0, 40])
    T, N = b[-1], 40
    C0 = ints(rng, (T, N), dtype=F32)
    bias = ints(rng, (3, N), dtype=F32)
    nan = torch.full((T, 64), float("nan"), dtype=BF, device=DEV)
    B = torch.full((3, 64, N), float("nan"), dtype=BF, device=DEV)
    want = ref.grouped(torch.zeros(T, 1), torch.zeros(3, 1, N), b, C0, 1.0, 0.5, bias, "bias")
    got = dg.grouped_gemm(nan, B, offs(b), C0.to(DEV), alpha=0.0, beta=0.5, bias=bias.to(DEV))
    equal(got, want, F32)
    got = dg.grouped_gemm(nan[:, :0], B[:, :0], offs(b), C0.to(DEV), beta=0.5, bias=bias.to(DEV))
    equal(got, want, F32)


def test_grouped_nothing_to_do():
    A = torch.empty((0, 16), dtype=BF, device=DEV)
    B = torch.empty((3, 16, 8), dtype=BF, device=DEV)
    assert dg.grouped_gemm(A, B, offs([0, 0, 0, 0])).shape == (0, 8)
    A = torch.empty((5, 16), dtype=BF, device=DEV)
    assert dg.grouped_gemm(A, B[:, :, :0], offs([0, 1, 2, 5])).shape == (5, 0)
    C = torch.full((5, 8), 7.0, dtype=BF, device=DEV)
    dg.grouped_gemm(A, B[:0], offs([0]), C)
    assert bool((C == 7).all())


@pytest.mark.parametrize("epilogue", ["gelu_tanh", "bias_gelu_tanh", "gelu_erf", "bias_gelu_erf"])
@pytest.mark.parametrize("counts", [[4, 1, 9], [200, 0, 70]])
def test_grouped_gelu(counts, epilogue):
    """fp32 output: the sum of K products of exact inputs is within K u S of the exact
    one (u = 2^-23, S the sum of magnitudes), GELU's slope is below 1.13, and its
    own evaluation is within 2^-20 of the value and its argument."""
    rng = np.random.default_rng(13)
    b = bounds_of(counts)
    K, N, E = 160, 72, 3
    A = torch.from_numpy(rng.standard_normal((b[-1], K)).astype(np.float32)).to(BF)
    B = torch.from_numpy(rng.standard_normal((E, K, N)).astype(np.float32) / 12).to(BF)
    bias = torch.from_numpy(rng.standard_normal((E, N)).astype(np.float32))
    use = bias if epilogue.startswith("bias") else None
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=F32, epilogue=epilogue,
                          bias=None if use is None else use.to(DEV))
    want = ref.grouped(A, B, b, bias=use, epilogue=epilogue)
    size = np.abs(ref.grouped(A.abs(), B.abs(), b, bias=None if use is None else use.abs()))
    assert np.all(np.abs(ref.f64(got) - want) <= 1.13 * K * 2.0 ** -23 * size + 2.0 ** -20 * (
        size + np.abs(want)))


def test_grouped_rows_do_not_mix():
    """NaN and infinite rows stay in their rows; NaN weights in their group."""
    rng = np.random.default_rng(14)
    b = bounds_of([20, 45, 3])
    A, B = ints(rng, (b[-1], 136)), ints(rng, (3, 136, 72))
    want = ref.grouped(A, B, b)
    A2, B2 = A.clone(), B.clone()
    A2[7], A2[30], B2[2] = float("nan"), float("inf"), float("nan")
    got = ref.f64(dg.grouped_gemm(A2.to(DEV), B2.to(DEV), offs(b), out_dtype=F32))
    keep = [i for i in range(b[2]) if i not in (7, 30)]
    assert np.array_equal(got[keep], want[keep])
    assert np.isnan(got[7]).all() and np.isnan(got[b[2]:]).all()


def test_grouped_repeats_and_is_independent_of_other_groups():
    g = torch.Generator(device=DEV).manual_seed(3)
    A = torch.randn((700, 512), generator=g, device=DEV).to(BF)
    B = torch.randn((4, 512, 256), generator=g, device=DEV).to(BF)
    o = offs([0, 100, 400, 400, 700])
    first = dg.grouped_gemm(A, B, o, out_dtype=F32)
    for _ in range(3):
        assert torch.equal(first, dg.grouped_gemm(A, B, o, out_dtype=F32))


def test_offsets_past_32_bits_of_elements():
    """Rows whose element offsets pass 2^31 (a C of 2.2e9 elements, most of it in no
    group)."""
    rng = np.random.default_rng(15)
    T, K, N = 70000, 64, 32768
    A = torch.zeros((T, K), dtype=BF, device=DEV)
    B = ints(rng, (2, K, N)).to(DEV)
    a = ints(rng, (5, K))
    A[-6:-1] = a.to(DEV)
    C = torch.empty((T, N), dtype=BF, device=DEV)
    C[-8:].fill_(9.0)
    dg.grouped_gemm(A, B, offs([T - 6, T - 4, T - 1]), C)
    want = ref.grouped(a, B, [0, 2, 5])
    equal(C[-6:-1], want, BF)
    assert bool((C[-8:-6] == 9).all()) and bool((C[-1] == 9).all())


@pytest.mark.parametrize("bad", [[0, 5, 3, 10], [0, 5, 8, 11], [-1, 5, 8, 10], [4, 3, 2, 1]])
def test_bad_offsets_are_reported_and_touch_nothing_else(bad):
    rng = np.random.default_rng(16)
    A, B = ints(rng, (10, 40)), ints(rng, (3, 40, 24))
    C = torch.full((12, 24), 5.0, dtype=F32, device=DEV)
    dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(bad), C[1:11])
    assert status() == dg.Status.ERR_INVALID_ARG
    assert bool((C[0] == 5).all()) and bool((C[11] == 5).all())
    dg.grouped_gemm_wgrad(A.to(DEV), A.to(DEV), offs(bad))
    assert status() == dg.Status.ERR_INVALID_ARG
    q = torch.zeros((3, 24, 32), dtype=torch.uint8, device=DEV)
    s = torch.ones((3, 24, 2), dtype=BF, device=DEV)
    x = torch.ones((10, 64), dtype=BF, device=DEV)
    dg.w4_gemm(x, q, s, offsets=offs(bad))
    assert status() == dg.Status.ERR_INVALID_ARG
    equal(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs([0, 5, 8, 10]), out_dtype=F32),
          ref.grouped(A, B, [0, 5, 8, 10]), F32)
    assert status() == 0


# ---------------------------------------------------------------- weight gradient

WCOUNTS = {
    "tails": [1, 15, 16, 17, 31, 0, 33],
    "stages": [127, 128, 129, 0, 255, 257],
    "one_row": [1],
    "none": [0, 0],
    "many_groups": [(5 * i) % 7 for i in range(70)],
}


@pytest.mark.parametrize("dtype,out", [(BF, F32), (BF, BF), (HF, F32), (HF, HF)])
@pytest.mark.parametrize("case", sorted(WCOUNTS))
@pytest.mark.parametrize("M,N", [(72, 136), (200, 264)])
def test_wgrad_exact(case, M, N, dtype, out):
    rng = np.random.default_rng(sorted(WCOUNTS).index(case) + M)
    b = bounds_of(WCOUNTS[case], 3)
    T = b[-1] + 2
    A, D = ints(rng, (T, M), -2, 2, dtype), ints(rng, (T, N), -2, 2, dtype)
    got = dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs(b), out_dtype=out)
    equal(got, ref.wgrad(A, D, b), out)
    assert status() == 0


def test_wgrad_pairs_exact():
    """Large enough for the two-CTA tiles."""
    rng = np.random.default_rng(21)
    b = bounds_of([300, 0, 77, 130, 16, 1000])
    A, D = ints(rng, (b[-1], 1000), -2, 2), ints(rng, (b[-1], 1032), -2, 2)
    for out in (F32, BF):
        equal(dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs(b), out_dtype=out),
              ref.wgrad(A, D, b), out)


@pytest.mark.parametrize("M,N", [(1, 1), (3, 130), (65, 7), (129, 33)])
def test_wgrad_odd_sizes_and_accumulation(M, N):
    rng = np.random.default_rng(M * 100 + N)
    b = bounds_of([9, 0, 130])
    A, D = ints(rng, (b[-1], M + 3)).to(DEV)[:, 1:1 + M], ints(rng, (b[-1], N)).to(DEV)
    for out in (F32, BF):
        C0 = ints(rng, (3, M, N), dtype=out)
        got = dg.grouped_gemm_wgrad(A, D, offs(b), C0.to(DEV), alpha=0.5, beta=2.0)
        equal(got, ref.wgrad(A, D, b, C0, 0.5, 2.0), out)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_wgrad_other_groups_rows_never_enter(value):
    """Every group's neighbours hold NaN or infinities, and so do the rows of no group."""
    rng = np.random.default_rng(22)
    counts = [20, 5, 131, 3]
    b = bounds_of(counts, 4)
    T = b[-1] + 20
    A, D = ints(rng, (T, 264), -2, 2), ints(rng, (T, 520), -2, 2)
    want = ref.wgrad(A, D, b)
    for e in range(len(counts)):
        A2, D2 = torch.full_like(A, value), torch.full_like(D, value)
        A2[b[e]:b[e + 1]], D2[b[e]:b[e + 1]] = A[b[e]:b[e + 1]], D[b[e]:b[e + 1]]
        got = ref.f64(dg.grouped_gemm_wgrad(A2.to(DEV), D2.to(DEV), offs(b), out_dtype=F32))
        assert np.array_equal(got[e], want[e])


def test_wgrad_without_rows_scales_its_input():
    C0 = torch.arange(2 * 3 * 8, dtype=F32, device=DEV).reshape(2, 3, 8)
    A, D = torch.empty((0, 3), dtype=BF, device=DEV), torch.empty((0, 8), dtype=BF, device=DEV)
    got = dg.grouped_gemm_wgrad(A, D, offs([0, 0, 0]), C0.clone(), beta=0.5)
    assert torch.equal(got, 0.5 * C0)
    assert bool((dg.grouped_gemm_wgrad(A, D, offs([0, 0, 0])) == 0).all())


def test_gradients_against_differences():
    """L = sum(D * Y) is linear in every weight and every input, so its central
    differences are exact on small integers: they have to equal the gradients
    entry for entry."""
    rng = np.random.default_rng(23)
    b = bounds_of([5, 0, 18])
    T, K, N = b[-1], 24, 40
    X, W, D = ints(rng, (T, K)), ints(rng, (3, K, N)), ints(rng, (T, N))
    o, Xd, Wd, Dd = offs(b), X.to(DEV), W.to(DEV), D.to(DEV)

    def loss(x, w):
        y = dg.grouped_gemm(x, w, o, out_dtype=F32)
        return float((y.double() * Dd.double()).sum())

    dW = dg.grouped_gemm_wgrad(Xd, Dd, o, out_dtype=F32)
    dX = dg.grouped_gemm(Dd, Wd.transpose(1, 2), o, out_dtype=F32)
    for _ in range(12):
        e, k, n = (int(rng.integers(s)) for s in W.shape)
        up, down = Wd.clone(), Wd.clone()
        up[e, k, n] += 1
        down[e, k, n] -= 1
        assert (loss(Xd, up) - loss(Xd, down)) / 2 == float(dW[e, k, n])
        t, k = int(rng.integers(T)), int(rng.integers(K))
        up, down = Xd.clone(), Xd.clone()
        up[t, k] += 1
        down[t, k] -= 1
        assert (loss(up, Wd) - loss(down, Wd)) / 2 == float(dX[t, k])


# ---------------------------------------------------------------- orthogonalised update

def ns_bound(steps):
    """Relative error in the Frobenius norm: X, S and the polynomial are rounded to
    fp16 (half an ulp: 2^-12 of a value at most twice its typical size) in each step,
    and a later step grows an error by at most 1.7, the largest slope of
    3.4445 x - 4.775 x^3 + 2.0315 x^5 where singular values settle."""
    return 3 * steps * 2.0 ** -12 * 1.7 ** steps


@pytest.mark.parametrize("gdt,odt", [(F32, BF), (BF, BF), (HF, HF), (F32, HF)])
@pytest.mark.parametrize("shape", [(1, 1), (1, 40), (33, 1), (5, 7), (64, 64), (128, 128),
                                   (129, 257), (300, 200), (3, 100, 130), (5, 200, 72)])
def test_newton_schulz(shape, gdt, odt):
    rng = np.random.default_rng(sum(shape))
    G = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(gdt)
    got = dg.newton_schulz(G.to(DEV), out_dtype=odt)
    want = ref.newton_schulz(G)
    err = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
    assert got.dtype == odt and got.shape == G.shape
    assert err <= ns_bound(5) + (2.0 ** -9 if odt == BF else 2.0 ** -12), err
    assert status() == 0


def test_newton_schulz_pairs_and_steps():
    rng = np.random.default_rng(31)
    G = torch.from_numpy(rng.standard_normal((10, 600, 520)).astype(np.float32))
    for steps in (1, 2, 4):
        got = dg.newton_schulz(G.to(DEV), steps=steps, out_dtype=HF)
        want = ref.newton_schulz(G, steps)
        err = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
        assert err <= ns_bound(steps) + 2.0 ** -12, (steps, err)


@pytest.mark.parametrize("coefficients,steps", [((1.5, -0.5, 0.0), 6), ((1.875, -1.25, 0.375), 4),
                                                ((2.0, -1.5, 0.3), 3), ((1.0, 0.0, -0.25), 2),
                                                ((0.5, 0.0, 0.0), 2)])
@pytest.mark.parametrize("shape", [(200, 136), (9, 130, 300)])
def test_newton_schulz_other_coefficients(shape, coefficients, steps):
    """Polynomials whose square is completed, and such (c zero or small) whose is not."""
    rng = np.random.default_rng(36)
    G = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    got = dg.newton_schulz(G.to(DEV), steps=steps, coefficients=coefficients, out_dtype=HF)
    want = ref.newton_schulz(G, steps, coefficients)
    err = np.linalg.norm(ref.f64(got) - want) / np.linalg.norm(want)
    assert err <= ns_bound(steps) + 2.0 ** -12, err


def test_newton_schulz_matrices_of_a_batch_do_not_depend_on_each_other():
    """Each matrix of a batch comes out as it does alone (which may take another tile
    shape, so to the output's rounding), and repeats bit for bit."""
    G = torch.randn((37, 256, 384), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    for _ in range(5):
        got = dg.newton_schulz(G)
        for i in (0, 17, 36):
            alone = dg.newton_schulz(G[i]).float()
            assert float((got[i].float() - alone).norm()) <= 2.0 ** -8 * float(alone.norm())
        assert torch.equal(got, dg.newton_schulz(G))


def test_newton_schulz_singular_values():
    rng = np.random.default_rng(32)
    G = torch.from_numpy(rng.standard_normal((96, 384)).astype(np.float32))
    s = np.linalg.svd(ref.f64(dg.newton_schulz(G.to(DEV))), compute_uv=False)
    assert s.min() > 0.6 and s.max() < 1.3


def test_newton_schulz_views_in_place_and_transposed():
    rng = np.random.default_rng(33)
    base = torch.from_numpy(rng.standard_normal((4, 70, 101)).astype(np.float32)).to(DEV)
    G = base[:, 3:63, 1:90]                                  # odd pitch and base
    want = ref.newton_schulz(G)
    out = torch.full((4, 60, 97), 4.0, dtype=BF, device=DEV)
    dg.newton_schulz(G, out[:, :, 2:91])
    assert np.linalg.norm(ref.f64(out[:, :, 2:91]) - want) <= (ns_bound(5) + 2.0 ** -9) * \
        np.linalg.norm(want)
    assert bool((out[:, :, :2] == 4).all()) and bool((out[:, :, 91:] == 4).all())
    H = torch.from_numpy(rng.standard_normal((60, 89)).astype(np.float32)).to(BF).to(DEV)
    want = ref.newton_schulz(H)
    dg.newton_schulz(H, H)
    assert np.linalg.norm(ref.f64(H) - want) <= (ns_bound(5) + 2.0 ** -9) * np.linalg.norm(want)


@pytest.mark.parametrize("scale", [1e-41, 1e-37, 1e-25, 1e-3, 1e18, 1e25, 3e38])
def test_newton_schulz_norm_does_not_leave_fp32(scale):
    """Squares of these entries, their sum, the norm or its inverse do; eps = 0 leaves
    the direction alone."""
    rng = np.random.default_rng(34)
    U = rng.uniform(0.2, 1.0, (40, 64)) * rng.choice([-1, 1], (40, 64))
    G = torch.from_numpy((U * scale).astype(np.float32))
    got = ref.f64(dg.newton_schulz(G.to(DEV), eps=0.0))
    want = ref.newton_schulz(torch.from_numpy(U))
    assert np.linalg.norm(got - want) <= (ns_bound(5) + 2.0 ** -8) * np.linalg.norm(want)


def test_newton_schulz_zero_and_nan_matrices_stay_apart():
    rng = np.random.default_rng(35)
    G = torch.from_numpy(rng.standard_normal((3, 48, 56)).astype(np.float32))
    want = ref.newton_schulz(G)[1]
    G[0] = 0
    G[2, 5, 5] = float("nan")
    got = ref.f64(dg.newton_schulz(G.to(DEV)))
    assert np.all(got[0] == 0) and np.isnan(got[2]).all()
    assert np.linalg.norm(got[1] - want) <= (ns_bound(5) + 2.0 ** -9) * np.linalg.norm(want)


def test_newton_schulz_repeats():
    G = torch.randn((2, 640, 520), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    first = dg.newton_schulz(G)
    for _ in range(3):
        assert torch.equal(first, dg.newton_schulz(G))


# ---------------------------------------------------------------- 4-bit weights

def w4_case(rng, T, N, K, group, zeros, dtype=BF, experts=0):
    lead = (experts,) if experts else ()
    x = ints(rng, (T, K), -3, 3, dtype)
    q = torch.from_numpy(rng.integers(0, 256, lead + (N, K // 2)).astype(np.uint8))
    s = torch.from_numpy(2.0 ** rng.integers(-2, 2, lead + (N, K // group)).astype(np.float32)).to(dtype)
    z = torch.from_numpy(rng.integers(0, 16, lead + (N, K // group)).astype(np.uint8)) if zeros else None
    return x, q, s, z


def w4_run(x, q, s, z, **kw):
    return dg.w4_gemm(x.to(DEV), q.to(DEV), s.to(DEV), zeros=None if z is None else z.to(DEV), **kw)


@pytest.mark.parametrize("group,K", [(32, 32), (32, 160), (32, 1056), (64, 64), (64, 576),
                                     (128, 128), (128, 1152), (128, 2048), (32, 2048), (64, 4096)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("T", [1, 8, 9, 33])
def test_w4_exact(T, group, K, zeros):
    rng = np.random.default_rng(T * 7 + K + group)
    N = [1, 63, 130, 200][T % 4]
    x, q, s, z = w4_case(rng, T, N, K, group, zeros, BF if T % 2 else HF)
    equal(w4_run(x, q, s, z, out_dtype=F32), ref.w4(x, q, s, z), F32)
    assert status() == 0


@pytest.mark.parametrize("T", [2, 16, 17, 32, 64, 65, 100, 300])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_w4_token_counts_and_16_bit_outputs(T, dtype):
    """From 65 rows on a 16-bit output takes the other route, through 16-bit weights
    (exact here: (q - z) s has at most 5 bits)."""
    rng = np.random.default_rng(T)
    x, q, s, z = w4_case(rng, T, 192, 512, 64, True, dtype)
    bias = ints(rng, (192,), dtype=F32)
    got = w4_run(x, q, s, z, bias=bias.to(DEV), epilogue="bias_relu")
    equal(got, ref.w4(x, q, s, z, bias=bias, epilogue="bias_relu"), dtype)


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [0, 20, 0, 7, 70], [3] * 40, [0, 0, 5]])
@pytest.mark.parametrize("out", [HF, F32])
def test_w4_experts(counts, out):
    rng = np.random.default_rng(len(counts))
    E, b = len(counts), bounds_of(counts, 2)
    T = b[-1] + 1
    x, q, s, z = w4_case(rng, T, 136, 320, 32, True, HF, E)
    bias = ints(rng, (E, 136), dtype=F32)
    res = torch.full((T, 136), float("nan"), dtype=out, device=DEV)
    w4_run(x, q, s, z, offsets=offs(b), bias=bias.to(DEV), out=res)
    equal(res, ref.w4(x, q, s, z, b, bias, "bias"), out)


def test_w4_many_rows_per_expert_take_the_16_bit_route():
    rng = np.random.default_rng(41)
    b = bounds_of([150, 0, 90])
    x, q, s, z = w4_case(rng, b[-1], 264, 256, 128, False, BF, 3)
    equal(w4_run(x, q, s, z, offsets=offs(b)), ref.w4(x, q, s, z, b), BF)


def test_w4_unaligned_rows_scales_and_zeros():
    rng = np.random.default_rng(42)
    x, q, s, z = w4_case(rng, 6, 70, 512, 32, True)
    xp = torch.zeros((6, 519), dtype=BF, device=DEV)
    xp[:, 3:515] = x.to(DEV)
    sp = torch.zeros(70 * 16 + 1, dtype=BF, device=DEV)
    zp = torch.zeros(70 * 16 + 3, dtype=torch.uint8, device=DEV)
    sp[1:], zp[3:] = s.reshape(-1).to(DEV), z.reshape(-1).to(DEV)
    res = torch.full((6, 75), 2.0, dtype=F32, device=DEV)
    dg.w4_gemm(xp[:, 3:515], q.to(DEV), sp[1:].reshape(70, 16), zeros=zp[3:].reshape(70, 16),
               out=res[:, 4:74])
    equal(res[:, 4:74], ref.w4(x, q, s, z), F32)
    assert bool((res[:, :4] == 2).all()) and bool((res[:, 74:] == 2).all())


def test_w4_rows_do_not_mix():
    rng = np.random.default_rng(43)
    for T in (5, 40, 100):
        x, q, s, z = w4_case(rng, T, 80, 256, 64, True)
        want = ref.w4(x, q, s, z)
        x2 = x.clone()
        x2[3], x2[1] = float("nan"), float("inf")
        got = ref.f64(w4_run(x2, q, s, z, out_dtype=F32))
        keep = [i for i in range(T) if i not in (1, 3)]
        assert np.array_equal(got[keep], want[keep]) and np.isnan(got[3]).all()


@pytest.mark.parametrize("group", [32, 128])
def test_w4_infinite_scale_in_a_last_partial_stage(group):
    """The row's output is infinite, and no other one changes."""
    rng = np.random.default_rng(44)
    x, q, s, z = w4_case(rng, 2, 20, 384, group, False)
    s[7, -1] = float("inf")
    x[:, -group:] = 1                        # (the last group's sum of q - 8, made positive)
    q[7, -group // 2:] = 0x99
    want = ref.w4(x, q, s, z)
    got = ref.f64(w4_run(x, q, s, z, out_dtype=F32))
    assert np.isposinf(want[:, 7]).all() and np.array_equal(got, want)


def test_w4_repeats():
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((3, 4096), generator=g, device=DEV).to(BF)
    q = torch.randint(0, 256, (512, 2048), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand((512, 32), generator=g, device=DEV).to(BF)
    first = dg.w4_gemm(x, q, s, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(first, dg.w4_gemm(x, q, s, out_dtype=F32))


# ---------------------------------------------------------------- streams, graphs, failures

def test_side_stream_and_caller_workspace():
    rng = np.random.default_rng(51)
    b = bounds_of([40, 90])
    A, B = ints(rng, (130, 131)), ints(rng, (2, 131, 70))      # both operands are copied
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Ad, Bd, o = A.to(DEV), B.to(DEV), offs(b)
        got = dg.grouped_gemm(Ad, Bd, o, out_dtype=F32)
        G = torch.randn((70, 90), device=DEV)
        ws = torch.empty(dg.gemm_newton_schulz_workspace_size(1, 70, 90), dtype=torch.uint8,
                         device=DEV)
        y = dg.newton_schulz(G, workspace=ws)
    s.synchronize()
    equal(got, ref.grouped(A, B, b), F32)
    want = ref.newton_schulz(G)
    assert np.linalg.norm(ref.f64(y) - want) <= (ns_bound(5) + 2.0 ** -9) * np.linalg.norm(want)
    with pytest.raises(dg.GemmError) as e:
        dg.newton_schulz(G, workspace=ws[:1024])
    assert e.value.status == dg.Status.ERR_WORKSPACE


def test_explicit_stream():
    """Outputs and copies of operands are allocated for the stream that is named."""
    rng = np.random.default_rng(55)
    b = bounds_of([40, 90])
    A, B, o = ints(rng, (130, 131)).to(DEV), ints(rng, (2, 131, 70)).to(DEV), offs(b)
    G = torch.randn((70, 90), device=DEV)
    x, q, s, z = (t.to(DEV) for t in w4_case(rng, 5, 70, 320, 64, True))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = dg.grouped_gemm(A, B, o, out_dtype=F32, stream=side.cuda_stream)
    w = dg.grouped_gemm_wgrad(A, A, o, out_dtype=F32, stream=side.cuda_stream)
    n = dg.newton_schulz(G, stream=side.cuda_stream)
    v = dg.w4_gemm(x, q, s, zeros=z, out_dtype=F32, stream=side.cuda_stream)
    side.synchronize()
    equal(y, ref.grouped(A, B, b), F32)
    equal(w, ref.wgrad(A, A, b), F32)
    equal(v, ref.w4(x, q, s, z), F32)
    want = ref.newton_schulz(G)
    assert np.linalg.norm(ref.f64(n) - want) <= (ns_bound(5) + 2.0 ** -9) * np.linalg.norm(want)


def test_graph_replays_read_offsets_and_inputs_anew():
    rng = np.random.default_rng(52)
    K, N, E, T = 256, 192, 3, 60
    A, B = ints(rng, (T, K)).to(DEV), ints(rng, (E, K, N)).to(DEV)
    x, q, s, z = (t.to(DEV) for t in w4_case(rng, T, N, K, 64, True, BF, E))
    G = torch.randn((96, 160), device=DEV)
    o = offs([0, 10, 30, 60])
    ws = torch.empty(dg.gemm_newton_schulz_workspace_size(1, 96, 160), dtype=torch.uint8, device=DEV)

    def calls():
        return (dg.grouped_gemm(A, B, o, out_dtype=F32), dg.grouped_gemm_wgrad(A, x, o),
                dg.w4_gemm(x, q, s, zeros=z, offsets=o, out_dtype=F32),
                dg.newton_schulz(G, workspace=ws))

    calls()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, w, v, n = calls()
    for b in ([0, 10, 30, 60], [0, 0, 59, 60], [5, 25, 25, 40]):
        o.copy_(offs(b))
        A.copy_(ints(rng, (T, K)))
        G.copy_(torch.randn((96, 160)))
        y.zero_(), v.zero_()
        g.replay()
        torch.cuda.synchronize()
        lo, hi = b[0], b[-1]
        equal(y[lo:hi], ref.grouped(A, B, b)[lo:hi], F32)
        equal(v[lo:hi], ref.w4(x, q, s, z, b)[lo:hi], F32)
        equal(w, ref.wgrad(A, x, b), BF)
        want = ref.newton_schulz(G)
        assert np.linalg.norm(ref.f64(n) - want) <= (ns_bound(5) + 2.0 ** -9) * np.linalg.norm(want)


@pytest.mark.parametrize("counts", [[1] * 8, [0, 5, 0, 40], [64], [3, 0, 13], [2] * 32])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("K,N", [(64, 40), (200, 72), (2048, 1000), (72, 4096)])
def test_few_rows(counts, layout, K, N):
    """Up to 64 rows: K split over clusters, tiles of 8 and 16 tokens, both layouts."""
    rng = np.random.default_rng(K + N + len(counts))
    b = bounds_of(counts)
    E = len(counts)
    A = ints(rng, (b[-1], K), -2, 2)
    B = ints(rng, (E, K, N) if layout == "row" else (E, N, K), -2, 2)
    B = B if layout == "row" else B.transpose(1, 2)
    bias = ints(rng, (E, N), dtype=F32)
    C0 = ints(rng, (b[-1], N), dtype=F32)
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), C0.to(DEV), alpha=0.5, beta=2.0,
                          bias=bias.to(DEV), epilogue="bias_relu")
    equal(got, ref.grouped(A, B, b, C0, 0.5, 2.0, bias, "bias_relu"), F32)
    equal(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b)), ref.grouped(A, B, b), BF)
    W = B[:1].to(DEV).expand(E, K, N)
    equal(dg.grouped_gemm(A.to(DEV), W, offs(b), out_dtype=F32),
          ref.grouped(A, B[:1].expand(E, K, N), b), F32)
    assert status() == 0


@pytest.mark.parametrize("layout", ["row", "col"])
def test_few_rows_do_not_mix(layout):
    """NaN and infinite rows stay in their rows, NaN weights in their group, and what lies
    beside the operands in padded rows stays out."""
    rng = np.random.default_rng(17)
    b = bounds_of([20, 1, 0, 30, 3], 1)
    K, N, E = 136, 72, 5
    A = ints(rng, (b[-1] + 2, K))
    B = ints(rng, (E, K, N))
    want = ref.grouped(A, B, b)
    Ap = torch.full((b[-1] + 2, K + 8), float("nan"), dtype=BF, device=DEV)
    Ap[:, :K] = A.to(DEV)
    Ap[8], Ap[30] = float("nan"), float("inf")
    if layout == "row":
        Bp = torch.full((E, K, N + 8), float("nan"), dtype=BF, device=DEV)
        Bp[:, :, :N] = B.to(DEV)
        Bd = Bp[:, :, :N]
    else:
        Bp = torch.full((E, N, K + 8), float("nan"), dtype=BF, device=DEV)
        Bp[:, :, :K] = B.transpose(1, 2).to(DEV)
        Bd = Bp[:, :, :K].transpose(1, 2)
    Bd[4] = float("nan")
    got = ref.f64(dg.grouped_gemm(Ap[:, :K], Bd, offs(b), out_dtype=F32))
    keep = [i for i in range(b[0], b[4]) if i not in (8, 30)]
    assert np.array_equal(got[keep], want[keep])
    assert np.isnan(got[8]).all() and np.isnan(got[b[4]:b[5]]).all()
    assert not np.isfinite(got[30]).any()


@pytest.mark.parametrize("rows", [8, 70, 200, 3000])
def test_a_stalled_pipeline_reports_a_timeout_and_recovers(rows):
    """One stage is left unfilled (a flag that nothing sets), in each tile shape."""
    rng = np.random.default_rng(53)
    A, B = ints(rng, (rows, 256)), ints(rng, (2, 256, 1024))
    b = [0, rows // 2, rows]
    dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b))
    dg.gemm_set_option(dg.Option.TIMEOUT_US, 20000)
    try:
        dg.gemm_set_option(dg.Option.TEST_STALL, 1)
        dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b))
        assert status() == dg.Status.ERR_TIMEOUT
    finally:
        dg.gemm_set_option(dg.Option.TEST_STALL, 0)
        dg.gemm_set_option(dg.Option.TIMEOUT_US, 1000000)
    equal(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=F32), ref.grouped(A, B, b), F32)
    assert status() == 0


def test_debug_build_trips_no_check():
    """The same sources with device-side bounds checks: each operator at ragged sizes."""
    D = dg.debug_lib()
    rng = np.random.default_rng(54)
    st = torch.cuda.current_stream().cuda_stream
    b = bounds_of([0, 33, 200, 7], 1)
    T, K, N, E = b[-1] + 2, 72, 136, 4
    A, B, X = ints(rng, (T, K)).to(DEV), ints(rng, (E, K, N)).to(DEV), ints(rng, (T, N)).to(DEV)
    o = offs(b)
    C = torch.full((T, N), float("nan"), dtype=F32, device=DEV)
    assert D.gemm_grouped(0, E, T, N, K, A.data_ptr(), K, B.data_ptr(), N, 0, K * N, C.data_ptr(), N,
                          2, o.data_ptr(), 1.0, 0.0, 0, 0, 0, 0, 0, st) == 0
    few = [0, 3, 20, 20, 33]
    of = offs(few)
    C2 = torch.full((33, N), float("nan"), dtype=BF, device=DEV)
    assert D.gemm_grouped(0, E, 33, N, K, A.data_ptr(), K, B.data_ptr(), N, 0, K * N, C2.data_ptr(),
                          N, 0, of.data_ptr(), 1.0, 0.0, 0, 0, 0, 0, 0, st) == 0
    W = torch.empty((E, K, N), dtype=BF, device=DEV)
    assert D.gemm_grouped_wgrad(0, E, T, K, N, A.data_ptr(), K, X.data_ptr(), N, W.data_ptr(), N,
                                K * N, 0, o.data_ptr(), 1.0, 0.0, 0, 0, st) == 0
    G = torch.randn((2, 130, 200), device=DEV)
    need = D.gemm_newton_schulz_workspace_size(2, 130, 200)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    O = torch.empty((2, 130, 200), dtype=BF, device=DEV)
    assert D.gemm_newton_schulz(2, 2, 130, 200, G.data_ptr(), 200, 26000, O.data_ptr(), 200, 26000,
                                0, 5, 3.4445, -4.775, 2.0315, 1e-7, ws.data_ptr(), need, st) == 0
    x, q, s, z = (t.to(DEV) for t in w4_case(rng, 5, 70, 320, 64, True))
    Y = torch.empty((5, 70), dtype=F32, device=DEV)
    assert D.gemm_w4(0, 1, 5, 70, 320, x.data_ptr(), 320, q.data_ptr(), s.data_ptr(), z.data_ptr(),
                     64, Y.data_ptr(), 70, 2, 0, 0, 0, 0, 0, 0, st) == 0
    assert D.gemm_check_device_status(st) == 0
    equal(C, ref.grouped(A, B, b), F32)
    equal(C2, ref.grouped(A[:33], B, few), BF)
    equal(W, ref.wgrad(A, X, b), BF)
    equal(Y, ref.w4(x, q, s, z), F32)
    want = ref.newton_schulz(G)
    assert np.linalg.norm(ref.f64(O) - want) <= (ns_bound(5) + 2.0 ** -9) * np.linalg.norm(want)


def test_example_runs():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    first, last, gap = mod.main(tokens=512, width=256, hidden=512, experts=8, top=2, steps=12,
                                quiet=True)
    assert last < 0.9 * first and gap < 0.2


def test_more_groups_than_a_grid_holds_are_copied():
    """65537 matrices that TMA cannot address (5 columns), and as many groups in place."""
    rng = np.random.default_rng(61)
    E, K, N = 65537, 3, 5
    rows = [0, 1, 65534, 65535, 65536]
    counts = np.zeros(E, dtype=np.int64)
    counts[rows] = [2, 1, 3, 30, 40]
    b = bounds_of(counts)
    A, B = ints(rng, (b[-1], K)), ints(rng, (E, K, N))
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=F32)
    want = np.concatenate([ref.f64(A[b[e]:b[e + 1]]) @ ref.f64(B[e]) for e in rows])
    equal(got, want, F32)
    W = ints(rng, (E, 8, 8)).to(DEV)
    A = ints(rng, (b[-1], 8))
    got = dg.grouped_gemm(A.to(DEV), W, offs(b), out_dtype=F32)
    want = np.concatenate([ref.f64(A[b[e]:b[e + 1]]) @ ref.f64(W[e]) for e in rows])
    equal(got, want, F32)
    assert status() == 0


FIRST_CALLS = """
import torch
import dense_gemm_bf16_gb300 as dg
A = torch.ones((256, 256), dtype=torch.bfloat16, device="cuda:0")
B = torch.ones((2, 256, 256), dtype=torch.bfloat16, device="cuda:0")
o = torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda:0")
C, Y = torch.empty_like(A), torch.empty_like(A)
from dense_gemm_bf16_gb300 import api, experts

def free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]

at_first = free()
dg.gemm(A, A, C)
dense = free()
if {capture}:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.grouped_gemm(A, B, o, Y)
    g.replay()
else:
    dg.grouped_gemm(A, B, o, Y)
with_experts = free()
assert bool((Y == 256).all()) and dg.gemm_check_device_status(0) == 0
assert dense < at_first
assert {capture} or with_experts < dense, "the dense product loaded the expert kernels"
"""


@pytest.mark.parametrize("capture", [False, True])
def test_a_dense_product_does_not_load_the_expert_kernels(capture):
    """In a process of its own: kernels take device memory when they are prepared, the
    dense ones at the first dense call and the others at the first call of theirs, which
    may be a captured one."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(capture=capture)], cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


# rows in all, experts, N: few rows, and the ragged kernel in tiles of 32 columns, of 128,
# and in pairs (at least 38 tiles of 256 x 256)
VARIANTS = {"few": (60, 4, 256), "t32": (110, 4, 256), "t128": (700, 4, 256),
            "pairs": (3000, 4, 1000)}


@pytest.mark.parametrize("case", sorted(VARIANTS))
@pytest.mark.parametrize("layout", ["row", "col"])
def test_grouped_results_do_not_depend_on_the_other_groups(case, layout):
    """At equal T and number of groups the others' rows, weights and sizes change, and the
    one group's place with them; its fp32 sums stay equal bit for bit."""
    T, E, N = VARIANTS[case]
    K, n = 520, T // 3
    g = torch.Generator(device=DEV).manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(BF)

    rows, weights = rand(n, K), rand(K, N) if layout == "row" else rand(N, K).t()
    got = []
    for sizes, e in (([n // 2, n, T - n - n // 2, 0], 1), ([0, T - n, n, 0], 2),
                     ([n, 1, T - n - 5, 4], 0), ([T - n, 0, 0, n], 3)):
        b = bounds_of(sizes)
        assert b[-1] == T
        A, B = rand(T, K) * 100, rand(E, K, N) if layout == "row" else rand(E, N, K).transpose(1, 2)
        A[b[e]:b[e + 1]], B[e] = rows, weights
        got.append(dg.grouped_gemm(A, B, offs(b), out_dtype=F32)[b[e]:b[e + 1]])
    assert float(got[0].abs().max()) > 1.0
    for other in got[1:]:
        assert torch.equal(got[0], other)
    assert status() == 0


@pytest.mark.parametrize("T,out", [(30, BF), (30, F32), (150, F32), (200, BF)])
def test_w4_results_do_not_depend_on_the_other_experts(T, out):
    """The same for 4-bit experts: the integers themselves, and 16-bit weights (200 rows)."""
    E, K, N, n = 4, 512, 200, T // 3
    g = torch.Generator(device=DEV).manual_seed(6)
    q0 = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s0 = torch.rand((N, K // 64), generator=g, device=DEV).to(BF)
    rows = torch.randn((n, K), generator=g, device=DEV).to(BF)
    got = []
    for sizes, e in (([n // 2, n, T - n - n // 2, 0], 1), ([0, T - n, n, 0], 2), ([T - n, 0, 0, n], 3)):
        b = bounds_of(sizes)
        x = torch.randn((T, K), generator=g, device=DEV).to(BF)
        q = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        s = torch.rand((E, N, K // 64), generator=g, device=DEV).to(BF)
        x[b[e]:b[e + 1]], q[e], s[e] = rows, q0, s0
        got.append(dg.w4_gemm(x, q, s, offsets=offs(b), out_dtype=out)[b[e]:b[e + 1]])
    for other in got[1:]:
        assert torch.equal(got[0], other)


# ---------------------------------------------------------------- CTA pairs
# Row products and the 16-bit route of 4-bit ones take pairs of CTAs (tiles of 256 x 256)
# from half as many tiles on as pairs fit the GPU (38 of 76): groups * ceil(N / 256) *
# ceil(rows of a group on average / 256) of them, and more than 128 rows and columns.

PAIR_COUNTS = [300, 0, 513, 700, 31, 257]               # 1801 rows, 301 on average: 2 x 6 x
                                                        # ceil(N / 256) >= 48 tiles


def on_pairs(E, T, N):
    avg = -(-T // E)
    return avg > 128 and N > 128 and E * -(-N // 256) * -(-avg // 256) >= 38


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, F32), (HF, HF), (HF, F32)])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("K,N", [(320, 1000), (200, 1032), (64, 1001), (136, 1288)])
def test_grouped_pairs_exact(K, N, layout, dtype, out):
    """Both layouts (two K blocks a load where K is a multiple of 64), widths in steps of
    32, and rows of C that start on odd addresses (N = 1001)."""
    rng = np.random.default_rng(K + N)
    b = bounds_of(PAIR_COUNTS, 2)
    T, E = b[-1] + 1, len(PAIR_COUNTS)
    assert on_pairs(E, T, N)
    A = ints(rng, (T, K), dtype=dtype)
    B = ints(rng, (E, K, N) if layout == "row" else (E, N, K), dtype=dtype)
    B = B if layout == "row" else B.transpose(1, 2)
    C = torch.full((T, N), float("nan"), dtype=out, device=DEV)
    dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), C)
    equal(C, ref.grouped(A, B, b), out)
    assert status() == 0


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("N", [1000, 1001])
def test_grouped_pairs_beta_bias_relu(N, out, layout):
    rng = np.random.default_rng(71)
    b = bounds_of(PAIR_COUNTS, 1)
    T, K, E = b[-1] + 2, 200, len(PAIR_COUNTS)
    assert on_pairs(E, T, N)
    A, bias, C0 = ints(rng, (T, K)), ints(rng, (E, N), dtype=F32), ints(rng, (T, N), dtype=out)
    B = ints(rng, (E, K, N)) if layout == "row" else ints(rng, (E, N, K)).transpose(1, 2)
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), C0.to(DEV), alpha=2.0, beta=-0.5,
                          bias=bias.to(DEV), epilogue="bias_relu")
    equal(got, ref.grouped(A, B, b, C0, 2.0, -0.5, bias, "bias_relu"), out)


@pytest.mark.parametrize("copied", ["A", "B", "both"])
def test_grouped_pairs_with_copied_operands(copied):
    """Operands of odd pitch: the product is launched while their copy runs."""
    rng = np.random.default_rng(72)
    b = bounds_of(PAIR_COUNTS)
    T, K, N, E = b[-1], 192, 1000, len(PAIR_COUNTS)
    assert on_pairs(E, T, N)
    A = ints(rng, (T, K + (copied != "B"))).to(DEV)[:, :K]
    B = ints(rng, (E, K, N + (copied != "A"))).to(DEV)[:, :, :N]
    for _ in range(3):
        equal(dg.grouped_gemm(A, B, offs(b), out_dtype=F32), ref.grouped(A, B, b), F32)
    assert status() == 0


@pytest.mark.parametrize("epilogue", ["bias_gelu_tanh", "gelu_erf"])
def test_grouped_pairs_gelu(epilogue):
    """The bound of test_grouped_gelu, for a 16-bit output with its own rounding (2^-8)."""
    rng = np.random.default_rng(73)
    b = bounds_of(PAIR_COUNTS)
    T, K, N, E = b[-1], 320, 1000, len(PAIR_COUNTS)
    assert on_pairs(E, T, N)
    A = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(BF)
    B = torch.from_numpy(rng.standard_normal((E, N, K)).astype(np.float32) / 18).to(BF).transpose(1, 2)
    bias = torch.from_numpy(rng.standard_normal((E, N)).astype(np.float32))
    use = bias if epilogue.startswith("bias") else None
    want = ref.grouped(A, B, b, bias=use, epilogue=epilogue)
    size = ref.grouped(A.abs(), B.abs(), b, bias=None if use is None else use.abs())
    for out in (F32, BF):
        got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=out, epilogue=epilogue,
                              bias=None if use is None else use.to(DEV))
        bound = 1.13 * K * 2.0 ** -23 * size + 2.0 ** -20 * (size + np.abs(want))
        if out == BF:
            bound = bound + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(ref.f64(got) - want) <= bound)


def test_grouped_pairs_do_not_mix_rows():
    rng = np.random.default_rng(74)
    b = bounds_of(PAIR_COUNTS)
    T, K, N, E = b[-1], 136, 1000, len(PAIR_COUNTS)
    A, B = ints(rng, (T, K)), ints(rng, (E, K, N))
    want = ref.grouped(A, B, b)
    A[7], A[900], B[5] = float("nan"), float("inf"), float("nan")
    got = ref.f64(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=F32))
    keep = [i for i in range(b[5]) if i not in (7, 900)]
    assert np.array_equal(got[keep], want[keep])
    assert np.isnan(got[7]).all() and np.isnan(got[b[5]:]).all()


def test_grouped_pairs_replayed_from_a_graph():
    rng = np.random.default_rng(75)
    b = bounds_of(PAIR_COUNTS)
    T, K, N, E = b[-1], 128, 1000, len(PAIR_COUNTS)
    A, B, o = ints(rng, (T, K)).to(DEV), ints(rng, (E, K, N)).to(DEV), offs(b)
    odd = ints(rng, (E, K, N + 1)).to(DEV)[:, :, :N]       # copied in every replay
    y, z = (torch.empty((T, N), dtype=F32, device=DEV) for _ in range(2))
    dg.grouped_gemm(A, odd, o, z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.grouped_gemm(A, B, o, y)
        dg.grouped_gemm(A, odd, o, z)
    for counts in (PAIR_COUNTS, PAIR_COUNTS[::-1], [0, 0, T, 0, 0, 0]):
        b = bounds_of(counts)
        o.copy_(offs(b))
        A.copy_(ints(rng, (T, K)))
        y.zero_(), z.zero_()
        g.replay()
        torch.cuda.synchronize()
        equal(y, ref.grouped(A, B, b), F32)
        equal(z, ref.grouped(A, odd, b), F32)
    assert status() == 0


@pytest.mark.parametrize("out", [F32, BF])
@pytest.mark.parametrize("odd", [0, 1])
def test_wgrad_pairs_accumulate(odd, out):
    """beta on the pair tiles; odd: copied operands, and a C of odd rows (no TMA stores)."""
    rng = np.random.default_rng(76)
    b = bounds_of([300, 0, 77, 130, 16, 1000], 1)
    M, N, T = 1000 + odd, 1032 + odd, b[-1] + 1
    A, D = ints(rng, (T, M), -2, 2), ints(rng, (T, N), -2, 2)
    C0 = ints(rng, (6, M, N), dtype=out)
    got = dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs(b), C0.to(DEV), alpha=0.5, beta=2.0)
    equal(got, ref.wgrad(A, D, b, C0, 0.5, 2.0), out)
    assert status() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("experts", [0, 4])
def test_w4_pairs(experts, dtype):
    """The 16-bit route on pair tiles: one matrix (equal widths), and experts."""
    rng = np.random.default_rng(77 + experts)
    counts = [900, 0, 513, 700] if experts else [2000]
    b = bounds_of(counts)
    T, N, K = b[-1], 1032, 320
    assert on_pairs(len(counts), T, N)
    x, q, s, z = w4_case(rng, T, N, K, 64, True, dtype, experts)
    bias = ints(rng, (N,), dtype=F32)
    got = w4_run(x, q, s, z, bias=bias.to(DEV), epilogue="bias_relu",
                 offsets=offs(b) if experts else None)
    equal(got, ref.w4(x, q, s, z, b if experts else None, bias, "bias_relu"), dtype)
    assert status() == 0


# ---------------------------------------------------------------- K over four CTAs
# Few rows and the direct 4-bit form cut K over a cluster of four where the units (tiles
# of 64 rows by the tokens of a tile) are at most 38 (a quarter of the SMs) and K has
# 16 stages: of 128 with 16-bit weights, of 256 (groups of 32, more than 16 tokens) or 512.

@pytest.mark.parametrize("group,K", [(32, 8192), (64, 16384), (128, 16384), (128, 16512), (32, 8224)])
@pytest.mark.parametrize("T,N", [(1, 200), (9, 130), (33, 70)])
def test_w4_split_over_four(T, N, group, K):
    rng = np.random.default_rng(T + K)
    x, q, s, z = w4_case(rng, T, N, K, group, True)
    x = x.clamp(-1, 1)                                     # sums below 2^24 quarters
    bias = ints(rng, (N,), dtype=F32)
    for out in (F32, BF):
        equal(w4_run(x, q, s, z, out_dtype=out, bias=bias.to(DEV), epilogue="bias_relu"),
              ref.w4(x, q, s, z, bias=bias, epilogue="bias_relu"), out)
    assert status() == 0


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("counts", [[1], [1, 0, 1], [5, 0, 9], [30]])
@pytest.mark.parametrize("K,N", [(4096, 200), (4104, 130), (5000, 72)])
def test_few_rows_split_over_four(K, N, counts, layout):
    rng = np.random.default_rng(K + N)
    b = bounds_of(counts, 1)
    E, T = len(counts), b[-1] + 1
    A, bias = ints(rng, (T, K), -2, 2), ints(rng, (E, N), dtype=F32)
    B = ints(rng, (E, K, N), -2, 2) if layout == "row" else \
        ints(rng, (E, N, K), -2, 2).transpose(1, 2)
    C0 = ints(rng, (T, N), dtype=F32)
    got = dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), C0.to(DEV), alpha=0.5, beta=2.0,
                          bias=bias.to(DEV), epilogue="bias_relu")
    equal(got, ref.grouped(A, B, b, C0, 0.5, 2.0, bias, "bias_relu"), F32)
    assert status() == 0


# ---------------------------------------------------------------- fp32 sums of other numbers

def prefix_norms(A, D, step=16):
    """sum over the MMA steps j of |P_j|_F, P_j the exact sum after j steps of 16."""
    P, total = np.zeros((A.shape[1], D.shape[1])), 0.0
    for k in range(0, A.shape[0], step):
        P += A[k:k + step].T @ D[k:k + step]
        total += np.linalg.norm(P)
    return P, total


@pytest.mark.parametrize("counts,M,N", [([900, 77, 1500], 120, 136), ([513, 0, 1000, 300, 700, 31], 1000, 1032)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_wgrad_fp32_sums(counts, M, N, dtype):
    """Normal inputs: the accumulator holds 24 bits and each step of 16 may lose one unit
    in the last place of it, so the error's norm is at most 2^-23 times the sum of the
    norms of the partial sums."""
    rng = np.random.default_rng(81)
    b = bounds_of(counts)
    A = torch.from_numpy(rng.standard_normal((b[-1], M)).astype(np.float32)).to(dtype)
    D = torch.from_numpy(rng.standard_normal((b[-1], N)).astype(np.float32)).to(dtype)
    got = ref.f64(dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs(b), out_dtype=F32))
    a, d = ref.f64(A), ref.f64(D)
    for e in range(len(counts)):
        want, size = prefix_norms(a[b[e]:b[e + 1]], d[b[e]:b[e + 1]])
        assert np.linalg.norm(got[e] - want) <= 2.0 ** -23 * size


@pytest.mark.parametrize("counts,K,N", [([20, 3, 30], 1000, 136), ([40, 30, 60], 2000, 136),
                                        ([300, 0, 513, 700, 31, 257], 1500, 1000)])
def test_grouped_fp32_sums(counts, K, N):
    """The same for the row products, by group: few rows, single CTAs, pairs.  (Few rows:
    slices of K are summed apart, which only shortens the partial sums' paths.)"""
    rng = np.random.default_rng(82)
    b = bounds_of(counts)
    A = torch.from_numpy(rng.standard_normal((b[-1], K)).astype(np.float32)).to(BF)
    B = torch.from_numpy(rng.standard_normal((len(counts), K, N)).astype(np.float32)).to(BF)
    got = ref.f64(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=F32))
    for e in range(len(counts)):
        if b[e] < b[e + 1]:
            want, size = prefix_norms(ref.f64(A[b[e]:b[e + 1]]).T, ref.f64(B[e]))
            assert np.linalg.norm(got[b[e]:b[e + 1]] - want) <= 2.0 ** -23 * size


# ---------------------------------------------------------------- Newton-Schulz, block by block

@pytest.mark.parametrize("shape", [(64, 64), (129, 257), (300, 200), (96, 1000), (3, 200, 264),
                                   (128, 2048), (6, 257, 130),                            # 64-column tiles
                                   (15, 257, 300), (15, 300, 257), (40, 100, 300),  # 128 columns
                                   (10, 520, 600), (20, 512, 640), (10, 600, 520),  # pairs
                                   (2100, 2304), (2310, 2100)])
@pytest.mark.parametrize("steps", [1, 5])
def test_newton_schulz_block_by_block(shape, steps):
    """Against the 64-bit result, the error may be 1.5 times that of the same steps with X,
    Y and the polynomial rounded to fp16 between exact products (fp32 sums and roundings
    that fall the other way add little to it): over every matrix, over its worst 32 x 32
    block, and twice that for its worst entry.  One wrong 8 x 8 part of a block is two
    hundred times its error."""
    rng = np.random.default_rng(sum(shape) + steps)
    G = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    got = ref.f64(dg.newton_schulz(G.to(DEV), steps=steps, out_dtype=HF))
    assert status() == 0
    want, near = ref.newton_schulz(G, steps), ref.newton_schulz_fp16(G, steps)
    if len(shape) == 2:
        got, want, near = got[None], want[None], near[None]
    for g, w, n in zip(got, want, near):
        for size in (w.shape, (32, 32), (1, 1)):
            allowed = max(blocks(n - w, size)) * (1.5 if size != (1, 1) else 2.0)
            assert max(blocks(g - w, size)) <= allowed, size


def blocks(x, size):
    """Root mean squares of the blocks of x."""
    if size == (1, 1):
        return [np.abs(x).max()]
    return [np.sqrt((x[i:i + size[0], j:j + size[1]] ** 2).mean())
            for i in range(0, x.shape[0], size[0]) for j in range(0, x.shape[1], size[1])
            if x[i:i + size[0], j:j + size[1]].size >= 256]   # (slivers: by entries)


# ---------------------------------------------------------------- waits that run out

def stalled(call):
    """`call` with one stage left unfilled and a short limit: its status."""
    dg.gemm_set_option(dg.Option.TIMEOUT_US, 20000)
    try:
        dg.gemm_set_option(dg.Option.TEST_STALL, 1)
        call()
        return status()
    finally:
        dg.gemm_set_option(dg.Option.TEST_STALL, 0)
        dg.gemm_set_option(dg.Option.TIMEOUT_US, 1000000)


@pytest.mark.parametrize("M,N", [(72, 136), (1000, 1032)])
@pytest.mark.parametrize("out", [F32, BF])
def test_a_stalled_weight_gradient_recovers(M, N, out):
    """Ragged groups, so that the tail warp waits too; single CTAs and pairs."""
    rng = np.random.default_rng(91)
    b = bounds_of([300, 0, 77, 130, 17, 401])
    A, D = ints(rng, (b[-1], M), -2, 2).to(DEV), ints(rng, (b[-1], N), -2, 2).to(DEV)
    assert stalled(lambda: dg.grouped_gemm_wgrad(A, D, offs(b), out_dtype=out)) == \
        dg.Status.ERR_TIMEOUT
    equal(dg.grouped_gemm_wgrad(A, D, offs(b), out_dtype=out), ref.wgrad(A, D, b), out)
    assert status() == 0


@pytest.mark.parametrize("shape", [(100, 140), (15, 257, 300), (20, 512, 640), (10, 600, 520)])
def test_a_stalled_newton_schulz_recovers(shape):
    """CTAs whose own pipeline does not stall wait for a matrix's counter in vain."""
    G = torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(7), device=DEV)
    want = dg.newton_schulz(G)
    assert status() == 0
    assert stalled(lambda: dg.newton_schulz(G)) == dg.Status.ERR_TIMEOUT
    assert torch.equal(dg.newton_schulz(G), want)
    assert status() == 0


@pytest.mark.parametrize("T,N,K,experts", [(1, 200, 16384, 0), (2, 2500, 4096, 0), (40, 300, 512, 0),
                                           (12, 136, 320, 4)])
def test_a_stalled_4_bit_product_recovers(T, N, K, experts):
    """Four and two CTAs of a cluster, whose barriers go on after the failed wait; single
    CTAs with one and with several units."""
    rng = np.random.default_rng(92)
    x, q, s, z = (t.to(DEV) for t in w4_case(rng, T, N, K, 64, True, BF, experts))
    x = x.clamp(-1, 1)
    b = bounds_of([3, 0, 8, 1]) if experts else None

    def call():
        return dg.w4_gemm(x, q, s, zeros=z, offsets=offs(b) if b else None, out_dtype=F32)

    assert stalled(call) == dg.Status.ERR_TIMEOUT
    equal(call(), ref.w4(x, q, s, z, b), F32)
    assert status() == 0


# ---------------------------------------------------------------- process-wide options

def elapsed(call):
    """The shortest of five calls, in ms."""
    times = []
    for _ in range(5):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        call()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end))
    return min(times)


@pytest.mark.parametrize("cap", [1, 4, 7])
def test_the_cap_on_ctas_holds(cap):
    """GEMM_OPT_MAX_CTAS leaves the other SMs to other work: the same results, in at least
    four times the time of the whole GPU for products that fill it."""
    rng = np.random.default_rng(95)
    b = bounds_of([700, 0, 1300, 1096, 500, 500])
    T, K, N, E = b[-1], 2048, 2048, 6
    A, B, D = ints(rng, (T, K)).to(DEV), ints(rng, (E, K, N)).to(DEV), ints(rng, (T, N)).to(DEV)
    x, q, s, z = (t.to(DEV) for t in w4_case(rng, 6, 32768, 4096, 64, True))
    G, o = torch.randn((24, 512, 640), device=DEV), offs(b)
    few = offs([0, 3, 3, 5, 6, 6, 6])
    calls = (lambda: dg.grouped_gemm(A, B, o, out_dtype=F32),
             lambda: dg.grouped_gemm_wgrad(A, D, o, out_dtype=F32),
             lambda: dg.w4_gemm(x, q, s, zeros=z, out_dtype=F32),
             lambda: dg.grouped_gemm(x[:, :K], B, few, out_dtype=F32),
             lambda: dg.newton_schulz(G))
    free = [c() for c in calls]
    fast = [elapsed(c) for c in calls]
    dg.gemm_set_option(dg.Option.MAX_CTAS, cap)
    try:
        capped = [c() for c in calls]
        slow = [elapsed(c) for c in calls]
    finally:
        dg.gemm_set_option(dg.Option.MAX_CTAS, 0)
    for u, v in zip(free[:4], capped[:4]):
        assert torch.equal(u, v)                       # (exact)
    assert float((free[4].float() - capped[4].float()).norm()) <= \
        2.0 ** -8 * float(free[4].float().norm())
    for i in (0, 1, 2, 4):
        assert slow[i] > 4 * fast[i], (i, slow[i], fast[i])
    assert status() == 0


@pytest.mark.parametrize("overlap", [0, 1])
def test_copied_operands_with_and_without_overlap(overlap):
    """GEMM_OPT_OVERLAP_COPY: the product starts while its operand is prepared, or after."""
    rng = np.random.default_rng(96)
    b = bounds_of(PAIR_COUNTS)
    T, K, N, E = b[-1], 201, 1000, len(PAIR_COUNTS)
    A, B, D = ints(rng, (T, K)), ints(rng, (E, K, N)), ints(rng, (T, N))
    x, q, s, z = w4_case(rng, 300, 1032, 320, 64, True)
    dg.gemm_set_option(dg.Option.OVERLAP_COPY, overlap)
    try:
        for _ in range(3):
            equal(dg.grouped_gemm(A.to(DEV), B.to(DEV), offs(b), out_dtype=F32),
                  ref.grouped(A, B, b), F32)
            equal(dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs(b), out_dtype=F32),
                  ref.wgrad(A, D, b), F32)
            equal(w4_run(x, q, s, z), ref.w4(x, q, s, z), BF)
    finally:
        dg.gemm_set_option(dg.Option.OVERLAP_COPY, 0)
    assert status() == 0


# ---------------------------------------------------------------- fp32 sums of any length

def segment_bound(A, D, length=768, step=128):
    """(exact A^T D, bound on the norm of an fp32 result's error).  Each step of 16 may lose
    one unit in the last place of its accumulator (2^-23 of the partial sum's norm, taken
    at the nearer end of a block of eight steps); accumulators of `length` products err
    independently (normal inputs), so their errors add in squares; adding them up rounds
    to nearest, 2^-24 of the running sum each time."""
    total, squares = np.zeros((A.shape[1], D.shape[1])), 0.0
    for s in range(0, A.shape[0], length):
        P, before, size = np.zeros_like(total), 0.0, 0.0
        for k in range(s, min(s + length, A.shape[0]), step):
            e = min(k + step, s + length)
            P += A[k:e].T @ D[k:e]
            after = np.linalg.norm(P)
            size += step / 16 * max(before, after)
            before = after
        total += P
        squares += (2.0 ** -23 * size) ** 2 + (2.0 ** -24 * np.linalg.norm(total)) ** 2
    return total, np.sqrt(squares)


@pytest.mark.parametrize("M,N", [(120, 136), (1600, 1608)])
@pytest.mark.parametrize("odd", [0, 9])
def test_wgrad_fp32_sums_do_not_lose_with_their_length(M, N, odd):
    """16384 rows in one group (and nine more, a ragged tail): single CTAs and pairs."""
    rng = np.random.default_rng(97)
    T = 16384 + odd
    A = torch.from_numpy(rng.standard_normal((T, M)).astype(np.float32)).to(BF)
    D = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).to(BF)
    got = ref.f64(dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs([0, T]), out_dtype=F32))[0]
    want, bound = segment_bound(ref.f64(A), ref.f64(D))
    assert np.linalg.norm(got - want) <= bound
    assert status() == 0


@pytest.mark.parametrize("T,N", [(90, 200), (300, 200), (1600, 1608)])
@pytest.mark.parametrize("K", [16384, 16394])
def test_grouped_fp32_sums_do_not_lose_with_their_length(T, N, K):
    """Tiles of 32 columns, of 128, and pairs; K in whole stages and not."""
    rng = np.random.default_rng(98)
    A = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(BF)
    B = torch.from_numpy(rng.standard_normal((1, K, N)).astype(np.float32)).to(BF)
    E = 4 if T == 90 else 1
    b = bounds_of([T // E] * (E - 1) + [T - T // E * (E - 1)])
    got = ref.f64(dg.grouped_gemm(A.to(DEV), B.to(DEV).expand(E, K, N), offs(b), out_dtype=F32))
    want, bound = segment_bound(ref.f64(A).T, ref.f64(B[0]))
    assert np.linalg.norm(got - want) <= bound
    assert status() == 0


@pytest.mark.parametrize("T", [4, 30])
@pytest.mark.parametrize("layout", ["row", "col"])
def test_few_rows_fp32_sums_do_not_lose_with_their_length(T, layout):
    """131072 products, 128 of them in a matrix instruction's accumulator at a time."""
    rng = np.random.default_rng(99)
    K, N = 131072, 200
    A = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(BF)
    B = torch.from_numpy(rng.standard_normal((K, N)).astype(np.float32)).to(BF)
    Bd = B.to(DEV) if layout == "row" else B.t().contiguous().to(DEV).t()
    got = ref.f64(dg.grouped_gemm(A.to(DEV), Bd[None], offs([0, T]), out_dtype=F32))
    want, bound = segment_bound(ref.f64(A).T, ref.f64(B), 128, 16)
    assert np.linalg.norm(got - want) <= bound
    assert status() == 0


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts", [None, [200, 0, 160, 3]])
def test_w4_exact_option_rounds_once(counts, dtype):
    """Many rows with a 16-bit output, as the caller asks: the fp32 result (of the integers
    themselves), rounded once.  By default the weights' own rounding is in it too."""
    rng = np.random.default_rng(100)
    E, N, K = (len(counts) if counts else 0), 264, 512
    b = bounds_of(counts) if counts else None
    T = b[-1] if counts else 300
    x, q, s, z = w4_case(rng, T, N, K, 64, True, dtype, E)
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(dtype)
    s = torch.from_numpy(rng.uniform(0.01, 0.02, s.shape).astype(np.float32)).to(dtype)
    kw = dict(offsets=offs(b)) if counts else {}
    once = w4_run(x, q, s, z, out_dtype=F32, **kw).to(dtype)
    default = w4_run(x, q, s, z, **kw)
    dg.gemm_set_option(dg.Option.W4_EXACT, 1)
    try:
        got = w4_run(x, q, s, z, **kw)
    finally:
        dg.gemm_set_option(dg.Option.W4_EXACT, 0)
    assert torch.equal(got, once)
    assert not torch.equal(default, once)
    assert status() == 0


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("counts", [[5, 0, 20], [300, 77, 900]])
def test_weights_side_by_side(counts, layout):
    """The experts' weights as column (row) blocks of one wide matrix, and their gradients
    into such blocks: neighbours' columns stay what they were."""
    rng = np.random.default_rng(101)
    b, E, K, N = bounds_of(counts), len(counts), 264, 136
    T = b[-1]
    A, D = ints(rng, (T, K), -2, 2), ints(rng, (T, N), -2, 2)
    wide = ints(rng, (K, E * N)) if layout == "row" else ints(rng, (N, E * K))
    B = wide.view(K, E, N).transpose(0, 1) if layout == "row" else \
        wide.view(N, E, K).permute(1, 2, 0)
    Bd = wide.to(DEV)
    Bd = Bd.view(K, E, N).transpose(0, 1) if layout == "row" else Bd.view(N, E, K).permute(1, 2, 0)
    assert Bd.stride() == B.stride() and Bd.shape == (E, K, N)
    equal(dg.grouped_gemm(A.to(DEV), Bd, offs(b), out_dtype=F32), ref.grouped(A, B, b), F32)
    for out in (F32, BF):
        C = torch.full((K, E * N + 8), 3.0, dtype=out, device=DEV)
        blocks = C.as_strided((E, K, N), (N, E * N + 8, 1))
        dg.grouped_gemm_wgrad(A.to(DEV), D.to(DEV), offs(b), blocks, beta=1.0)
        equal(blocks, ref.wgrad(A, D, b, torch.full((E, K, N), 3.0), beta=1.0), out)
        assert bool((C[:, E * N:] == 3).all())
    assert status() == 0


def test_newton_schulz_results_side_by_side():
    G = torch.randn((3, 40, 56), generator=torch.Generator(device=DEV).manual_seed(8), device=DEV)
    wide = torch.full((40, 3 * 56 + 4), 2.0, dtype=BF, device=DEV)
    out = wide.as_strided((3, 40, 56), (56, 3 * 56 + 4, 1))
    dg.newton_schulz(G, out)
    assert torch.equal(out, dg.newton_schulz(G)) and bool((wide[:, 168:] == 2).all())
