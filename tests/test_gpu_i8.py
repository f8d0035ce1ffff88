"""Rows quantised to 8 bits and products of 8-bit integers on the GPU, against plain 64-bit
references: the integers and the sums exactly, results without bias bit for bit."""
import numpy as np
import pytest
import torch

import dense_gemm_bf16_gb300 as dg
import experts_ref
import routing_ref as ref
from routing_ref import HALF_STEP, TINIEST

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
DEV = "cuda:0"


def status():
    return dg.gemm_check_device_status(torch.cuda.current_stream().cuda_stream)


def offs(bounds):
    return torch.tensor(bounds, dtype=torch.int32, device=DEV)


def bounds_of(counts, start=0):
    return [start + int(v) for v in np.concatenate(([0], np.cumsum(counts)))]


# ---------------------------------------------------------------- quantise

def quantized_exactly(x, q, s):
    want, scales = ref.quantize(x)
    assert np.array_equal(q.cpu().numpy(), want)
    got = experts_ref.f64(s)
    assert np.array_equal(np.isnan(got), np.isnan(scales))
    ok = ~np.isnan(scales)
    assert np.array_equal(got[ok], scales[ok].astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,K", [(1, 1), (3, 7), (5, 64), (64, 255), (33, 1024), (9, 4096), (1001, 130),
                                 (2, 8192), (3, 8200), (2, 40001), (700, 2048), (4, 16384)])
def test_quantize(T, K, dtype):
    rng = np.random.default_rng(T * 31 + K)
    x = rng.standard_normal((T, K)) * np.exp(2 * rng.standard_normal((T, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(dtype)
    q, s = dg.i8_quantize(x.to(DEV))
    quantized_exactly(x, q, s)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_quantize_borders_and_ties(dtype):
    """Rows whose largest magnitude is 127 times a power of two, with every half integer and
    its neighbours among the elements, both signs."""
    half = torch.arange(0, 127, dtype=torch.float64) + 0.5
    rows = []
    for e in (-8, -1, 0, 3):
        v = half.to(dtype)
        bits = v.view(torch.int32 if dtype == F32 else torch.int16)
        near = [v, (bits + 1).view(dtype), (bits - 1).view(dtype)]
        v = torch.cat(near + [-n for n in near] + [torch.full((2,), 127.0, dtype=dtype)])
        rows.append((v.double() * 2.0 ** e).to(dtype))
    x = torch.stack(rows)
    q, s = dg.i8_quantize(x.to(DEV))
    quantized_exactly(x, q, s)


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantize_every_pair_of_significands(dtype):
    """Each row's largest element has another significand, and the row holds all significands
    from there down to quotients below one half: 16-bit quotients are decided by their distance
    from a border, which no pair may come below."""
    ones = 128 if dtype == BF else 1024          # the lowest significand, as an integer
    tops = torch.arange(ones, 2 * ones, device=DEV)[:, None]
    halvings = 10
    m = torch.arange(ones, 2 * ones, device=DEV).repeat(halvings)
    down = torch.arange(halvings, device=DEV).repeat_interleave(ones)
    num, den = 127 * m[None], tops * 2 ** down[None]              # 127 x / max |x|
    over = (down[None] == 0) & (m[None] > tops)                   # (they would be the maximum)
    num, den = torch.where(over, 127, num), torch.where(over, 1, den)
    q = num // den
    twice = 2 * (num - q * den)
    want = q + ((twice > den) | ((twice == den) & (q % 2 == 1))).long()
    x = torch.where(over, tops.double(), m[None].double() / 2.0 ** down[None].double())
    sign = torch.where((m + down) % 2 == 0, 1, -1)[None]
    x = torch.cat([x * sign, tops.double()], 1).to(dtype)
    assert bool((x.double().abs().amax(1) == tops[:, 0]).all())
    got, scales = dg.i8_quantize(x)
    assert bool((got[:, :-1].long() == want * sign).all()) and bool((got[:, -1] == 127).all())
    assert bool((scales == (tops[:, 0].double() / 127).float()).all())


def test_quantize_longest_row():
    K = 2 ** 31 - 4097
    x = torch.empty((1, K), dtype=BF, device=DEV).uniform_(-3, 3)
    x[0, K // 2] = 5.0
    q, s = dg.i8_quantize(x)
    assert s.item() == np.float32(5.0 / 127)
    for part in (slice(0, 10000), slice(K // 2 - 5000, K // 2 + 5000), slice(K - 10000, K)):
        # (a quotient is on a border, which 64 bits hold, or 2^-16 of itself away from one)
        assert torch.equal(q[0, part].double(), torch.round(127 * x[0, part].double() / 5.0))


@pytest.mark.parametrize("top", [3.3895e38, 1e37, 1e-10, 1e-30, 1.1e-38, 3e-42, 1.4e-45])
def test_quantize_extreme_rows(top):
    rng = np.random.default_rng(1)
    x = rng.uniform(-1, 1, (4, 300))
    x[:, 0] = 1.0
    with np.errstate(over="ignore"):
        x = torch.from_numpy((x * top).astype(np.float32))
    for dtype in (F32, BF):
        v = x.to(dtype)
        q, s = dg.i8_quantize(v.to(DEV))
        quantized_exactly(v, q, s)


def test_quantize_zero_nan_and_infinite_rows():
    x = torch.randn((6, 500))
    x[1], x[2, 7], x[3, 499], x[4, 0] = 0.0, float("nan"), float("inf"), -float("inf")
    for dtype in (BF, HF, F32):
        q, s = dg.i8_quantize(x.to(dtype).to(DEV))
        quantized_exactly(x.to(dtype), q, s)
        assert s[1] == 0 and torch.isnan(s[2:5]).all() and not torch.isnan(s[[0, 1, 5]]).any()


def test_quantize_views_and_leading_dimensions():
    rng = np.random.default_rng(2)
    w = torch.from_numpy(rng.standard_normal((3, 5, 48)).astype(np.float32))
    q, s = dg.i8_quantize(w.to(DEV))
    assert q.shape == (3, 5, 48) and s.shape == (3, 5)
    quantized_exactly(w, q, s)
    wide = w.to(DEV).to(BF)
    for view in (wide[:, :, 3:40], wide[:, 1:2], wide[:, :1, 5:6]):
        q, s = dg.i8_quantize(view)
        quantized_exactly(view.cpu(), q, s)
    with pytest.raises(ValueError, match="distance"):
        dg.i8_quantize(wide[:, :3])
    out = torch.full((5, 60), 9, dtype=torch.int8, device=DEV)
    dg.i8_quantize(wide[0], out=out[:, 7:55])
    quantized_exactly(wide[0].cpu(), out[:, 7:55], dg.i8_quantize(wide[0])[1])
    assert bool((out[:, :7] == 9).all()) and bool((out[:, 55:] == 9).all())
    assert dg.i8_quantize(wide[0, :0])[0].shape == (0, 48)
    assert dg.i8_quantize(wide[0, :, :0])[1].tolist() == [0.0] * 5


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [5, 37, 96, 1030])
@pytest.mark.parametrize("x_off,x_pad,q_off,q_pad", [(0, 0, 0, 0), (1, 0, 1, 0), (3, 5, 3, 13), (1, 7, 2, 6),
                                                     (8, 0, 8, 0), (2, 2, 4, 2), (5, 0, 0, 3)])
def test_quantize_strides(dtype, K, x_off, x_pad, q_off, q_pad):
    """Rows that start anywhere in their units, where X's and Q's places agree and where not;
    what lies around them is neither read as theirs nor written."""
    rng = np.random.default_rng(K)
    T = 19
    wide = torch.full((T, x_off + K + x_pad), float("nan"), dtype=dtype)
    wide[:, x_off:x_off + K] = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).to(dtype)
    x = wide.to(DEV)[:, x_off:x_off + K]
    out = torch.full((T, q_off + K + q_pad), 77, dtype=torch.int8, device=DEV)
    q, s = dg.i8_quantize(x, out=out[:, q_off:q_off + K])
    quantized_exactly(x.cpu(), q, s)
    assert bool((out[:, :q_off] == 77).all()) and bool((out[:, q_off + K:] == 77).all())


# ---------------------------------------------------------------- products

def case(rng, T, N, K, experts=0, full=False):
    lead = (experts,) if experts else ()
    if full:                                     # the largest magnitudes there are
        x = rng.choice([-128, 127], (T, K)).astype(np.int8)
        q = rng.choice([-128, 127], lead + (N, K)).astype(np.int8)
    else:
        x = rng.integers(-128, 128, (T, K)).astype(np.int8)
        q = rng.integers(-128, 128, lead + (N, K)).astype(np.int8)
    sx = rng.uniform(0.5, 1.5, T).astype(np.float32) * 0.01
    sw = rng.uniform(0.5, 1.5, lead + (N,)).astype(np.float32) * 0.01
    return x, q, sx, sw


def run(x, q, sx, sw, **kw):
    to = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    return dg.i8_gemm(to(x), to(q), to(sw), x_scales=to(sx), **kw)


def equal_bits(got, x, q, sx, sw, offsets=None):
    want = ref.i8_bits(ref.integer_sums(x, q, offsets), sx, sw, got.dtype, offsets)
    rows = slice(0, x.shape[0]) if offsets is None else slice(offsets[0], offsets[-1])
    assert torch.equal(got.cpu()[rows], want[rows])


@pytest.mark.parametrize("T,N,K", [(1, 128, 128), (1, 1, 16), (2, 130, 48), (16, 128, 128), (17, 300, 256),
                                   (32, 128, 1024), (33, 129, 1040), (64, 256, 2048), (1, 1000, 4096),
                                   (5, 72, 8192), (65, 136, 640), (100, 1000, 272), (129, 128, 1152)])
@pytest.mark.parametrize("out", [BF, HF, F32])
def test_products(T, N, K, out):
    rng = np.random.default_rng(T * 1000 + N + K)
    c = case(rng, T, N, K)
    equal_bits(run(*c, out_dtype=out), *c)
    assert status() == 0


@pytest.mark.parametrize("T,N,K", [(200, 2000, 300), (700, 3000, 1100), (1500, 1016, 2064), (385, 5003, 160)])
def test_products_on_pairs(T, N, K):
    rng = np.random.default_rng(T)
    c = case(rng, T, N, K)
    equal_bits(run(*c, out_dtype=F32), *c)
    assert status() == 0


@pytest.mark.parametrize("T,N", [(3, 200), (70, 200), (260, 5000)])
@pytest.mark.parametrize("K", [1024, 1025, 2047, 2048, 2049, 4096, 16400])
def test_sums_are_exact_at_full_magnitude(T, N, K):
    """Sums past what fp32 holds: all products +-2^14 or near, some rows with one sign."""
    rng = np.random.default_rng(K + T)
    x, q, sx, sw = case(rng, T, N, K, full=True)
    x[0], q[0], q[1] = -128, -128, 127
    x[1] = 127
    x[2, ::2], x[2, 1::2] = 127, -128
    sx[:], sw[:] = 1.0, 1.0
    got = run(x, q, sx, sw, out_dtype=F32)
    equal_bits(got, x, q, sx, sw)


def test_the_longest_contraction():
    rng = np.random.default_rng(9)
    K = 131071
    x, q, sx, sw = case(rng, 3, 5, K, full=True)
    x[0], q[0] = -128, -128                     # 2^31 - 2^14
    sx[:], sw[:] = 1.0, 1.0
    equal_bits(run(x, q, sx, sw, out_dtype=F32), x, q, sx, sw)
    with pytest.raises(dg.GemmError):
        run(np.zeros((1, K + 1), np.int8), np.zeros((1, K + 1), np.int8), sx[:1], sw[:1])


@pytest.mark.parametrize("T,N,K", [(1500, 4096, 4096), (900, 8192, 2048), (2000, 8192, 1024), (100, 30000, 2048),
                                   (20, 40000, 4096)])
def test_many_tiles_a_cta(T, N, K):
    """Tiles whose output leaves while the next one's weights are on their way: the stages
    come round many times under load.  (Sums below 2^53 are exact in 64 bits.)"""
    gen = torch.Generator(device=DEV).manual_seed(K)
    x = torch.randint(-128, 128, (T, K), generator=gen, device=DEV, dtype=torch.int8)
    q = torch.randint(-128, 128, (N, K), generator=gen, device=DEV, dtype=torch.int8)
    want = (x.double() @ q.double().T).float()
    for _ in range(4):
        assert torch.equal(dg.i8_gemm(x, q, torch.ones(N, device=DEV), x_scales=torch.ones(T, device=DEV),
                                      out_dtype=F32), want)


COUNTS = [[1], [1, 0, 1, 1, 0, 0, 1], [3, 0, 31, 32, 33, 1], [0, 100, 129, 64, 127, 128, 0],
          [255, 256, 257, 0, 513, 40], [(7 * i) % 5 for i in range(100)], [0, 0, 0], [2] * 40, [64, 0, 300]]


@pytest.mark.parametrize("i", range(len(COUNTS)))
@pytest.mark.parametrize("K,N", [(200, 264), (1296, 136)])
def test_experts(i, K, N):
    rng = np.random.default_rng(i * 10 + K)
    counts = COUNTS[i]
    b = bounds_of(counts, 2)                    # rows of no expert before and after
    T = b[-1] + 3
    x, q, sx, sw = case(rng, T, N, K, len(counts))
    out = torch.full((T, N), 7.0, dtype=F32, device=DEV)
    got = run(x, q, sx, sw, offsets=offs(b), out=out)
    assert got is out
    equal_bits(got, x, q, sx, sw, b)
    assert bool((out[:2] == 7).all()) and bool((out[b[-1]:] == 7).all())
    assert status() == 0


@pytest.mark.parametrize("counts,N", [([700, 0, 900, 1000], 3000), ([300] * 8, 1000), ([2500, 3], 2056)])
@pytest.mark.parametrize("out", [BF, F32])
def test_experts_on_pairs(counts, N, out):
    rng = np.random.default_rng(N)
    b = bounds_of(counts)
    c = case(rng, b[-1], N, 272, len(counts))
    equal_bits(run(*c, offsets=offs(b), out_dtype=out), *c, b)


@pytest.mark.parametrize("K", [1, 3, 15, 17, 63, 65, 127, 130, 1001])
@pytest.mark.parametrize("experts", [0, 3])
def test_odd_contractions(K, experts):
    """Rows of weights that no 16-byte boundary divides are copied."""
    rng = np.random.default_rng(K)
    b = bounds_of([20, 0, 30]) if experts else None
    c = case(rng, 50, 70, K, experts)
    equal_bits(run(*c, out_dtype=F32, offsets=None if b is None else offs(b)), *c, b)


def test_strides_and_broadcast():
    rng = np.random.default_rng(5)
    b = bounds_of([30, 90, 0, 7])
    T, K, N = b[-1], 100, 80
    x, q, sx, sw = case(rng, T, N, K, 4)
    to = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    xp = to(np.pad(x, ((0, 0), (3, 5))))[:, 3:3 + K]
    outs = []
    for left, right in ((0, 12), (16, 12), (1, 0)):  # in place, in place, copied
        qp = to(np.pad(q, ((0, 0), (0, 0), (left, right))))[:, :, left:left + K]
        sp = to(np.pad(sw, ((0, 0), (2, 1))))[:, 2:2 + N]
        C = torch.full((T, N + 5), 3.0, dtype=HF, device=DEV)
        dg.i8_gemm(xp, qp, sp, x_scales=to(sx), offsets=offs(b), out=C[:, 2:2 + N])
        equal_bits(C[:, 2:2 + N], x, q, sx, sw, b)
        assert bool((C[:, :2] == 3).all()) and bool((C[:, 2 + N:] == 3).all())
        outs.append(C)
    q1, s1 = to(q[0]), to(sw[0])
    got = dg.i8_gemm(xp, q1.expand(4, N, K), s1.expand(4, N), x_scales=to(sx), offsets=offs(b))
    equal_bits(got, x, np.broadcast_to(q[0], q.shape), sx, np.broadcast_to(sw[0], sw.shape), b)


@pytest.mark.parametrize("epilogue", ["bias", "gelu_tanh", "bias_gelu_tanh", "bias_relu", "bias_gelu_erf"])
@pytest.mark.parametrize("per_expert", [False, True])
@pytest.mark.parametrize("T,N", [(40, 72), (900, 1500)])
def test_epilogues(epilogue, per_expert, T, N):
    """Before the activation the value is within 2^-22 of its parts' magnitudes (four fp32
    roundings: sum, two scales, bias); GELU's slope is below 1.13 and its own evaluation
    within 2^-20 of the value and its argument."""
    rng = np.random.default_rng(T)
    b = bounds_of([T // 4, 0, T - T // 4])
    x, q, sx, sw = case(rng, T, N, 160, 3)
    sw *= 0.05
    bias = rng.standard_normal((3, N) if per_expert else (N,)).astype(np.float32)
    use = bias if epilogue.startswith("bias") else None
    got = run(x, q, sx, sw, offsets=offs(b), out_dtype=F32, epilogue=epilogue,
              bias=None if use is None else torch.from_numpy(use).to(DEV))
    want, size = ref.i8(ref.integer_sums(x, q, b), sx, sw, b, use, epilogue)
    assert np.all(np.abs(experts_ref.f64(got) - want) <=
                  1.13 * 2.0 ** -22 * size + 2.0 ** -20 * (size + np.abs(want)))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,N,K", [(1, 300, 2048), (20, 130, 1001), (500, 1500, 320), (3, 64, 9000)])
def test_tokens_quantised_on_the_way(T, N, K, dtype):
    """The same bits as i8_quantize and the product of its integers."""
    rng = np.random.default_rng(K)
    x = torch.from_numpy((rng.standard_normal((T, K)) * 3).astype(np.float32)).to(dtype).to(DEV)
    _, q, _, sw = case(rng, 1, N, K)
    q, sw = torch.from_numpy(q).to(DEV), torch.from_numpy(sw).to(DEV)
    xi, sx = dg.i8_quantize(x)
    got = dg.i8_gemm(x, q, sw)
    assert got.dtype == dtype
    assert torch.equal(got, dg.i8_gemm(xi, q, sw, x_scales=sx, out_dtype=dtype))
    equal_bits(got, xi.cpu().numpy(), q.cpu().numpy(), sx.cpu().numpy(), sw.cpu().numpy())


def test_rows_do_not_mix_and_do_not_depend_on_their_number():
    """A NaN scale stays in its row (or channel); a row's bits are the same alone, in every
    form of the kernel, as an expert's row and in a batch."""
    rng = np.random.default_rng(6)
    T, N, K = 900, 1400, 2320
    x, q, sx, sw = case(rng, T, N, K)
    full = run(x, q, sx, sw, out_dtype=F32)
    for n in (1, 20, 50, 100, 300):
        assert torch.equal(run(x[:n], q, sx[:n], sw, out_dtype=F32), full[:n])
    lone = run(x[7:8], q[:100], sx[7:8], sw[:100], out_dtype=F32)
    assert torch.equal(lone, full[7:8, :100])
    b = [0, 5, 300, 300, 900]
    assert torch.equal(run(x, np.stack([q] * 4), sx, np.stack([sw] * 4), offsets=offs(b), out_dtype=F32), full)
    sx2, sw2 = sx.copy(), sw.copy()
    sx2[13], sw2[21] = np.nan, np.inf
    got = run(x, q, sx2, sw2, out_dtype=F32)
    keep = [i for i in range(T) if i != 13]
    cols = [i for i in range(N) if i != 21]
    assert torch.equal(got[keep][:, cols], full[keep][:, cols]) and torch.isnan(got[13]).all()


def test_empty():
    q, sw = torch.zeros((24, 64), dtype=torch.int8, device=DEV), torch.ones(24, device=DEV)
    x = torch.ones((5, 64), dtype=BF, device=DEV)
    assert dg.i8_gemm(x[:0], q, sw).shape == (0, 24)
    assert dg.i8_gemm(x, q[:0], sw[:0]).shape == (5, 0)
    bias = torch.randn(24, device=DEV)
    got = dg.i8_gemm(x[:, :0], q[:, :0], sw, bias=bias, out_dtype=F32)
    assert torch.equal(got, bias.expand(5, 24))
    C = torch.full((5, 24), 7.0, dtype=BF, device=DEV)
    dg.i8_gemm(x, q[None][:0], sw[None][:0], offsets=offs([0]), out=C)
    assert bool((C == 7).all())


@pytest.mark.parametrize("bad", [[0, 5, 3, 10], [0, 5, 8, 11], [-1, 5, 8, 10], [4, 3, 2, 1]])
def test_bad_offsets_are_reported_and_touch_nothing_else(bad):
    rng = np.random.default_rng(10)
    x, q, sx, sw = case(rng, 10, 40, 64, 3)
    C = torch.full((12, 40), 5.0, dtype=F32, device=DEV)
    run(x, q, sx, sw, offsets=offs(bad), out=C[:10])
    assert status() == dg.Status.ERR_INVALID_ARG
    assert status() == 0
    assert bool((C[10:] == 5).all())


@pytest.mark.parametrize("T,N,K", [(1, 300, 8192), (20, 3000, 1024), (50, 3000, 512), (100, 8000, 512),
                                   (700, 3000, 1100)])
def test_a_stalled_pipeline_reports_a_timeout_and_recovers(T, N, K):
    rng = np.random.default_rng(11)
    c = case(rng, T, N, K)
    good = run(*c, out_dtype=F32)
    dg.gemm_set_option(dg.Option.TIMEOUT_US, 2000)
    dg.gemm_set_option(dg.Option.TEST_STALL, 1)
    try:
        run(*c, out_dtype=F32)
        assert status() == dg.Status.ERR_TIMEOUT
    finally:
        dg.gemm_set_option(dg.Option.TEST_STALL, 0)
        dg.gemm_set_option(dg.Option.TIMEOUT_US, 1000000)
    assert status() == 0
    assert torch.equal(run(*c, out_dtype=F32), good)


@pytest.mark.parametrize("cap", [1, 5])
def test_the_cap_on_ctas(cap):
    rng = np.random.default_rng(13)
    for T, N, K in ((1, 1000, 4096), (600, 2000, 300)):
        c = case(rng, T, N, K)
        free = run(*c, out_dtype=F32)
        dg.gemm_set_option(dg.Option.MAX_CTAS, cap)
        try:
            assert torch.equal(run(*c, out_dtype=F32), free)
        finally:
            dg.gemm_set_option(dg.Option.MAX_CTAS, 0)


def test_graph_replay_side_stream_and_workspace():
    rng = np.random.default_rng(14)
    x, q, sx, sw = case(rng, 90, 200, 700)
    xd = torch.randn((90, 700), device=DEV).to(BF)
    qd, sd = torch.from_numpy(q).to(DEV), torch.from_numpy(sw).to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = dg.i8_gemm(xd, qd, sd)
    side.synchronize()
    assert torch.equal(y, dg.i8_gemm(xd, qd, sd))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dg.i8_gemm(xd, qd, sd)
    for _ in range(3):
        xd.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, dg.i8_gemm(xd, qd, sd))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    assert torch.equal(y, dg.i8_gemm(xd, qd, sd, workspace=ws))
    with pytest.raises(dg.GemmError):
        dg.i8_gemm(xd, qd, sd, workspace=ws[:1024])


def test_the_operators_together():
    """An expert layer in 8 bits: quantise, dispatch the integers, two products, combine;
    against the definition in 64 bits on the same integers."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    T, D, H, E, top = 70, 192, 320, 12, 3
    x = torch.randn((T, D), generator=gen, device=DEV).to(BF)
    w1 = torch.randn((E, H, D), generator=gen, device=DEV) * D ** -0.5
    w2 = torch.randn((E, D, H), generator=gen, device=DEV) * H ** -0.5
    q1, s1 = dg.i8_quantize(w1)
    q2, s2 = dg.i8_quantize(w2.to(BF))
    share, ids = torch.softmax(torch.randn((T, E), generator=gen, device=DEV), -1).topk(top)
    xi, xs = dg.i8_quantize(x)
    rows, offsets, slots, rs = dg.expert_dispatch(xi, ids, E, scales=xs)
    h = dg.i8_gemm(rows, q1, s1, x_scales=rs, offsets=offsets, epilogue="gelu_tanh")
    y2 = dg.i8_gemm(h, q2, s2, offsets=offsets)
    y = dg.expert_combine(y2, slots, share, out_dtype=F32)
    hi, hs = dg.i8_quantize(h)
    want = np.zeros((T, D))
    f = experts_ref.f64
    for t in range(T):
        for j in range(top):
            e, s = int(ids[t, j]), int(slots[t, j])
            a = (f(q1[e]) @ f(xi[t])) * f(xs[t]) * f(s1[e])
            g = experts_ref.gelu_tanh(a)
            assert np.all(np.abs(f(h[s]) - g) <= 2.0 ** -8 * np.abs(g) + 2.0 ** -19 * (np.abs(a) + np.abs(g)))
            b = (f(q2[e]) @ f(hi[s])) * f(hs[s]) * f(s2[e])
            assert np.all(np.abs(f(y2[s]) - b) <= (2.0 ** -8 + 2.0 ** -22) * np.abs(b))
            want[t] += f(share[t, j]) * f(y2[s])
    size = ref.combine(y2, slots.cpu().numpy(), share)[1]
    assert np.all(np.abs(f(y) - want) <= (top + 2) * 2.0 ** -24 * size)
    assert status() == 0


def test_debug_build_trips_no_check():
    """The same sources with device-side bounds checks, in every form of the kernel."""
    D = dg.debug_lib()
    rng = np.random.default_rng(21)
    st = torch.cuda.current_stream().cuda_stream
    for T, N, K, E in ((3, 200, 8192, 0), (20, 136, 272, 3), (60, 3000, 256, 0), (120, 8200, 256, 2),
                       (700, 3001, 272, 0), (900, 2056, 272, 3)):
        x, q, sx, sw = case(rng, T, N, K, E)
        b = bounds_of([T // 3, 0, T - T // 3 - 1][:E], 1) if E else None
        if E == 2:
            b = [1, T // 3, T]
        xd, qd, sxd, swd = (torch.from_numpy(v).to(DEV) for v in (x, q, sx, sw))
        o = offs(b) if E else None
        need = D.gemm_i8_workspace_size(3, max(E, 1), T, N, K, qd.data_ptr(), K, N * K)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        for out, code in ((BF, 0), (F32, 2)):
            C = torch.full((T, N), 7.0, dtype=out, device=DEV)
            assert D.gemm_i8(3, max(E, 1), T, N, K, xd.data_ptr(), K, sxd.data_ptr(), qd.data_ptr(), K,
                             N * K, swd.data_ptr(), N, C.data_ptr(), N, code,
                             o.data_ptr() if E else 0, 0, 0, 0, ws.data_ptr(), need, st) == 0
            assert D.gemm_check_device_status(st) == 0
            equal_bits(C, x, q, sx, sw, b)


@pytest.mark.parametrize("overlap", [0, 1])
def test_with_and_without_overlap(overlap):
    """GEMM_OPT_OVERLAP_COPY: the product starts while its tokens are prepared, or after; weights
    that are copied are waited for either way."""
    rng = np.random.default_rng(22)
    dg.gemm_set_option(dg.Option.OVERLAP_COPY, overlap)
    try:
        for T, N, K in ((40, 300, 1001), (900, 1500, 320)):
            c = case(rng, T, N, K)
            for _ in range(3):
                equal_bits(run(*c, out_dtype=F32), *c)
        x = torch.randn((3000, 64), device=DEV).to(BF)
        ids = torch.randint(0, 30, (3000, 3), device=DEV)
        rows, offsets, slots = dg.expert_dispatch(x, ids, 30)
        assert torch.equal(rows[slots.long()], x[:, None].expand(3000, 3, 64))
    finally:
        dg.gemm_set_option(dg.Option.OVERLAP_COPY, 0)


def test_two_streams_at_once():
    """Two products and two dispatches in flight together, each with its own workspace."""
    gen = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn((900, 1024), generator=gen, device=DEV).to(BF)
    q = torch.randint(-127, 128, (3000, 1024), generator=gen, device=DEV, dtype=torch.int8)
    s = torch.rand(3000, generator=gen, device=DEV)
    ids = torch.randint(0, 50, (900, 6), generator=gen, device=DEV)
    want, (rows, offsets, slots) = dg.i8_gemm(x, q, s), dg.expert_dispatch(x, ids, 50)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for st in streams:
            with torch.cuda.stream(st):
                got.append((dg.i8_gemm(x, q, s), *dg.expert_dispatch(x, ids, 50)))
    torch.cuda.synchronize()
    for y, r, o, sl in got:
        assert torch.equal(y, want) and torch.equal(r, rows) and torch.equal(o, offsets)
        assert torch.equal(sl, slots)
    assert status() == 0


def test_the_tokens_pass_does_not_count_as_a_wait():
    """A short bound on waits inside the product, and tokens whose preparation takes longer."""
    T, N, K = 400000, 128, 1024
    x = torch.ones((T, K), dtype=F32, device=DEV)
    q, s = torch.ones((N, K), dtype=torch.int8, device=DEV), torch.ones(N, device=DEV)
    dg.gemm_set_option(dg.Option.TIMEOUT_US, 100)
    try:
        for _ in range(3):
            y = dg.i8_gemm(x, q, s, out_dtype=BF)
            assert status() == 0
    finally:
        dg.gemm_set_option(dg.Option.TIMEOUT_US, 1000000)
    assert bool((y == 1024).all())


@pytest.mark.parametrize("T,N,K", [(1, 300, 8192), (32, 1000, 1024)])
def test_sums_that_never_arrive_report_a_timeout_and_recover(T, N, K):
    """CTAs that share a tile's contraction: the first one's wait for the others' sums runs out
    (four CTAs, then two)."""
    rng = np.random.default_rng(12)
    c = case(rng, T, N, K)
    good = run(*c, out_dtype=F32)
    dg.gemm_set_option(dg.Option.TIMEOUT_US, 2000)
    try:
        for _ in range(5):
            dg.gemm_set_option(dg.Option.TEST_STALL, 2)
            run(*c, out_dtype=F32)
            assert status() == dg.Status.ERR_TIMEOUT
    finally:
        dg.gemm_set_option(dg.Option.TEST_STALL, 0)
        dg.gemm_set_option(dg.Option.TIMEOUT_US, 1000000)
    assert status() == 0
    assert torch.equal(run(*c, out_dtype=F32), good)
    assert status() == 0


@pytest.mark.parametrize("T,N,splits", [(32, 1024, 4), (32, 9000, 2), (20, 10240, 1), (64, 10240, 1),
                                        (100, 10240, 1), (130, 10240, 1)])
def test_a_long_pass_beside_few_tiles_does_not_count_as_a_wait(T, N, splits):
    """Few long rows that start on odd elements: their quantisation takes some hundred
    microseconds on as many SMs, while the product's CTAs wait on the others.  Every form: a
    tile shared by four CTAs and by two, 32, 64 and 128 columns, pairs."""
    K = 131056
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, K + 2), generator=gen, device=DEV)[:, 1:-1]
    q = torch.randint(-127, 128, (N, K), generator=gen, device=DEV, dtype=torch.int8)
    s = torch.rand(N, generator=gen, device=DEV)
    xi, sx = dg.i8_quantize(x)
    want = dg.i8_gemm(xi, q, s, x_scales=sx, out_dtype=F32)
    dg.gemm_set_option(dg.Option.TIMEOUT_US, 50)
    try:
        for _ in range(3):
            y = dg.i8_gemm(x, q, s)
            assert status() == 0
            assert torch.equal(y, want)
    finally:
        dg.gemm_set_option(dg.Option.TIMEOUT_US, 1000000)


@pytest.mark.parametrize("epilogue", ["relu", "bias_relu", "gelu_tanh", "bias_gelu_erf"])
@pytest.mark.parametrize("T,N,K", [(5, 130, 2048), (40, 300, 160), (100, 9001, 64), (700, 3000, 96)])
def test_tokens_without_a_scale_are_nan_through_every_activation(epilogue, T, N, K):
    """A token with a NaN or an infinity has a NaN scale, and so has a channel: neither may
    come out as zeros.  All others are as in the call on their own."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn((T, K), generator=gen, device=DEV)
    q = torch.randint(-127, 128, (N, K), generator=gen, device=DEV, dtype=torch.int8)
    s = torch.rand(N, generator=gen, device=DEV) * 1e-3
    bias = torch.randn(N, generator=gen, device=DEV) if epilogue.startswith("bias") else None
    want = dg.i8_gemm(x, q, s, bias=bias, epilogue=epilogue)
    assert not torch.isnan(want).any()
    if epilogue.endswith("relu"):
        plain = dg.i8_gemm(x, q, s, bias=bias)
        assert torch.equal(want, plain.clamp(min=0)) and (plain < 0).any()
    x[1, K // 2], x[3, 0], s[7] = float("nan"), -float("inf"), float("nan")
    want[1], want[3], want[:, 7] = float("nan"), float("nan"), float("nan")
    for out in (F32, BF):
        got = dg.i8_gemm(x, q, s, bias=bias, epilogue=epilogue, out_dtype=out)
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(-9.0), want.to(out).nan_to_num(-9.0))


def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("T", [1, 33])
def test_the_example_answers_in_8_bits(T):
    """Against its own steps, token by token and expert by expert without a dispatch: products
    have the same bits alone, and the sum of `top` terms is off by an fp32 rounding for each."""
    mod = example()
    gen = torch.Generator(device=DEV).manual_seed(T)
    D, H, E, top = 256, 512, 8, 2
    x = torch.randn((T, D), generator=gen, device=DEV).to(BF)
    w1 = dg.i8_quantize(torch.randn((E, H, D), generator=gen, device=DEV) * D ** -0.5)
    w2 = dg.i8_quantize(torch.randn((E, D, H), generator=gen, device=DEV) * H ** -0.5)
    expert, share = mod.route(x, torch.randn((D, E), generator=gen, device=DEV), top)
    got = mod.answer_in_8_bits(x, w1, w2, (expert, share))
    assert got.dtype == F32 and got.shape == (T, D)
    for t in range(T):
        want, size = torch.zeros(D, dtype=torch.float64, device=DEV), 0.0
        for j in range(top):
            e = int(expert[t, j])
            h = dg.i8_gemm(x[t:t + 1], w1[0][e], w1[1][e], epilogue="gelu_tanh")
            y = dg.i8_gemm(h, w2[0][e], w2[1][e])[0].double() * share[t, j].double()
            want, size = want + y, size + y.abs()
        assert bool(((got[t].double() - want).abs() <= (top + 1) * 2.0 ** -24 * size).all())
    assert status() == 0


@pytest.mark.parametrize("T", [20, 2500])
def test_a_layer_in_8_bits_captured_whole(T):
    """Quantise, dispatch (one launch, then two), two products and combine in one graph, replayed
    on new tokens and routes: the bits of the calls one by one."""
    mod = example()
    gen = torch.Generator(device=DEV).manual_seed(T)
    D, H, E, top = 320, 640, 12, 3
    x = torch.randn((T, D), generator=gen, device=DEV).to(BF)
    w1 = dg.i8_quantize(torch.randn((E, H, D), generator=gen, device=DEV) * D ** -0.5)
    w2 = dg.i8_quantize(torch.randn((E, D, H), generator=gen, device=DEV) * H ** -0.5)
    expert, share = mod.route(x, torch.randn((D, E), generator=gen, device=DEV), top)
    mod.answer_in_8_bits(x, w1, w2, (expert, share))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mod.answer_in_8_bits(x, w1, w2, (expert, share))
    for _ in range(3):
        x.copy_(torch.randn((T, D), generator=gen, device=DEV))
        expert.copy_(torch.randint(0, E, (T, top), generator=gen, device=DEV))
        share.copy_(torch.rand((T, top), generator=gen, device=DEV))
        for _ in range(3):
            graph.replay()
        assert torch.equal(y, mod.answer_in_8_bits(x, w1, w2, (expert, share)))
    assert status() == 0
