"""Tokens to their experts' rows and back, and the gradient of that, on the GPU against
plain 64-bit references."""
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


def route(rng, T, top, E, drop=0.0, skew=0.0, twice=False):
    """[T, top] ids: distinct per token unless `twice`, -1 where dropped."""
    p = 1.0 / np.arange(1, E + 1) ** skew
    score = np.log(p) + rng.gumbel(size=(T, E))
    ids = np.argsort(-score, axis=1)[:, :top] if not twice else rng.integers(0, E, (T, top))
    ids = ids.astype(np.int64)
    if drop:
        ids[rng.random((T, top)) < drop] = -1
    return ids


def values(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def same(a, b):
    return torch.equal(a.cpu(), b.cpu())


# (tokens, choices, experts, features, dropped share)
SIZES = [(1, 1, 1, 1, 0.0), (1, 8, 8, 2048, 0.0), (5, 2, 3, 7, 0.5), (48, 4, 64, 2048, 0.0),
         (33, 3, 100, 130, 0.2), (152, 2, 7, 64, 0.0), (153, 6, 160, 1001, 0.1), (1000, 5, 33, 24, 0.0),
         (683, 6, 40, 96, 0.0), (700, 6, 40, 100, 0.1), (4096, 2, 256, 72, 0.0), (5000, 8, 64, 40, 0.1),
         (20000, 1, 1, 16, 0.0), (9001, 4, 1500, 8, 0.3), (3000, 2, 4096, 10, 0.0)]


@pytest.mark.parametrize("T,top,E,K,drop", SIZES)
@pytest.mark.parametrize("kind", ["i64", "i32"])
def test_dispatch(T, top, E, K, drop, kind):
    rng = np.random.default_rng(T * 7 + top)
    ids = route(rng, T, top, E, drop, skew=0.7)
    offsets, slots = ref.places(ids, E)
    P = int(offsets[-1])
    x = values(rng, (T, K), BF if kind == "i64" else F32).to(DEV)
    out = torch.full((T * top, K), 7.0, dtype=x.dtype, device=DEV)
    di = torch.from_numpy(ids).to(DEV, torch.int64 if kind == "i64" else torch.int32)
    rows, off, sl = dg.expert_dispatch(x, di, E, out=out)
    assert rows is out and off.dtype == sl.dtype == torch.int32
    assert np.array_equal(off.cpu().numpy(), offsets)
    assert np.array_equal(sl.cpu().numpy(), slots)
    want = torch.full((T * top, K), 7.0, dtype=x.dtype)
    t, j = np.nonzero(slots >= 0)
    want[torch.from_numpy(slots[t, j])] = x.cpu()[torch.from_numpy(t)]
    assert same(rows, want) and P == len(t)
    assert status() == 0


@pytest.mark.parametrize("dtype", [torch.int8, BF, F32])
@pytest.mark.parametrize("pad,shift", [(0, 0), (16, 0), (8, 4), (3, 1)])
def test_dispatch_strides_types_and_scales(dtype, pad, shift):
    """Rows and ids inside wider ones, from aligned to odd addresses; the scales go along."""
    rng = np.random.default_rng(pad * 5 + shift)
    T, top, E, K = 77, 3, 12, 112
    ids = route(rng, T, top, E, 0.2, twice=True)
    offsets, slots = ref.places(ids, E)
    wide = (values(rng, (T, K + pad + shift), F32) * 40).to(dtype).to(DEV)
    x = wide[:, shift:shift + K]
    out = torch.zeros((T * top, K + pad + shift), dtype=dtype, device=DEV)[:, shift:shift + K]
    scales = values(rng, (T,), F32).to(DEV)
    di = torch.from_numpy(np.pad(ids, ((0, 0), (1, 2)), constant_values=5)).to(DEV)[:, 1:1 + top]
    rows, off, sl, rs = dg.expert_dispatch(x, di, E, scales=scales, out=out,
                                           out_scales=torch.zeros(T * top, device=DEV))
    assert np.array_equal(off.cpu().numpy(), offsets) and np.array_equal(sl.cpu().numpy(), slots)
    t, j = np.nonzero(slots >= 0)
    want, ws = torch.zeros((T * top, K), dtype=dtype), torch.zeros(T * top)
    want[torch.from_numpy(slots[t, j])] = x.cpu()[torch.from_numpy(t)]
    ws[torch.from_numpy(slots[t, j])] = scales.cpu()[torch.from_numpy(t)]
    assert same(rows, want) and same(rs, ws)


@pytest.mark.parametrize("dtype", [torch.int8, HF, F32])
@pytest.mark.parametrize("T,top,K,x_shift,shift,pad", [
    (40, 3, 3, 0, 0, 0), (6000, 2, 15, 1, 0, 0), (77, 4, 17, 0, 3, 5), (6000, 3, 33, 2, 1, 0),
    (500, 2, 255, 0, 0, 0), (400, 3, 2047, 3, 0, 2), (300, 2, 2049, 0, 0, 0), (31, 40, 130, 1, 2, 3),
    (400, 2, 20001, 1, 3, 0), (155, 2, 16390, 0, 2, 0), (90, 2, 1026, 0, 0, 0)])
def test_dispatch_to_rows_on_any_address(T, top, K, x_shift, shift, pad, dtype):
    """Tokens and rows that start anywhere in their 16 bytes, several rounds a block and several
    rounds a row among them; what lies beside the rows stays."""
    rng = np.random.default_rng(K + T)
    ids = route(rng, T, top, 9, 0.1, twice=True)
    offsets, slots = ref.places(ids, 9)
    x = torch.from_numpy(rng.integers(-100, 100, (T, x_shift + K))).to(DEV, dtype)[:, x_shift:]
    wide = torch.full((T * top, shift + K + pad), 101, dtype=dtype, device=DEV)
    scales = values(rng, (T,), F32).to(DEV)
    _, off, sl, rs = dg.expert_dispatch(x, torch.from_numpy(ids).to(DEV), 9, scales=scales,
                                        out=wide[:, shift:shift + K])
    assert np.array_equal(off.cpu().numpy(), offsets) and np.array_equal(sl.cpu().numpy(), slots)
    t, j = (torch.from_numpy(v).to(DEV) for v in np.nonzero(slots >= 0))
    want = torch.full((T * top, K), 101, dtype=dtype, device=DEV)
    want[sl[t, j].long()] = x[t]
    assert torch.equal(wide[:, shift:shift + K], want)
    assert bool((wide[:, :shift] == 101).all()) and bool((wide[:, shift + K:] == 101).all())
    assert torch.equal(rs[sl[t, j].long()], scales[t]) and status() == 0


def test_longest_rows():
    """Rows as long as extents may be, and odd: columns counted in steps come close to 2^31."""
    K = 2 ** 31 - 4097
    x = torch.randint(-100, 100, (1, K), dtype=torch.int8, device=DEV)
    ids = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    rows, off, slots = dg.expert_dispatch(x, ids, 1)
    assert off.tolist() == [0, 1] and slots.tolist() == [[0]] and torch.equal(rows, x)
    del x
    wide = rows.to(HF)
    assert torch.equal(dg.expert_combine(wide, slots), wide)
    assert status() == 0


def test_dispatch_nothing_and_all_dropped():
    x = torch.zeros((0, 8), dtype=BF, device=DEV)
    rows, off, sl = dg.expert_dispatch(x, torch.zeros((0, 2), dtype=torch.int32, device=DEV), 5)
    assert rows.shape == (0, 8) and off.tolist() == [0] * 6 and sl.shape == (0, 2)
    x = torch.zeros((4, 8), dtype=BF, device=DEV)
    rows, off, sl = dg.expert_dispatch(x, torch.zeros((4, 0), dtype=torch.int32, device=DEV), 3)
    assert rows.shape == (0, 8) and off.tolist() == [0] * 4
    ids = torch.full((4, 2), -1, dtype=torch.int64, device=DEV)
    out = torch.full((8, 8), 3.0, dtype=BF, device=DEV)
    rows, off, sl = dg.expert_dispatch(x, ids, 3, out=out)
    assert off.tolist() == [0] * 4 and bool((sl == -1).all()) and bool((rows == 3).all())
    rows, off, sl = dg.expert_dispatch(x, ids, 0)
    assert off.tolist() == [0] and bool((sl == -1).all())
    rows, off, sl = dg.expert_dispatch(x[:, :0], ids + 1, 3)
    assert off.tolist() == [0, 8, 8, 8] and sl.flatten().tolist() == list(range(8))
    assert status() == 0


@pytest.mark.parametrize("T", [40, 6000])
def test_ids_past_the_experts_are_reported_and_get_no_row(T):
    rng = np.random.default_rng(3)
    E, top = 9, 2
    ids = route(rng, T, top, E)
    ids[T // 2, 1], ids[3, 0], ids[T - 1, 0] = 9, 1 << 40, -(1 << 40)
    offsets, slots = ref.places(ids, E)
    x = values(rng, (T, 32), HF).to(DEV)
    rows, off, sl = dg.expert_dispatch(x, torch.from_numpy(ids).to(DEV), E)
    assert status() == dg.Status.ERR_INVALID_ARG
    assert status() == 0
    assert np.array_equal(off.cpu().numpy(), offsets) and np.array_equal(sl.cpu().numpy(), slots)


def test_dispatch_repeats_and_keeps_to_the_cap():
    rng = np.random.default_rng(4)
    ids = torch.from_numpy(route(rng, 7000, 4, 50, skew=1.0)).to(DEV)
    x = values(rng, (7000, 64), BF).to(DEV)
    first = dg.expert_dispatch(x, ids, 50)
    for cap in (0, 1, 7):
        dg.gemm_set_option(dg.Option.MAX_CTAS, cap)
        try:
            again = dg.expert_dispatch(x, ids, 50)
        finally:
            dg.gemm_set_option(dg.Option.MAX_CTAS, 0)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("T,top,E,K,drop", [s for s in SIZES if s[0] <= 1000])
@pytest.mark.parametrize("dtype,wdt,out", [(BF, F32, BF), (HF, HF, F32), (F32, BF, F32), (BF, None, F32)])
def test_combine(T, top, E, K, drop, dtype, wdt, out):
    """Within top + 1 roundings of fp32 of the magnitudes (a product's is fused with its
    sum), and half a step of the result's type."""
    rng = np.random.default_rng(T + top)
    _, slots = ref.places(route(rng, T, top, E, drop), E)
    rows = values(rng, (T * top, K), dtype)
    w = None if wdt is None else values(rng, (T, top), wdt)
    got = dg.expert_combine(rows.to(DEV), torch.from_numpy(slots).to(DEV, torch.int32),
                            None if w is None else w.to(DEV), out_dtype=out)
    want, size = ref.combine(rows, slots, w)
    assert got.dtype == out
    err = np.abs(experts_ref.f64(got) - want)
    fp32 = (top + 1) * 2.0 ** -24 * size
    assert np.all(err <= fp32 + HALF_STEP[out] * (np.abs(want) + fp32) + TINIEST[out])
    assert status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
def test_combine_strides(dtype, shift):
    """Small integers, exact in any order; rows, weights and result inside wider ones."""
    rng = np.random.default_rng(shift)
    T, top, E, K = 50, 3, 9, 88
    _, slots = ref.places(route(rng, T, top, E, 0.3), E)
    rows = experts_ref.ints(rng, (T * top, K + 16), dtype=dtype).to(DEV)[:, shift:shift + K]
    w = experts_ref.ints(rng, (T, top + 2), dtype=F32).to(DEV)[:, 1:1 + top]
    out = torch.full((T, K + 9), 5.0, dtype=dtype, device=DEV)
    y = dg.expert_combine(rows, torch.from_numpy(slots).to(DEV, torch.int32), w, out=out[:, shift:shift + K])
    assert np.array_equal(experts_ref.f64(y), ref.combine(rows, slots, w)[0])
    assert bool((out[:, :shift] == 5).all()) and bool((out[:, shift + K:] == 5).all())


def test_combine_skips_pairs_without_a_row():
    """What a dropped pair's weight or the rows past the last hold never enters a sum."""
    rows = torch.full((6, 16), float("nan"), dtype=BF, device=DEV)
    rows[:2] = 1.0
    slots = torch.tensor([[0, -1], [-1, -1], [-7, 1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[2.0, float("nan")], [float("inf"), 1.0], [float("nan"), 3.0]], device=DEV)
    y = dg.expert_combine(rows, slots, w)
    assert y[:, 0].tolist() == [2.0, 0.0, 3.0] and bool((y == y[:, :1]).all())
    d_rows, d_w = dg.expert_combine_grad(torch.ones((3, 16), dtype=BF, device=DEV), slots, w,
                                         rows=rows, out=torch.full_like(rows, 9.0))
    assert d_w.tolist() == [[16.0, 0.0], [0.0, 0.0], [0.0, 16.0]]
    assert d_rows[:, 0].tolist() == [2.0, 3.0, 9.0, 9.0, 9.0, 9.0]


def test_slots_past_the_rows_are_reported_and_add_nothing():
    rows = torch.ones((4, 24), dtype=HF, device=DEV)
    slots = torch.tensor([[0, 4], [2147483647, 3]], dtype=torch.int32, device=DEV)
    assert dg.expert_combine(rows, slots)[:, 5].tolist() == [1.0, 1.0]
    assert status() == dg.Status.ERR_INVALID_ARG
    d_rows, d_w = dg.expert_combine_grad(torch.ones((2, 24), dtype=HF, device=DEV), slots,
                                         rows=rows, out=torch.zeros_like(rows))
    assert status() == dg.Status.ERR_INVALID_ARG
    assert d_w.tolist() == [[24.0, 0.0], [0.0, 24.0]] and d_rows[:, 0].tolist() == [1, 0, 0, 1]
    assert status() == 0


def test_combine_nothing():
    rows = torch.ones((0, 8), dtype=BF, device=DEV)
    slots = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    assert bool((dg.expert_combine(rows, slots) == 0).all())
    none = torch.zeros((3, 0), dtype=torch.int32, device=DEV)
    assert bool((dg.expert_combine(torch.ones((2, 8), dtype=BF, device=DEV), none) == 0).all())
    assert dg.expert_combine(rows, slots[:0]).shape == (0, 8)
    d_rows, d_w = dg.expert_combine_grad(torch.ones((3, 8), dtype=BF, device=DEV), slots, rows=rows)
    assert d_rows.shape == (0, 8) and bool((d_w == 0).all())
    d_rows, d_w = dg.expert_combine_grad(torch.ones((3, 0), dtype=BF, device=DEV), slots.clamp(min=0),
                                         rows=torch.ones((6, 0), dtype=BF, device=DEV))
    assert bool((d_w == 0).all())
    assert status() == 0


# ---------------------------------------------------------------- its gradient

@pytest.mark.parametrize("T,top,E,K,drop", [s for s in SIZES if s[0] <= 1000] + [(40, 9, 20, 300, 0.1),
                                                                              (17, 17, 30, 2000, 0.0)])
@pytest.mark.parametrize("dtype,wdt", [(BF, F32), (HF, HF), (F32, F32), (BF, None)])
def test_combine_grad(T, top, E, K, drop, dtype, wdt):
    """d_rows: one fp32 product and a rounding to its type.  d_weights: a sum of K products
    in some order, within K roundings of fp32 of the magnitudes, and a rounding."""
    rng = np.random.default_rng(T * 3 + top)
    _, slots = ref.places(route(rng, T, top, E, drop), E)
    dy, rows = values(rng, (T, K), dtype), values(rng, (T * top, K), dtype)
    w = None if wdt is None else values(rng, (T, top), wdt)
    like = torch.full((T * top, K), 4.0, dtype=dtype)
    d_rows, d_w = dg.expert_combine_grad(dy.to(DEV), torch.from_numpy(slots).to(DEV, torch.int32),
                                         None if w is None else w.to(DEV), rows=rows.to(DEV),
                                         out=like.to(DEV))
    want, want_w, size = ref.combine_grad(dy, slots, w, rows, like)
    err = np.abs(experts_ref.f64(d_rows) - want)
    assert np.all(err <= (HALF_STEP[dtype] + 2.0 ** -23) * np.abs(want) + TINIEST[dtype])
    kind = F32 if wdt is None else wdt
    assert d_w.dtype == kind
    fp32 = K * 2.0 ** -24 * size
    assert np.all(np.abs(experts_ref.f64(d_w) - want_w) <=
                  fp32 + HALF_STEP[kind] * (np.abs(want_w) + fp32) + TINIEST[kind])
    only, none = dg.expert_combine_grad(dy.to(DEV), torch.from_numpy(slots).to(DEV, torch.int32),
                                        None if w is None else w.to(DEV), out=like.to(DEV))
    assert none is None and torch.equal(only, d_rows)
    assert status() == 0


@pytest.mark.parametrize("shift", [0, 1, 2, 8])
def test_combine_grad_strides(shift):
    rng = np.random.default_rng(shift + 20)
    T, top, E, K = 41, 5, 9, 72
    _, slots = ref.places(route(rng, T, top, E, 0.3), E)
    dy = experts_ref.ints(rng, (T, K + 8), dtype=HF).to(DEV)[:, shift:shift + K]
    rows = experts_ref.ints(rng, (T * top, K + 11), dtype=HF).to(DEV)[:, shift:shift + K]
    w = experts_ref.ints(rng, (T, top), dtype=F32)
    out = torch.full((T * top, K + 10), 5.0, dtype=HF, device=DEV)
    d_rows, d_w = dg.expert_combine_grad(dy, torch.from_numpy(slots).to(DEV, torch.int32), w.to(DEV),
                                         rows=rows, out=out[:, shift:shift + K])
    want, want_w, _ = ref.combine_grad(dy, slots, w, rows, torch.full((T * top, K), 5.0))
    assert np.array_equal(experts_ref.f64(d_rows), want)
    assert np.array_equal(experts_ref.f64(d_w), want_w)
    assert bool((out[:, :shift] == 5).all()) and bool((out[:, shift + K:] == 5).all())


@pytest.mark.parametrize("dtype", [HF, F32])
@pytest.mark.parametrize("T,top,K,shift", [(9, 3, 8, 1), (33, 6, 9, 0), (7, 9, 15, 3), (40, 2, 23, 5),
                                           (300, 5, 130, 0), (5, 4, 2047, 1), (6, 8, 2049, 0),
                                           (3, 2, 2056, 7), (4, 6, 4099, 2)])
def test_rows_on_any_address(T, top, K, shift, dtype):
    """Rows, results and gradients that start anywhere in their 16 bytes, the matrix's first and
    last row included; what lies beside them is neither used nor written."""
    rng = np.random.default_rng(K + shift)
    _, slots = ref.places(route(rng, T, top, 12, 0.2), 12)
    where = torch.from_numpy(slots).to(DEV, torch.int32)

    def inside(rows, pitch):
        wide = torch.full((rows, pitch), float("nan"), dtype=dtype, device=DEV)
        view = wide.view(-1)[shift:shift + (rows - 1) * pitch + K].as_strided((rows, K), (pitch, 1))
        view.copy_(experts_ref.ints(rng, (rows, K), dtype=dtype))
        return view

    rows, dy = inside(T * top, K + shift), inside(T, K + shift + 3)
    w = experts_ref.ints(rng, (T, top), dtype=F32)
    for kind in {dtype, F32}:
        wide = torch.full((T, K + shift + 1), 5.0, dtype=kind, device=DEV)
        dg.expert_combine(rows, where, w.to(DEV), out=wide[:, shift:shift + K])
        want, _ = ref.combine(rows, slots, w)
        assert np.array_equal(experts_ref.f64(wide[:, shift:shift + K]), want)
        assert bool((wide[:, :shift] == 5).all()) and bool((wide[:, shift + K:] == 5).all())
    for pitch in (K + shift, K + shift + 1):
        wide = torch.full((T * top, pitch), 5.0, dtype=dtype, device=DEV)
        d_rows, d_w = dg.expert_combine_grad(dy, where, w.to(DEV), rows=rows,
                                             out=wide[:, shift:shift + K])
        want, want_w, _ = ref.combine_grad(dy, slots, w, rows, torch.full((T * top, K), 5.0))
        assert np.array_equal(experts_ref.f64(d_rows), want)
        assert np.array_equal(experts_ref.f64(d_w), want_w)
        assert bool((wide[:, :shift] == 5).all()) and bool((wide[:, shift + K:] == 5).all())
    assert status() == 0


def test_gradients_against_differences():
    """L = <g, combine(dispatch(x) * a, w)> is linear in x and in w: on small integers a
    difference quotient is its slope exactly."""
    rng = np.random.default_rng(8)
    T, top, E, K = 12, 3, 5, 40
    ids = torch.from_numpy(route(rng, T, top, E, 0.2)).to(DEV)
    x, g = (experts_ref.ints(rng, (T, K), dtype=F32).to(DEV) for _ in range(2))
    w = experts_ref.ints(rng, (T, top), dtype=F32).to(DEV)
    a = experts_ref.ints(rng, (T * top, K), dtype=F32).to(DEV)

    def loss(x, w):
        rows, _, slots = dg.expert_dispatch(x, ids, E)
        rows = torch.where(torch.arange(T * top, device=DEV)[:, None] <= slots.max(), rows * a, 0.0)
        return float((dg.expert_combine(rows, slots, w).double() * g.double()).sum()), rows, slots

    base, rows, slots = loss(x, w)
    d_rows, d_w = dg.expert_combine_grad(g, slots, w, rows=rows, out=torch.zeros_like(rows))
    d_x = dg.expert_combine(d_rows * a, slots)
    for _ in range(40):
        t, k, j = int(rng.integers(T)), int(rng.integers(K)), int(rng.integers(top))
        x2, w2 = x.clone(), w.clone()
        x2[t, k] += 1
        w2[t, j] += 1
        assert loss(x2, w)[0] - base == float(d_x[t, k])
        assert loss(x, w2)[0] - base == float(d_w[t, j])


def test_rows_past_32_bits_of_elements():
    """A buffer of 2.4e9 elements: rows whose element offsets pass 2^31."""
    T, K = 73000, 32768
    x = torch.empty((T, K), dtype=torch.int8, device=DEV)
    x[:] = torch.arange(T, device=DEV, dtype=torch.int32)[:, None].to(torch.int8)
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    ids[:5] = 1                               # the first five go to the end
    rows, off, slots = dg.expert_dispatch(x, ids, 2)
    assert off.tolist() == [0, T - 5, T] and slots[:6, 0].tolist() == [T - 5, T - 4, T - 3, T - 2, T - 1, 0]
    want = torch.cat([x[5:, 0], x[:5, 0]])
    assert torch.equal(rows[:, 0], want) and torch.equal(rows[:, -1], want)
    del rows, x
    big = torch.empty((T, K), dtype=BF, device=DEV)
    big[-3:] = 2.0
    got = dg.expert_combine(big, torch.tensor([[T - 1, T - 3]], dtype=torch.int32, device=DEV))
    assert bool((got == 4).all())
    d_rows, _ = dg.expert_combine_grad(torch.full((1, K), 6.0, dtype=BF, device=DEV),
                                       torch.tensor([[T - 2, T - 3]], dtype=torch.int32, device=DEV),
                                       out=big)
    assert bool((big[-3:-1] == 6).all()) and bool((big[-1] == 2).all())
    assert status() == 0


def test_side_stream_graph_and_replay():
    """Captured once (both forms of the sort), replayed on new inputs."""
    rng = np.random.default_rng(12)
    for T in (100, 3000):
        top, E, K = 3, 40, 128
        ids = torch.from_numpy(route(rng, T, top, E, 0.1)).to(DEV)
        x = values(rng, (T, K), BF).to(DEV)
        w = values(rng, (T, top), F32).to(DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                rows, off, slots = dg.expert_dispatch(x, ids, E)
                y = dg.expert_combine(rows, slots, w)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rows, off, slots = dg.expert_dispatch(x, ids, E)
            y = dg.expert_combine(rows, slots, w)
            d_rows, d_w = dg.expert_combine_grad(y, slots, w, rows=rows)
        for _ in range(2):
            new = route(rng, T, top, E, 0.2)
            ids.copy_(torch.from_numpy(new))
            x.copy_(values(rng, (T, K), BF))
            graph.replay()
            torch.cuda.synchronize()
            offsets, want = ref.places(new, E)
            assert np.array_equal(slots.cpu().numpy(), want)
            again = dg.expert_combine(*dg.expert_dispatch(x, ids, E)[::2], w)
            assert torch.equal(y, again)
            assert torch.equal(d_w, dg.expert_combine_grad(y, slots, w, rows=rows)[1])
    assert status() == 0
