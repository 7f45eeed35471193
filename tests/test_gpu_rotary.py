"""GPU parity of the rotary positions, with and without the cache's write.

Tolerance of a turned element a cos - b sin (amplitude m, s = m (|a| + |b|)), in units of s: the fraction of a
turn rounded to 24 bits is off by 2^-25 of at most half a turn, pi 2^-24 as an angle (2^-22.3); sincospif by at
most 2^-23; products with m, with a and b, and their sum by four roundings of 2^-24; the frequencies' 53 bits times
positions up to 2^31 by at most 2^-22 as an angle.  Together below 2^-20 s; then the rounding to fp16, half a step:
2^-11 of the value, 2^-25 below its normal range.  What is copied is equal bit by bit.
"""
import numpy as np
import pytest

from oracle import mixers, serving

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KINDS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def make_plan(R, base=1e4, scaling="none", factor=1.0, original=2048.0, **kw):
    import ternary_hadamard_rotated_gb300 as tb

    plan = torch.full((tb.tb_rotary_plan_size(R),), 0xAB, dtype=torch.uint8, device="cuda")
    tb.tb_rotary_plan(plan, R, base=base, scaling=KINDS[scaling], factor=factor, original=original, **kw)
    f, amp = serving.rotary_freqs(R, base, scaling, factor, original)
    return plan, f, kw.get("amplitude") or amp


def close(got, want, size):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -20 * size
    assert (np.abs(got - want) <= tol).all(), np.nanmax(np.abs(got - want) / tol)


def bits(t):
    return t.cpu().numpy().view(np.uint16)


def inputs(rng, T, Hq, Hk, D, extra=0):
    """q, k, v as slices of one projection (host and device)."""
    w = (Hq + 2 * Hk) * D + extra
    x = torch.from_numpy(rng.standard_normal((T, w)).astype(np.float16)).cuda()
    cut = [0, Hq * D, (Hq + Hk) * D, (Hq + 2 * Hk) * D]
    return [x[:, a:b].unflatten(1, (-1, D)) for a, b in zip(cut, cut[1:])]


@pytest.mark.parametrize("T,Hq,Hk,D,R,pairs,inverse,scaling,factor", [
    (1, 24, 4, 256, 64, False, False, "none", 1.0), (1, 1, 1, 8, 2, True, False, "none", 1.0), (5, 3, 1, 64, 64, True, True, "linear", 4.0),
    (37, 4, 2, 128, 128, False, True, "base", 8.0), (33, 2, 1, 80, 80, False, False, "parts", 32.0), (64, 6, 2, 96, 48, True, False, "parts", 2.0),
    (9, 2, 2, 72, 34, False, False, "none", 1.0), (9, 2, 2, 72, 34, True, False, "linear", 2.5), (3, 2, 0, 1024, 1024, False, False, "none", 1.0),
    (700, 2, 1, 64, 16, False, False, "none", 1.0), (11, 1, 3, 16, 10, False, True, "base", 0.5), (2, 130, 7, 40, 24, True, False, "none", 1.0)])
def test_rotary_matches(T, Hq, Hk, D, R, pairs, inverse, scaling, factor):
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(T * 1000 + D)
    plan, f, amp = make_plan(R, 1e4, scaling, factor)
    q, k, _ = inputs(rng, T, Hq, Hk, D, 8)
    pos = rng.integers(0, 262144, T)
    pos[: 4] = [0, 2 ** 31 - 1, -2 ** 31, -7][: T] if T < 4 else [0, 2 ** 31 - 1, -2 ** 31, -7]
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    qn, kn = q.cpu().numpy(), k.cpu().numpy()
    qo, ko = torch.full((T + 1, Hq, D), 7.0, dtype=torch.float16, device="cuda"), torch.full((T + 1, max(Hk, 1), D), 7.0, dtype=torch.float16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tb.tb_rotary(q, k if Hk else None, p, plan, R, int(pairs), qo[:T], ko[:T] if Hk else None, inverse=inverse, dev_status=st)
    assert np.array_equal(bits(q), qn.view(np.uint16))
    for x, y in ((qn, qo),) + (((kn, ko),) if Hk else ()):
        want, size = serving.rotary(x, pos, f, amp, R, pairs, inverse)
        close(y[:T].cpu().numpy(), want, size)
        assert np.array_equal(bits(y[:T])[..., R:], x.view(np.uint16)[..., R:])
        assert (y[T] == 7).all()
    assert int(st) == 0
    first = qo.clone(), ko.clone()
    tb.tb_rotary(q, k if Hk else None, p, plan, R, int(pairs), q, k if Hk else None, inverse=inverse)  # in place: the same bits
    assert torch.equal(q, first[0][:T]) and (not Hk or torch.equal(k, first[1][:T]))


@pytest.mark.parametrize("T,Hq,Hk,D,R,page,pairs,k_out", [
    (1, 24, 4, 256, 64, 64, False, None), (64, 8, 2, 128, 128, 16, False, "own"), (130, 3, 1, 64, 34, 32, True, "k"), (77, 2, 2, 80, 20, 256, True, None),
    (41, 4, 4, 8, 8, 128, False, "own")])
def test_rotary_cache_write_is_rotary_and_cache_write(T, Hq, Hk, D, R, page, pairs, k_out):
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(T + D)
    plan, f, amp = make_plan(R, 5e5, "parts", 4.0)
    q, k, v = inputs(rng, T, Hq, Hk, D)
    pos = torch.from_numpy(rng.integers(0, 100000, T).astype(np.int32)).cuda()
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.from_numpy(rng.standard_normal((pages, Hk, page, D)).astype(np.float16)).cuda() for _ in range(2))
    wq, wk = torch.empty_like(q), torch.empty_like(k)
    tb.tb_rotary(q, k, pos, plan, R, int(pairs), wq, wk)
    want = mixers.cache_write(wk.cpu().numpy(), v.cpu().numpy(), slots, kc.cpu().numpy(), vc.cpu().numpy())
    qo = torch.empty_like(q)
    ko = {None: None, "own": torch.zeros(T, Hk, D, dtype=torch.float16, device="cuda"), "k": k}[k_out]
    tb.tb_rotary_cache_write(q, k, v, pos, torch.from_numpy(slots).cuda(), plan, R, int(pairs), qo, kc, vc, k_out=ko, dev_status=st)
    assert torch.equal(qo, wq) and (ko is None or torch.equal(ko, wk))
    assert np.array_equal(bits(kc), want[0].view(np.uint16)) and np.array_equal(bits(vc), want[1].view(np.uint16))
    assert int(st) == 0
    slots[-1] = pages * page  # just past the cache
    before = kc.clone(), vc.clone()
    tb.tb_rotary_cache_write(q, wk, v, pos, torch.from_numpy(np.where(slots < pages * page, -1, slots)).cuda(), plan, R, int(pairs), qo, kc, vc, dev_status=st)
    assert int(st) == tb.TB_DEV_BAD_SLOT and torch.equal(kc, before[0]) and torch.equal(vc, before[1])


def test_many_tokens_and_few_heads():
    """More tiles than CTAs: against 64 bits on the device."""
    import ternary_hadamard_rotated_gb300 as tb

    T, D, R = 30011, 64, 32
    plan, f, amp = make_plan(R)
    q = torch.randn(T, 1, D, device="cuda").half()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    tb.tb_rotary(q, None, pos, plan, R, 0, out, None)
    w = pos.double()[:, None, None] * torch.from_numpy(f).cuda()
    a, b = q[..., : R // 2].double(), q[..., R // 2: R].double()
    want = torch.cat([a * w.cos() - b * w.sin(), a * w.sin() + b * w.cos(), q[..., R:].double()], -1)
    size = torch.cat([a.abs() + b.abs()] * 2 + [0 * q[..., R:].double()], -1)
    close(out.cpu().numpy(), want.cpu().numpy(), size.cpu().numpy())


def test_explicit_frequencies_and_amplitude():
    import ternary_hadamard_rotated_gb300 as tb

    f = np.array([0.0, 1.0, -2.5, 100.0, 1e-9, 6.283185307179586, 3.0, 0.1])
    plan, _, _ = make_plan(16, freqs=torch.from_numpy(f).cuda(), amplitude=1.5)
    rng = np.random.default_rng(3)
    q = torch.from_numpy(rng.standard_normal((40, 2, 16)).astype(np.float16)).cuda()
    pos = np.arange(40) * 1003 - 77
    out = torch.empty_like(q)
    tb.tb_rotary(q, None, torch.from_numpy(pos.astype(np.int32)).cuda(), plan, 16, 0, out, None)
    want, size = serving.rotary(q.cpu().numpy(), pos, f, 1.5, 16, False)
    close(out.cpu().numpy(), want, size)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    f[[1, 6]] = np.nan, np.inf
    tb.tb_rotary_plan(plan, 16, freqs=torch.from_numpy(f).cuda(), dev_status=st)
    assert int(st) == tb.TB_DEV_BAD_PLAN
    f[[1, 6]] = 0
    tb.tb_rotary(q, None, torch.from_numpy(pos.astype(np.int32)).cuda(), plan, 16, 0, out, None)
    want, size = serving.rotary(q.cpu().numpy(), pos, f, 1.0, 16, False)
    close(out.cpu().numpy(), want, size)


def test_a_plan_of_another_width_computes_nothing():
    import ternary_hadamard_rotated_gb300 as tb

    plan, _, _ = make_plan(64)
    q = torch.ones(3, 2, 64, dtype=torch.float16, device="cuda")
    pos = torch.ones(3, dtype=torch.int32, device="cuda")
    for p in (plan, torch.zeros_like(plan)):
        out, st = torch.full_like(q, 5), torch.zeros(1, dtype=torch.int32, device="cuda")
        tb.tb_rotary(q, None, pos, p, 32, 0, out, None, dev_status=st)
        assert int(st) == tb.TB_DEV_BAD_PLAN and (out == 5).all()


@pytest.mark.parametrize("R,pairs", [(32, False), (32, True), (22, False), (22, True)])
def test_what_is_not_finite_stays_in_its_pair(R, pairs):
    import ternary_hadamard_rotated_gb300 as tb

    plan, f, amp = make_plan(R)
    q = torch.randn(6, 3, 64, device="cuda").half()
    pos = torch.arange(1, 7, dtype=torch.int32, device="cuda")
    clean, dirty = torch.empty_like(q), torch.empty_like(q)
    tb.tb_rotary(q, None, pos, plan, R, int(pairs), clean, None)
    x = q.clone()
    x[2, 1, 5], x[4, 0, 60] = float("nan"), float("inf")
    tb.tb_rotary(x, None, pos, plan, R, int(pairs), dirty, None)
    i = 5 // 2 if pairs else 5
    pair = (2 * i, 2 * i + 1) if pairs else (i, i + R // 2)
    assert dirty[2, 1, list(pair)].isnan().all() and dirty[4, 0, 60] == float("inf")
    dirty[2, 1, list(pair)], dirty[4, 0, 60] = clean[2, 1, list(pair)], clean[4, 0, 60]
    assert torch.equal(clean, dirty)


def test_inverse_is_the_gradient():
    """The transpose: <g, turn(x)> = <inverse turn(g), x>, against differences of a turned sum."""
    import ternary_hadamard_rotated_gb300 as tb

    plan, f, amp = make_plan(64, scaling="parts", factor=16.0)
    rng = np.random.default_rng(5)
    x, g = (torch.from_numpy(rng.standard_normal((20, 2, 64)).astype(np.float16)).cuda() for _ in range(2))
    pos = torch.arange(0, 2000, 100, dtype=torch.int32, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    tb.tb_rotary(x, None, pos, plan, 64, 0, y, None)
    tb.tb_rotary(g, None, pos, plan, 64, 0, dx, None, inverse=True)
    a, b = (g.double() * y.double()).sum((1, 2)), (dx.double() * x.double()).sum((1, 2))
    room = 2.0 ** -10 * amp * 2 * (g.double().norm(dim=(1, 2)) * x.double().norm(dim=(1, 2)))  # two fp16 roundings, Cauchy-Schwarz
    assert ((a - b).abs() <= room).all()
    e = torch.zeros_like(x)
    e[:, :, 7] = 1  # the difference of two turned inputs is the turned unit vector: a column of the matrix
    col = torch.empty_like(x)
    tb.tb_rotary(e, None, pos, plan, 64, 0, col, None)
    d = (g.double() * col.double()).sum(-1)
    assert ((d - dx[:, :, 7].double()).abs() <= 2.0 ** -10 * amp * 2 * g.double().norm(dim=-1)).all()


def test_graph_stream_and_far_offsets():
    import ternary_hadamard_rotated_gb300 as tb

    plan, f, amp = make_plan(64)
    pages, H, page, D = 2 ** 31 // (4 * 64 * 256) + 40, 4, 64, 256  # caches of more than 2^31 elements
    kc = torch.zeros((pages, H, page, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    q, k, v = inputs(np.random.default_rng(1), 3, 2, H, D)
    slots = torch.tensor([pages * page - 1, 0, (pages - 2) * page], device="cuda")
    pos = torch.tensor([5, 6, 7], dtype=torch.int32, device="cuda")
    qo = torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        tb.tb_rotary_cache_write(q, k, v, pos, slots, plan, 64, 0, qo, kc, vc)
    side.synchronize()
    wk, wq = torch.empty_like(k), torch.empty_like(q)
    tb.tb_rotary(q, k, pos, plan, 64, 0, wq, wk)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // page, :, s % page], wk[i]) and torch.equal(vc[s // page, :, s % page], v[i])
    assert torch.equal(qo, wq)
    del kc, vc
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.tb_rotary(q, k, pos, plan, 64, 0, qo, wk)
    pos.add_(1000)
    g.replay()
    tb.tb_rotary(q, None, pos, plan, 64, 0, wq, None)
    torch.cuda.synchronize()
    assert torch.equal(qo, wq)
