"""GPU parity of the adapters beside a shared linear.

Tolerance, with S = |scale| |B| sum |A x| (absolute terms) and H = |scale| |B| |A x|: a sum of K products in fp32,
in whatever order, of which a chain of at most K / 8 + 40 sums is truncated or rounded by 2^-23 of the terms so
far: (K/8 + 40) 2^-23 S; the scale's product and the two terms of 11 bits of A x: 2^-21 H; the second product in the
same way: (R/8 + 40) 2^-23 H and as much of S, H <= S; then the sum with y and the rounding to fp16, half a step:
2^-11 of the value, 2^-25 below its normal range.
"""
import numpy as np
import pytest

from oracle import serving

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def make(rng, n, R, K, N, T, wide=0):
    a = (rng.standard_normal((n, R, K)) * K ** -0.5).astype(np.float16)
    b = rng.standard_normal((n, N, R)).astype(np.float16)
    x = rng.standard_normal((T, K + wide)).astype(np.float16)
    y = rng.standard_normal((T, N + wide)).astype(np.float16)
    scale = (rng.standard_normal(n) * 2).astype(np.float32)
    return a, b, x, y, scale


def dev(*arrays):
    return [None if m is None else torch.from_numpy(np.ascontiguousarray(m)).cuda() for m in arrays]


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


class Step:
    """A plan on the device, and calls with it."""

    def __init__(self, lens, adapter, n, T=None, row_start=None):
        import ternary_hadamard_rotated_gb300 as tb

        self.T = int(sum(lens)) if T is None else T
        self.n = n
        self.rows, self.adapter = dev(starts(lens) if row_start is None else np.array(row_start, dtype=np.int32), np.array(adapter, dtype=np.int32))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.plan = torch.full((tb.tb_adapter_plan_size(self.T, n),), 0x5A, dtype=torch.uint8, device="cuda")
        tb.tb_adapter_plan(self.rows, self.adapter, self.T, n, self.plan, self.status)

    def __call__(self, x, a, b, scale, y, out=None, rank=None):
        import ternary_hadamard_rotated_gb300 as tb

        size = tb.tb_adapter_linear_workspace_size(self.T, self.n, x.shape[1], y.shape[1], a.shape[1])
        ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # (NaN wherever it is read before it is written)
        tb.tb_adapter_linear(x, a, b, scale, self.plan, y, ws[:size], out=out, rank=rank, dev_status=self.status)
        assert (ws[size:] == 0xFF).all()


def check(got, x, a, b, scale, rank, rows, adapter, y):
    want, S, H = serving.adapter_linear(x, a, b, scale, rank, rows, adapter, y)
    K, R = a.shape[2], a.shape[1]
    tol = (K / 8 + R / 8 + 80) * 2.0 ** -23 * S + 2.0 ** -21 * H + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    err = np.abs(np.asarray(got, dtype=np.float64) - want)
    assert (err <= tol).all(), np.nanmax(err / tol)
    bare = np.concatenate([np.arange(rows[i], rows[i + 1]) for i, g in enumerate(adapter) if g < 0] + [np.zeros(0, dtype=int)]).astype(int)
    assert np.array_equal(np.asarray(got)[bare].view(np.uint16), np.asarray(y)[bare].view(np.uint16))


@pytest.mark.parametrize("lens,adapter,n,R,K,N,ranks", [
    ([1], [0], 1, 16, 5120, 17408, False), ([1], [-1], 1, 8, 64, 64, False), ([1] * 5, [2, 2, 0, -1, 2], 3, 8, 8, 8, True), ([1] * 64, None, 40, 32, 2048, 1032, True),
    ([3, 0, 17, 1, 8], [1, 0, 1, 0, -1], 2, 24, 1000, 520, False), ([16, 16, 1], [0, 0, 0], 1, 64, 328, 4096, False), ([129, 5, 260], [1, 3, 1], 4, 64, 520, 264, True),
    ([700], [0], 2, 16, 5120, 1288, False), ([40, 300, 90, 1], [2, 0, -1, 2], 3, 128, 264, 776, True), ([33], [0], 1, 256, 5000, 72, False), ([500], [1], 2, 40, 40, 136, True),
    ([1000, 7], [0, 1], 2, 200, 128, 1000, True), ([2], [0], 1, 8, 17408, 5120, False),
    ([250, 6], [1, 0], 2, 24, 72, 2000, True), ([250, 7], [1, 0], 2, 24, 72, 2000, True), ([128, 128, 1, 0, 129], [0, 1, 0, 1, -1], 2, 56, 5120, 64, True),
    ([400, 3], [0, 1], 2, 256, 2048, 72, False)])
@pytest.mark.parametrize("place", ["out", "in"])
def test_adapters_match(lens, adapter, n, R, K, N, ranks, place):
    rng = np.random.default_rng(len(lens) * 1000 + K + N)
    if adapter is None:
        adapter = [int(g) for g in rng.integers(-1, n, len(lens))]
    T, wide = sum(lens), 8 if place == "in" else 0
    a, b, x, y, scale = make(rng, n, R, K, N, T, wide)
    rank = rng.integers(0, R + 1, n).astype(np.int32) if ranks else None
    if ranks:  # what lies behind a rank does not matter
        for g in range(n):
            a[g, rank[g]:], b[g, :, rank[g]:] = np.nan, np.inf
    step = Step(lens, adapter, n)
    ad, bd, xd, yd, sd, rd = dev(a, b, x, y, scale, rank)
    xs, ys = xd[:, :K], yd[:, wide: wide + N] if wide else yd
    if place == "in":
        step(xs, ad, bd, sd, ys, rank=rd)
        got = yd.cpu().numpy()
        assert np.array_equal(got[:, :wide].view(np.uint16), y[:, :wide].view(np.uint16))
        got = got[:, wide:]
    else:
        out = torch.full((T + 1, N), 9.0, dtype=torch.float16, device="cuda")
        step(xs, ad, bd, sd, ys, out=out[:T], rank=rd)
        assert torch.equal(yd, dev(y)[0]) and (out[T] == 9).all()
        got = out[:T].cpu().numpy()
        again = torch.empty_like(out[:T])
        step(xs, ad, bd, sd, ys, out=again, rank=rd)
        assert torch.equal(again, out[:T])  # repeats bit for bit
    assert int(step.status) == 0
    check(got, x[:, :K], a, b, scale, rank, starts(lens), adapter, y[:, wide:])


def test_many_requests_and_adapters():
    rng = np.random.default_rng(11)
    B, n = 5000, 3001
    lens = rng.integers(0, 4, B)
    lens[77], lens[4000] = 900, 300
    adapter = rng.integers(-1, n, B)
    a, b, x, y, scale = make(rng, n, 8, 16, 24, int(lens.sum()))
    step = Step(lens, adapter, n)
    ad, bd, xd, yd, sd = dev(a, b, x, y, scale)
    step(xd, ad, bd, sd, yd)
    assert int(step.status) == 0
    check(yd.cpu().numpy(), x, a, b, scale, None, starts(lens), adapter, y)


def test_a_row_depends_on_no_other():
    rng = np.random.default_rng(2)
    lens, adapter = [5, 40, 200, 3], [0, 1, 0, -1]
    a, b, x, y, scale = make(rng, 2, 16, 256, 136, sum(lens))
    step = Step(lens, adapter, 2)
    ad, bd, xd, yd, sd = dev(a, b, x, y, scale)
    clean, dirty = torch.empty_like(yd), torch.empty_like(yd)
    step(xd, ad, bd, sd, yd, out=clean)
    bad = [0, 44, 100, 244, 246]
    xd[0, 3], xd[44, 7], xd[100, 0], xd[244, 255], xd[246, 1] = (float(v) for v in ("nan", "inf", "-inf", "nan", "nan"))
    step(xd, ad, bd, sd, yd, out=dirty)
    assert not dirty[[0, 44, 100, 244]].isfinite().any()
    keep = [t for t in range(sum(lens)) if t not in bad[:4]]
    assert torch.equal(clean[keep], dirty[keep])
    one = torch.empty_like(yd[7:8])  # alone as in the batch, within the tolerance of both
    alone = Step([1], [1], 2)
    alone(xd[7:8], ad, bd, sd, yd[7:8], out=one)
    check(one.cpu().numpy(), x[7:8], a, b, scale, None, [0, 1], [1], y[7:8])


def test_wide_range_of_values():
    """A x far above fp16's range and far below it in one row, and scales that bring it back."""
    rng = np.random.default_rng(4)
    T, K, R, N = 40, 512, 16, 256
    a, b, x, y, _ = make(rng, 2, R, K, N, T)
    a[:] = np.abs(a)
    a[:, ::2] *= 2.0 ** 9  # rows of A of very different sizes
    a[:, 1::2] *= 2.0 ** -12
    b[:, :, ::2] *= np.float16(2.0 ** -14)
    x[:] = np.abs(x) * 64
    y *= 2.0 ** -6
    scale = np.array([2.0 ** -8, 2.0 ** 3], dtype=np.float32)
    lens, adapter = [1, 39], [0, 1]
    step = Step(lens, adapter, 2)
    ad, bd, xd, yd, sd = dev(a, b, x, y, scale)
    step(xd, ad, bd, sd, yd)
    check(yd.cpu().numpy(), x, a, b, scale, None, starts(lens), adapter, y)


def test_ids_row_starts_and_plans_that_do_not_fit():
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(6)
    a, b, x, y, scale = make(rng, 2, 8, 64, 40, 12)
    ad, bd, xd, yd, sd = dev(a, b, x, y, scale)

    def run(step):
        out = torch.full_like(yd, 3.0)
        step(xd, ad, bd, sd, yd, out=out)
        return out

    step = Step([4, 4, 4], [0, 2, 1], 2)  # adapter 2 of two: taken as none
    assert int(step.status) == tb.TB_DEV_BAD_ID
    check(run(step).cpu().numpy(), x, a, b, scale, None, [0, 4, 8, 12], [0, -1, 1], y)
    for rows, live in (([0, 5, 3, 9], {0: 5}), ([0, 4, 30, 12], {0: 4}), ([-3, 4, 8, 12], {4: 8, 8: 12}), ([2, 2, 6, 9], {2: 9}), ([0, 2 ** 31 - 1, -2 ** 31, 12], {}),
                       ([6, 8, 8, 6], {6: 8})):
        step = Step([4, 4, 4], [0, 1, 0], 2, T=12, row_start=rows)
        assert int(step.status) == (0 if rows[0] == 2 else tb.TB_DEV_BAD_LEN)
        out = run(step)
        inside = [t for s, e in live.items() for t in range(s, e)]
        rest = [t for t in range(12) if t not in inside]
        assert (out[rest] == 3).all()
        check(out[inside].cpu().numpy(), x[inside], a, b, scale, None, list(range(len(inside) + 1)),
              [[0, 1, 0][[i for i in range(3) if rows[i] <= t < rows[i + 1] and i < 3][0]] for t in inside], y[inside])
    small = Step([4, 4], [0, 1], 2)  # another step's plan, of fewer tokens (in a buffer that is large enough)
    other = Step([4, 4, 4], [0, 1, 0], 2)
    other.plan[: small.plan.numel()] = small.plan
    out = run(other)
    assert int(other.status) == tb.TB_DEV_BAD_PLAN and (out == 3).all()


def test_step_in_a_graph():
    """Plan and linear captured together; replayed for other adapters and tokens."""
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(8)
    lens, n, R, K, N = [1, 3, 1, 20, 1], 3, 16, 640, 1096
    a, b, x, y, scale = make(rng, n, R, K, N, sum(lens))
    step = Step(lens, [0, 1, 2, 0, -1], n)
    ad, bd, xd, yd, sd = dev(a, b, x, y, scale)
    out = torch.empty_like(yd)
    ws = torch.empty(tb.tb_adapter_linear_workspace_size(step.T, n, K, N, R), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        tb.tb_adapter_plan(step.rows, step.adapter, step.T, n, step.plan)
        tb.tb_adapter_linear(xd, ad, bd, sd, step.plan, yd, ws, out=out)
        tb.tb_adapter_linear(xd, ad, bd, sd, step.plan, out, ws)  # the same workspace, on what the first call wrote
    for k in range(3):
        lens = [int(v) for v in rng.permutation(lens)]
        adapter = [int(v) for v in rng.integers(-1, n, 5)]
        x = rng.standard_normal(x.shape).astype(np.float16)
        step.rows.copy_(dev(starts(lens))[0])
        step.adapter.copy_(dev(np.array(adapter, dtype=np.int32))[0])
        xd.copy_(dev(x)[0])
        g.replay()
        torch.cuda.synchronize()
        once = torch.empty_like(yd)
        Step(lens, adapter, n)(xd, ad, bd, sd, yd, out=once)
        check(once.cpu().numpy(), x, a, b, scale, None, starts(lens), adapter, y)
        check(out.cpu().numpy(), x, a, b, scale, None, starts(lens), adapter, once.cpu().numpy())


def test_weights_past_two_to_the_31_elements():
    rng = np.random.default_rng(9)
    n, R, K, N = 2100, 64, 17408, 64
    a = torch.zeros((n, R, K), dtype=torch.float16, device="cuda")  # 4.7 GB
    small, b, x, y, scale = make(rng, 1, R, K, N, 3)
    a[n - 1].copy_(torch.from_numpy(small[0]))
    bd = torch.zeros((n, N, R), dtype=torch.float16, device="cuda")
    bd[n - 1].copy_(torch.from_numpy(b[0]))
    sd = torch.full((n,), float(scale[0]), device="cuda")
    xd, yd = dev(x, y)
    Step([2, 1], [n - 1, 0], n)(xd, a, bd, sd, yd)
    got = yd.cpu().numpy()
    check(got[:2], x[:2], small, b, scale, None, [0, 2], [0], y[:2])
    assert np.array_equal(got[2], y[2])


@pytest.mark.parametrize("lens", [[4, 4, 4], [700, 1, 30]])
def test_a_plan_of_another_step_in_its_own_buffer(lens):
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(10)
    ad, bd, xd, yd, sd = dev(*make(rng, 2, 8, 64, 40, sum(lens)))
    for small in (Step([1, 1], [0, 1], 2), Step(lens, [0, 1, 1], 3)):  # of fewer tokens, in fewer bytes; of more adapters
        step = Step(lens, [0, 1, 0], 2)
        step.plan = small.plan
        out = torch.full_like(yd, 3.0)
        step(xd, ad, bd, sd, yd, out=out)
        assert int(step.status) == tb.TB_DEV_BAD_PLAN and (out == 3).all()


@pytest.mark.parametrize("T", [40, 300])
def test_steps_one_after_another_in_the_same_plan(T):
    """Steps with and without adapters in turn, each with its plan written over the one before it."""
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(11)
    n, R, K, N, count = 5, 16, 512, 264, 24
    a, b, x, y, scale = make(rng, n, R, K, N, T)
    ad, bd, xd, yd, sd = dev(a, b, x, y, scale)
    lens = [T - 12, 3, 9]
    rows = dev(starts(lens))[0]
    adapters = [[-1, -1, -1] if i % 2 else [int(v) for v in rng.integers(-1, n, 3)] for i in range(count)]
    ids = [dev(np.array(g, dtype=np.int32))[0] for g in adapters]
    plan = torch.empty(tb.tb_adapter_plan_size(T, n), dtype=torch.uint8, device="cuda")
    ws = torch.empty(tb.tb_adapter_linear_workspace_size(T, n, K, N, R), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(yd) for _ in range(count)]
    for g, out in zip(ids, outs):
        tb.tb_adapter_plan(rows, g, T, n, plan)
        tb.tb_adapter_linear(xd, ad, bd, sd, plan, yd, ws, out=out)
    for g, out in zip(adapters, outs):
        check(out.cpu().numpy(), x, a, b, scale, None, starts(lens), g, y)
