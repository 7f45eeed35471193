"""GPU parity of the adapters where a token's A x differ widely from rank to rank, and the largest do not reach a column.

Tolerance: that of the adapters' own tests ((K/8 + R/8 + 80) 2^-23 S + 2^-21 H, and half a step of fp16), with what the
second product's operand leaves of a rank that is far below the token's largest one, top = max |scale A x|: hi + lo 2^-12
with top's hi in [2^14, 2^15] and both of at least 2^-24's steps, so 2^-25 2^-12 2^-14 = 2^-51 of top a rank, times its |B|.

What those tests' bound leaves out, as they have no such elements beside large ones: the tensor core's sums are rounded to
2^-23 of their largest term's place, and that place goes by the operands' exponents, of which an fp16 number below 2^-14
has that of 2^-14.  (Measured, 16 ranks: h = top with B = 2^-24 or 2^-14, and a second rank 2^-16 to 2^-36 of it: the sum is off by
2^-39 top with the first, though its product is 2^-24 top, and by 2^-36 top with the second; not at all with B = 0.)  The second
product's chain of at most R/8 + 40 sums is therefore rounded to 2^-23 of H', which is H with max(|B|, 2^-14) where B is not 0.
"""
import numpy as np
import pytest

from oracle import serving

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("R", [8, 16, 32, 64, 200])
@pytest.mark.parametrize("below", [16, 22, 29, 34])
def test_small_ranks_beside_large_ones(T, R, below):
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(T + R + below)
    K, N, n = 256, 72, 2
    a = (rng.integers(1, 8, (n, R, K)) * 2.0 ** (10 - below)).astype(np.float16)  # (down to multiples of 2^-24, exact)
    b = (rng.standard_normal((n, N, R)) * 64).astype(np.float16)
    large = np.arange(3, R, 64)  # one in each block of ranks
    a[:, large] = (rng.integers(4, 8, (n, len(large), K)) * 2.0 ** 10).astype(np.float16)
    b[:, :, large] = 0
    b[:, 1::2, large] = (rng.integers(-3, 4, (n, N // 2, len(large))) * 2.0 ** -24).astype(np.float16)
    x = (rng.random((T, K)) + 0.5).astype(np.float16)
    y = np.zeros((T, N), dtype=np.float16)
    scale = np.array([2.0 ** (below - 30), -(2.0 ** (below - 29))], dtype=np.float32)
    rows, adapter = [0, T // 3, T], [1, 0]
    dev = lambda m: torch.from_numpy(m).cuda()  # noqa: E731
    plan = torch.empty(tb.tb_adapter_plan_size(T, n), dtype=torch.uint8, device="cuda")
    tb.tb_adapter_plan(dev(np.array(rows, dtype=np.int32)), dev(np.array(adapter, dtype=np.int32)), T, n, plan)
    ws = torch.empty(tb.tb_adapter_linear_workspace_size(T, n, K, N, R), dtype=torch.uint8, device="cuda")
    out = dev(y)
    tb.tb_adapter_linear(dev(x), dev(a), dev(b), dev(scale), plan, out, ws)
    got = out.cpu().numpy().astype(np.float64)
    want, S, H = serving.adapter_linear(x, a, b, scale, None, rows, adapter, y)
    assert np.isfinite(want).all() and np.abs(want).max() < 60000
    floor, H1 = np.zeros_like(want), np.zeros_like(want)
    for s, e, g in zip(rows, rows[1:], adapter):
        h, w = np.abs(float(scale[g]) * (x[s:e].astype(np.float64) @ a[g].astype(np.float64).T)), np.abs(b[g].astype(np.float64))
        floor[s:e] = 2.0 ** -51 * h.max(1, initial=0)[:, None] * w.sum(1)
        H1[s:e] = h @ np.where(w > 0, np.maximum(w, 2.0 ** -14), 0).T
    tol = (K / 8 + R / 8 + 80) * 2.0 ** -23 * S + 2.0 ** -21 * H + floor + (R / 8 + 40) * 2.0 ** -23 * H1 + 2.0 ** -11 * np.abs(want) + 2.0 ** -25
    err = np.abs(got - want)
    assert (err <= tol).all(), np.max(err / tol)


@pytest.mark.parametrize("T,R", [(1, 16), (40, 16), (300, 16), (40, 64), (300, 64), (40, 200), (300, 200)])
def test_an_infinite_rank_beside_large_ones(T, R):
    """One rank's A x is infinite, another's far above fp16's range: their sum is that infinity, where B reaches it."""
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(T + R)
    K, N, n = 64, 72, 2
    a = rng.standard_normal((n, R, K)).astype(np.float16)
    b = rng.standard_normal((n, N, R)).astype(np.float16)
    a[0, 7], b[0, :, 7] = 6e4, rng.choice([-9.0, 9.0], N)
    a[0, 2, 5], b[0, :, 2] = np.inf, rng.choice([-1.0, 0.0, 1.0], N)
    x = (rng.random((T, K)) + 0.5).astype(np.float16)
    x[:, 5] = rng.choice([-2.0, 0.5], T)
    y = rng.standard_normal((T, N)).astype(np.float16)
    scale = np.array([0.5, 2.0], dtype=np.float32)
    rows, adapter = [0, (T + 1) // 2, T], [0, 1]
    dev = lambda m: torch.from_numpy(m).cuda()  # noqa: E731
    plan = torch.empty(tb.tb_adapter_plan_size(T, n), dtype=torch.uint8, device="cuda")
    tb.tb_adapter_plan(dev(np.array(rows, dtype=np.int32)), dev(np.array(adapter, dtype=np.int32)), T, n, plan)
    ws = torch.empty(tb.tb_adapter_linear_workspace_size(T, n, K, N, R), dtype=torch.uint8, device="cuda")
    out = dev(y)
    tb.tb_adapter_linear(dev(x), dev(a), dev(b), dev(scale), plan, out, ws)
    got = out.cpu().numpy().astype(np.float64)
    with np.errstate(invalid="ignore"):
        want, _, _ = serving.adapter_linear(x, a, b, scale, None, rows, adapter, y)
    first = slice(0, rows[1])
    assert np.isinf(want[first]).any() and not np.isfinite(want[first]).any()
    assert np.array_equal(got[first], want[first], equal_nan=True)
    assert np.isfinite(got[rows[1]:]).all()
