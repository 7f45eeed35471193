"""GPU parity of the gated delta rule against the float64 recurrence.

Tolerances.  Outputs: half an fp16 ulp, and three operands that may be rounded to fp16 (the state,
the decayed products q . k, the corrections u) on the sum of absolute terms: 2^-11 |o| + 3 2^-11 mag.
States: operands of 22 bits or more in fp32 sums, in a recurrence that does not amplify (|k| <= 1,
beta <= 1, decays <= 1): 2^-17 of the 2-norm of each head's state (32 times 2^-22).
"""
import numpy as np
import pytest

from oracle import mixers

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D = 128


def make(seed, lens, Hk, Hv, normalise, rate=(-6, 0.5), fused=True):
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    wide = torch.randn(T, (2 * Hk + Hv) * D + 16, generator=gen).half()
    if not normalise:
        n = 2 * Hk * D
        x = wide[:, 8: 8 + n].float().unflatten(1, (2 * Hk, D))
        wide[:, 8: 8 + n] = (x / x.norm(dim=-1, keepdim=True) * 0.999).half().flatten(1)
    wide = wide.cuda()
    q = wide[:, 8: 8 + Hk * D].unflatten(1, (Hk, D))
    k = wide[:, 8 + Hk * D: 8 + 2 * Hk * D].unflatten(1, (Hk, D))
    v = wide[:, 8 + 2 * Hk * D: 8 + (2 * Hk + Hv) * D].unflatten(1, (Hv, D))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    g = -torch.exp(torch.linspace(*rate, Hv)) * torch.nn.functional.softplus(torch.randn(T, Hv, generator=gen))
    beta = torch.sigmoid(torch.randn(T, Hv, generator=gen))
    state = torch.randn(len(lens), Hv, D, D, generator=gen) * 0.3
    return q, k, v, g.cuda(), beta.cuda(), state.cuda()


def starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def workspace(T, B, n, Hk, Hv):
    import ternary_hadamard_rotated_gb300 as tb

    return torch.full((tb.tb_gated_delta_workspace_size(T, B, n, Hk, Hv),), 0xA5, dtype=torch.uint8, device="cuda")


def check(o, state, args, lens, init, normalise, scale=D ** -0.5):
    q, k, v, g, beta = (x.cpu().numpy() for x in args)
    want, fin, mag = mixers.gated_delta(q, k, v, g, beta, starts(lens).tolist(), init.cpu().numpy(), normalise, scale)
    got = o.double().cpu().numpy()
    tol = 2.0 ** -11 * np.abs(want) + 3 * 2.0 ** -11 * mag + 2.0 ** -25
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])
    if state is not None:
        s = state.double().cpu().numpy()
        err = np.linalg.norm((s - fin).reshape(*s.shape[:2], -1), axis=-1)
        ref = np.linalg.norm(fin.reshape(*s.shape[:2], -1), axis=-1)
        assert (err <= 2.0 ** -17 * ref + 1e-30).all(), float((err / np.maximum(ref, 1e-30)).max())


def run(seed, lens, Hk, Hv, normalise=True, max_len=None, with_state=True, **kw):
    import ternary_hadamard_rotated_gb300 as tb

    q, k, v, g, beta, init = make(seed, lens, Hk, Hv, normalise, **kw)
    T, B = sum(lens), len(lens)
    n = max(lens) if max_len is None else max_len
    full = torch.full((T + 1, Hv, D), 7.0, dtype=torch.float16, device="cuda")
    out = torch.full((B + 1, Hv, D, D), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if not with_state:
        init = torch.zeros_like(init)
    tb.tb_gated_delta(q, k, v, g, beta, starts(lens), n, full[:T], workspace(T, B, n, Hk, Hv),
                      state_in=init if with_state else None, state_out=out[:B], normalise=normalise, dev_status=st)
    torch.cuda.synchronize()
    assert (full[T:] == 7.0).all() and (out[B:] == 7.0).all() and int(st) == 0
    check(full[:T], out[:B], (q, k, v, g, beta), lens, init, normalise)


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 6), (4, 4)])
@pytest.mark.parametrize("lens", [[1], [1] * 9, [2, 1, 3], [5, 0, 1, 4]])
def test_few_tokens(Hk, Hv, lens):
    run(1, lens, Hk, Hv)
    run(2, lens, Hk, Hv, normalise=False)


def test_step_of_a_full_batch():
    run(3, [1] * 40, 16, 48)


@pytest.mark.parametrize("lens", [[16], [63], [64], [65], [128], [129, 1, 0, 64], [200, 17, 31], [700]])
@pytest.mark.parametrize("normalise", [True, False])
def test_prompts(lens, normalise):
    run(4, lens, 2, 6, normalise=normalise)


def test_prompts_of_all_heads():
    run(5, [130, 70], 16, 48)


def test_without_a_first_state():
    run(6, [100, 3], 2, 2, with_state=False)


@pytest.mark.parametrize("n", [0, 1, 7, 64, 100000])
def test_any_max_len_gives_the_same(n):
    run(7, [90, 1, 33], 2, 4, max_len=n)


def test_strong_and_vanishing_decays():
    run(8, [150], 2, 4, rate=(2.0, 5.0))     # the state is forgotten within a token or two
    run(9, [150], 2, 4, rate=(-20.0, -12.0))  # hardly ever


def test_small_and_large_values():
    """The state's relative precision does not hang on the values' size."""
    import ternary_hadamard_rotated_gb300 as tb

    for scale in (1e-3, 300.0):
        lens = [190]
        q, k, v, g, beta, init = make(10, lens, 1, 2, True)
        v = (v.float() * scale).half()
        init = init * scale
        o = torch.empty(190, 2, D, dtype=torch.float16, device="cuda")
        out = torch.empty_like(init)
        tb.tb_gated_delta(q, k, v, g, beta, starts(lens), 190, o, workspace(190, 1, 190, 1, 2), state_in=init, state_out=out, normalise=True)
        check(o, out, (q, k, v, g, beta), lens, init, True)


def test_keys_that_repeat():
    """The same key again and again, steps near 1: the triangular system at its hardest."""
    import ternary_hadamard_rotated_gb300 as tb

    lens = [200]
    q, k, v, g, beta, init = make(11, lens, 1, 2, True)
    k = k[:1].expand(200, 1, D) + 0.05 * k
    k = k.half().contiguous()
    beta = torch.full_like(beta, 0.97)
    g = g * 0.01
    o = torch.empty(200, 2, D, dtype=torch.float16, device="cuda")
    out = torch.empty_like(init)
    tb.tb_gated_delta(q, k, v, g, beta, starts(lens), 200, o, workspace(200, 1, 200, 1, 2), state_in=init, state_out=out, normalise=True)
    check(o, out, (q, k, v, g, beta), lens, init, True)


def test_a_decay_of_zero_forgets_everything():
    import ternary_hadamard_rotated_gb300 as tb

    lens = [70]
    q, k, v, g, beta, init = make(12, lens, 1, 1, True)
    g[30] = -float("inf")
    g[31] = -1e30
    o = torch.empty(70, 1, D, dtype=torch.float16, device="cuda")
    out = torch.empty_like(init)
    tb.tb_gated_delta(q, k, v, g, beta, starts(lens), 70, o, workspace(70, 1, 70, 1, 1), state_in=init, state_out=out, normalise=True)
    check(o, out, (q, k, v, g, beta), lens, init, True)


@pytest.mark.parametrize("lens", [[1, 1, 1, 1], [70, 1, 0, 90]])
def test_pools_and_slots(lens):
    """States in a pool, in place, with requests that start from nothing or keep nothing."""
    import ternary_hadamard_rotated_gb300 as tb

    Hk, Hv, T = 2, 4, sum(lens)
    q, k, v, g, beta, _ = make(13, lens, Hk, Hv, True)
    pool = torch.randn(9, Hv, D, D, device="cuda") * 0.3
    before = pool.clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    sin, sout = [7, -1, 3, 0], [7, 2, 3, -1]
    o = torch.empty(T, Hv, D, dtype=torch.float16, device="cuda")
    st = torch.zeros(1, **i32)
    tb.tb_gated_delta(q, k, v, g, beta, starts(lens), max(lens), o, workspace(T, 4, max(lens), Hk, Hv), state_in=pool, state_out=pool,
                      slot_in=torch.tensor(sin, **i32), slot_out=torch.tensor(sout, **i32), normalise=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    init = torch.stack([before[s] if s >= 0 else torch.zeros_like(before[0]) for s in sin])
    q_, want_state = None, pool.clone()
    got = torch.stack([pool[s] if s >= 0 else init[b] for b, s in enumerate(sout)])
    kept = [b for b, s in enumerate(sout) if s >= 0]
    args = (q, k, v, g, beta)
    check(o, None, args, lens, init, True)
    fin = mixers.gated_delta(*(x.cpu().numpy() for x in args), starts(lens).tolist(), init.cpu().numpy(), True, D ** -0.5)[1]
    for b in kept:
        s = got[b].double().cpu().numpy()
        assert np.linalg.norm(s - fin[b]) <= 2.0 ** -17 * np.linalg.norm(fin[b]) + 1e-30
    for r in set(range(9)) - {s for s in sout if s >= 0}:
        assert torch.equal(pool[r], before[r])
    # a slot past the pool
    tb.tb_gated_delta(q, k, v, g, beta, starts(lens), max(lens), o, workspace(T, 4, max(lens), Hk, Hv), state_in=pool, state_out=None,
                      slot_in=torch.tensor([9, 0, 1, 2], **i32), normalise=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == tb.TB_DEV_BAD_ID


def test_row_starts_that_do_not_fit():
    import ternary_hadamard_rotated_gb300 as tb

    q, k, v, g, beta, init = make(14, [20, 20], 1, 2, True)
    i32 = dict(dtype=torch.int32, device="cuda")
    for n in (1, 40):
        o = torch.full((41, 2, D), 7.0, dtype=torch.float16, device="cuda")
        out = torch.empty_like(init)
        st = torch.zeros(1, **i32)
        tb.tb_gated_delta(q, k, v, g, beta, torch.tensor([0, 20, 41], **i32), n, o[:40], workspace(40, 2, n, 1, 2), state_in=init, state_out=out,
                          normalise=True, dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == tb.TB_DEV_BAD_LEN
        assert torch.equal(out[1], init[1]) and (o[20:] == 7.0).all()


def test_a_step_goes_on_where_a_prompt_ended():
    """A prompt and then single tokens, against the whole at once."""
    import ternary_hadamard_rotated_gb300 as tb

    lens = [133]
    q, k, v, g, beta, init = make(15, lens, 2, 6, True)
    state = init.clone()
    o = torch.empty(133, 6, D, dtype=torch.float16, device="cuda")

    def part(a, b):
        n = b - a
        tb.tb_gated_delta(q[a:b], k[a:b], v[a:b], g[a:b], beta[a:b], starts([n]), n, o[a:b], workspace(n, 1, n, 2, 6), state_in=state, state_out=state,
                          normalise=True)

    part(0, 130)
    for t in range(130, 133):
        part(t, t + 1)
    torch.cuda.synchronize()
    check(o, state, (q, k, v, g, beta), lens, init, True)


@pytest.mark.parametrize("what", ["v", "k", "g", "beta", "q", "state"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 40, 131])
def test_what_is_not_finite_stays_behind_its_token(what, bad, at):
    """The tokens before it, the other requests, the other heads and (for v and a state) the other
    columns are as without it; from it on its own head (column) is not finite."""
    import ternary_hadamard_rotated_gb300 as tb

    lens, Hk, Hv, req, head, col = [70, 150, 65], 2, 4, 1, 3, 77
    x = dict(zip(("q", "k", "v", "g", "beta", "state"), make(20, lens, Hk, Hv, True)))
    row = lens[0] + at
    T, B = sum(lens), len(lens)

    def call(a):
        o = torch.empty(T, Hv, D, dtype=torch.float16, device="cuda")
        out = torch.empty_like(a["state"])
        tb.tb_gated_delta(a["q"], a["k"], a["v"], a["g"], a["beta"], starts(lens), max(lens), o, workspace(T, B, max(lens), Hk, Hv), state_in=a["state"],
                          state_out=out, normalise=True)
        torch.cuda.synchronize()
        return o, out

    want_o, want_s = call(x)
    y = {k: v.clone() for k, v in x.items()}
    if what == "state":
        y["state"][req, head, 5, col] = bad
        row = lens[0]
    elif what == "v":
        y["v"][row, head, col] = bad
    elif what in ("g", "beta"):
        y[what][row, head] = bad
    else:
        y[what][row, head // (Hv // Hk), 9] = bad
    o, s = call(y)
    touched = torch.zeros(T, Hv, D, dtype=torch.bool, device="cuda")  # what may differ
    state = torch.zeros(B, Hv, D, D, dtype=torch.bool, device="cuda")
    end = lens[0] + lens[1]
    heads = slice(2, 4) if what in ("k", "q") else slice(head, head + 1)
    if what == "q":
        touched[row, heads] = True
    elif what in ("v", "state"):
        touched[row:end, head, col] = True
        state[req, head, :, col] = True
    else:
        touched[row:end, heads] = True
        state[req, heads] = True
    assert torch.equal(o[~touched], want_o[~touched])
    assert torch.equal(s[~state], want_s[~state])
    assert not torch.isfinite(o[touched]).any() if bad != bad else not torch.isfinite(o[touched]).all()
    if what != "q" and bad != bad:
        assert not torch.isfinite(s[state]).any()


@pytest.mark.parametrize("B", [25, 70])
def test_many_requests_with_and_without_a_first_state(B):
    """More (request, head) pairs than the GPU has room for at once, states in a pool and in place, some
    requests from nothing, some without tokens."""
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(B)
    lens = [int(n) for n in rng.choice([0, 1, 17, 63, 64, 65, 130], B)]
    lens[0] = 130
    Hk, Hv, T = 4, 12, sum(lens)
    q, k, v, g, beta, _ = make(100 + B, lens, Hk, Hv, True)
    gen = torch.Generator().manual_seed(B)
    pool = (torch.randn(B + 3, Hv, D, D, generator=gen) * 0.3).cuda()
    before = pool.clone()
    slots = rng.permutation(B + 3)[:B]
    fresh = rng.random(B) < 0.4
    i32 = dict(dtype=torch.int32, device="cuda")
    sin = [-1 if f else int(s) for s, f in zip(slots, fresh)]
    o = torch.empty(T, Hv, D, dtype=torch.float16, device="cuda")
    st = torch.zeros(1, **i32)
    tb.tb_gated_delta(q, k, v, g, beta, starts(lens), max(lens), o, workspace(T, B, max(lens), Hk, Hv), state_in=pool, state_out=pool,
                      slot_in=torch.tensor(sin, **i32), slot_out=torch.tensor(slots, **i32), normalise=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    init = torch.stack([before[s] if s >= 0 else torch.zeros_like(before[0]) for s in sin])
    check(o, pool[torch.tensor(slots, device="cuda")], (q, k, v, g, beta), lens, init, True)
    for r in set(range(B + 3)) - set(slots.tolist()):
        assert torch.equal(pool[r], before[r])


@pytest.mark.parametrize("B", [3, 9, 81])
@pytest.mark.parametrize("T", [640, 650])
def test_row_starts_that_go_back(B, T):
    """Requests 0, 2, 4, .. all have rows [0, T), those between them run backwards: together they have more chunks
    than T tokens and B requests in order could.  What does not fit is taken as empty."""
    import ternary_hadamard_rotated_gb300 as tb

    Hk, Hv = 1, 2
    q, k, v, g, beta, init = make(30, [T], Hk, Hv, True)
    init = init.expand(B, -1, -1, -1).contiguous() * torch.arange(1, B + 1, device="cuda").view(-1, 1, 1, 1)
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, T] * ((B + 1) // 2), **i32)
    assert rows.numel() == B + 1
    o = torch.full((T + 1, Hv, D), 7.0, dtype=torch.float16, device="cuda")
    out = torch.full_like(init, 5.0)
    st = torch.zeros(1, **i32)
    tb.tb_gated_delta(q, k, v, g, beta, rows, T, o[:T], workspace(T, B, T, Hk, Hv), state_in=init, state_out=out, normalise=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == tb.TB_DEV_BAD_LEN and (o[T:] == 7.0).all()
    room, chunks, used = T // 64 + B, -(-T // 64), 0
    for b in range(B):
        if b % 2 or used + chunks > room:
            assert torch.equal(out[b], init[b]), b
        else:
            fin = mixers.gated_delta(*(x.cpu().numpy() for x in (q, k, v, g, beta)), [0, T], init[b: b + 1].cpu().numpy(), True, D ** -0.5)[1][0]
            assert np.linalg.norm(out[b].double().cpu().numpy() - fin) <= 2.0 ** -17 * np.linalg.norm(fin), b
        used += 0 if b % 2 else chunks


def small_steps_case(seed, n, step, rate=(-6, 0.5), v_scale=50.0, k_norm=None, scale=None, Hk=1, Hv=3):
    """Zero first state, chunked; step: beta [T, Hv] of the (T, Hv) shape it is given."""
    import ternary_hadamard_rotated_gb300 as tb

    q, k, v, g, beta, init = make(seed, [n], Hk, Hv, k_norm is None, rate=rate)
    v = (v.float() * v_scale).half()
    if k_norm is not None:
        k, q = (k.float() * k_norm).half(), (q.float() * k_norm).half()
    beta = step(beta)
    init = torch.zeros_like(init)
    o = torch.empty(n, Hv, D, dtype=torch.float16, device="cuda")
    out = torch.empty_like(init)
    scale = D ** -0.5 if scale is None else scale
    tb.tb_gated_delta(q, k, v, g, beta, starts([n]), n, o, workspace(n, 1, n, Hk, Hv), state_in=init, state_out=out, normalise=k_norm is None, scale=scale)
    # (check's sum of absolute terms takes the scale's sign along)
    check(o if scale > 0 else -o, out, (q, k, v, g, beta), [n], init, k_norm is None, abs(scale))


@pytest.mark.parametrize("step", [1e-2, 1e-4, 1e-6, 1e-9])
def test_chunks_of_small_steps(step):
    """The state's and the outputs' precision does not hang on the steps' size."""
    small_steps_case(21, 200, lambda beta: beta * step)


def test_chunks_of_steps_of_every_size():
    """Steps from 2^-30 to 1 in one chunk, the large ones forgotten behind decays of e^-8 and more."""
    gen = torch.Generator().manual_seed(3)

    def spread(beta):
        return torch.exp2(-30 * torch.rand(beta.shape, generator=gen)).cuda()

    small_steps_case(22, 200, spread)
    small_steps_case(23, 150, spread, rate=(2.0, 5.0))


@pytest.mark.parametrize("k_norm", [1e-2, 30.0, 200.0])
def test_chunks_of_keys_that_are_not_normalised(k_norm):
    """Keys and queries c times longer and steps c^2 times smaller: the recurrence of c = 1 with states c
    times smaller, so that the same bounds hold."""
    small_steps_case(24, 200, lambda beta: beta / k_norm ** 2, k_norm=k_norm)


@pytest.mark.parametrize("scale,v_scale", [(1e-6, 1000.0), (-1e-4, 50.0), (20.0, 1.0)])
def test_chunks_under_any_scale(scale, v_scale):
    """check() asks for 2^-25 beside the relative bounds; outputs here are at least a hundred times that."""
    small_steps_case(25, 130, lambda beta: beta, v_scale=v_scale, scale=scale)


@pytest.mark.parametrize("what", ["v", "k", "g", "beta", "q", "state"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("lens", [[3, 16, 5], [70, 150, 65]])
def test_what_is_not_finite_on_both_paths(what, bad, lens):
    """Up to 16 tokens a request and above: what a token's bad input does not reach is bit for bit as without it.
    What it reaches is NaN on the chunked path (a decay of minus infinity only forgets), and not finite on the
    other wherever an infinity is multiplied by nothing that is zero."""
    import ternary_hadamard_rotated_gb300 as tb

    Hk, Hv, req, head, col = 2, 4, 1, 3, 77
    x = dict(zip(("q", "k", "v", "g", "beta", "state"), make(40, lens, Hk, Hv, True)))
    row = lens[0] + lens[1] // 2
    T, B, end = sum(lens), len(lens), lens[0] + lens[1]
    chunked = max(lens) > 16

    def call(a):
        o = torch.empty(T, Hv, D, dtype=torch.float16, device="cuda")
        out = torch.empty_like(a["state"])
        tb.tb_gated_delta(a["q"], a["k"], a["v"], a["g"], a["beta"], starts(lens), max(lens), o, workspace(T, B, max(lens), Hk, Hv), state_in=a["state"],
                          state_out=out, normalise=True)
        torch.cuda.synchronize()
        return o, out

    want_o, want_s = call(x)
    y = {k: v.clone() for k, v in x.items()}
    if what == "state":
        y["state"][req, head, 5, col] = bad
        row = lens[0]
    elif what == "v":
        y["v"][row, head, col] = bad
    elif what in ("g", "beta"):
        y[what][row, head] = bad
    else:
        y[what][row, head // (Hv // Hk), 9] = bad
    o, s = call(y)
    touched = torch.zeros(T, Hv, D, dtype=torch.bool, device="cuda")
    state = torch.zeros(B, Hv, D, D, dtype=torch.bool, device="cuda")
    heads = slice(2, 4) if what in ("k", "q") else slice(head, head + 1)
    if what == "q":
        touched[row, heads] = True
    elif what in ("v", "state"):
        touched[row:end, head, col] = True
        state[req, head, :, col] = True
    else:
        touched[row:end, heads] = True
        state[req, heads] = True
    assert torch.equal(o[~touched], want_o[~touched])
    assert torch.equal(s[~state], want_s[~state])
    if what == "g" and bad < 0:  # forgets, and goes on
        assert torch.isfinite(o).all() and torch.isfinite(s).all()
        y["g"][row, head] = -1e4
        again_o, again_s = call(y)
        assert torch.equal(o, again_o) and torch.equal(s, again_s)
    elif chunked or bad != bad:
        assert torch.isnan(o[touched]).all() and torch.isnan(s[state]).all()
    else:
        assert not torch.isfinite(o[touched][:1]).any() and (what == "q" or not torch.isfinite(s[state]).all())


@pytest.mark.parametrize("grow", [3.0, 5.0, 7.0, 8.0])
@pytest.mark.parametrize("k_norm", [1.0, 50.0])
@pytest.mark.parametrize("n", [64, 128])
def test_chunks_of_steps_that_grow(grow, k_norm, n):
    """Steps with beta |k|^2 above 2, under which a state grows (over 64 tokens of random keys up to 10^4 times):
    the chunked path stays with the recurrent one as far as fp16 holds the outputs.  Both carry their rounding along
    with the growth, so that the bounds are those of check() times the largest growth of a step, grow - 1, and of
    the outputs as a whole."""
    import ternary_hadamard_rotated_gb300 as tb

    q, k, v, g, beta, _ = make(50, [n], 1, 2, False)
    k, q = (k.float() * k_norm).half(), (q.float() * k_norm).half()
    g = torch.full_like(g, -0.01)
    beta = torch.full_like(beta, grow / k_norm ** 2)
    want, fin, mag = mixers.gated_delta(*(x.cpu().numpy() for x in (q, k, v, g, beta)), [0, n], np.zeros((1, 2, D, D)), False, D ** -0.5)
    if np.abs(want).max() > 30000:
        pytest.skip("outputs past fp16")
    o = torch.empty(n, 2, D, dtype=torch.float16, device="cuda")
    out = torch.empty(1, 2, D, D, device="cuda")
    tb.tb_gated_delta(q, k, v, g, beta, starts([n]), n, o, workspace(n, 1, n, 1, 2), state_out=out, normalise=False)
    assert torch.isfinite(o).all() and torch.isfinite(out).all()
    err = np.abs(o.double().cpu().numpy() - want)
    tol = 2.0 ** -11 * np.abs(want) + (grow - 1) * 3 * 2.0 ** -11 * mag + 2.0 ** -25
    assert (err <= tol).all(), float((err / tol).max())
    assert np.linalg.norm(out.double().cpu().numpy() - fin) <= (grow - 1) * 2.0 ** -17 * np.linalg.norm(fin)
