"""GPU parity of the logits' penalties, biases and masks: every step is one fp32 operation rounded as written, so
the same steps in NumPy's fp32 give the same bits, and fp16 outputs are those rounded once.  Against 64 bits each
of the six operations is off by at most 2^-24 of its result, and what comes before it by as much as it was: the
result by at most 2^-21 of the sum of the absolute values of all terms."""
import numpy as np
import pytest

from oracle import serving

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def case(rng, lens, V, L, hist_hi, biases=0, grammar=0.0, tree=False, fresh=False, pad=0):
    """Arguments by name, as NumPy arrays (logits with pad columns behind V)."""
    B, T = len(lens), sum(lens)
    ids = lambda *s: np.minimum(np.exp(rng.random(s) * np.log(V)) - 1, V - 1).astype(np.int32)  # noqa: E731
    c = dict(logits=(rng.standard_normal((T, V + pad)) * 4).astype(np.float16), row_start=np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), history=ids(B + 2, L),
             slot=rng.permutation(B + 2)[:B].astype(np.int32), hist_len=rng.integers(0, hist_hi + 1, B).astype(np.int32))
    c["prompt_len"] = (c["hist_len"] * rng.random(B)).astype(np.int32)
    c["repetition"] = np.where(rng.random(B) < 0.2, 1, 1 + rng.random(B)).astype(np.float32)
    c["presence"], c["frequency"] = rng.standard_normal(B).astype(np.float32), rng.random(B).astype(np.float32)
    if fresh or tree:
        c["fresh"] = ids(T)
    if tree:
        words = []
        for n in lens:
            own = []
            for i in range(n):
                p = int(rng.integers(-1, i)) if i else -1
                own.append((1 << i) | (own[p] if p >= 0 else 0))
            words += own
        c["tree"] = np.array([w - (1 << 64) if w >> 63 else w for w in words], dtype=np.int64)
    if biases:
        c["biases"] = [[(int(v), float(np.float32(rng.standard_normal()))) for v in rng.choice(V, size=min(V, int(rng.integers(0, biases + 1))), replace=False)] for _ in lens]
    if grammar:
        rows = np.where(rng.random(T) < grammar, rng.integers(0, T, T), -1).astype(np.int32)
        c["mask"], c["mask_row"] = rng.integers(0, 2 ** 32, (T, -(-V // 32)), dtype=np.uint32).view(np.int32), rows
    return c


def lists(biases):
    """The requests' lists as bias_start, bias_ids, bias_values."""
    flat = [e for row in biases for e in row]
    return (np.concatenate([[0], np.cumsum([len(row) for row in biases])]).astype(np.int32), np.array([v for v, _ in flat], dtype=np.int32).reshape(-1),
            np.array([w for _, w in flat], dtype=np.float32).reshape(-1))


def run(c, V, out_type, in_place=False, pad_out=0):
    import ternary_hadamard_rotated_gb300 as tb

    d = {k: torch.from_numpy(v).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    if "biases" in c:
        d["bias_start"], d["bias_ids"], d["bias_values"] = (torch.from_numpy(m).cuda() for m in lists(c["biases"]))
    x = d.pop("logits")
    T = x.shape[0]
    out = x if in_place else torch.full((T + 1, V + pad_out), 77.0, dtype=out_type, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = x.clone()
    tb.tb_logits_adjust(x[:, :V], out[:T, :V], d.pop("history"), d.pop("hist_len"), dev_status=st, **d)
    torch.cuda.synchronize()
    if in_place:
        assert torch.equal(out[:, V:], before[:, V:])
    else:
        assert torch.equal(x.view(torch.int16), before.view(torch.int16)) and (out[T] == 77).all() and (out[:, V:] == 77).all()
    return out[:T, :V].cpu().numpy(), int(st)


def expect(c, V, dtype):
    args = {k: v for k, v in c.items() if k not in ("logits", "row_start", "history", "hist_len")}
    return serving.logits_adjust(c["logits"][:, :V], c["row_start"], c["history"], c["hist_len"], dtype=dtype, **args)


def same(got, want):
    want = want.astype(got.dtype)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want[ok])


@pytest.mark.parametrize("lens,V,L,hist_hi,kw", [
    ([1], 248320, 900, 700, {}), ([1], 1, 3, 3, dict(biases=1, grammar=1.0)), ([1, 1, 1], 31, 40, 40, dict(biases=9, grammar=0.7)),
    ([1] * 9, 50257, 3000, 3000, dict(biases=300, grammar=0.5, pad=7)), ([1] * 3, 8192, 0, 0, dict(biases=5)), ([1] * 2, 131072, 40000, 40000, dict(pad=64)),
    ([4, 0, 1, 9], 32000, 500, 500, dict(tree=True, grammar=0.3)), ([64, 3], 1000, 100, 100, dict(tree=True, biases=4)), ([5, 2], 300007, 60, 60, dict(fresh=True, biases=1000)),
    ([1] * 200, 129, 20, 20, dict(grammar=0.5)), ([1] * 6, 8200, 64, 64, dict(fresh=True, biases=20, pad=8)),
    ([1] * 64, 50000, 300, 300, dict(grammar=0.6)), ([7, 50, 30], 50003, 5000, 5000, dict(grammar=0.6, tree=True, biases=2000, pad=5))])
@pytest.mark.parametrize("kind", ["half", "float", "in place"])
def test_logits_match(lens, V, L, hist_hi, kw, kind):
    rng = np.random.default_rng(V + L)
    c = case(rng, lens, V, L, hist_hi, **kw)
    got, st = run(c, V, torch.float32 if kind == "float" else torch.float16, kind == "in place", pad_out=kw.get("pad", 0) if kind == "half" else 0)
    assert st == 0
    same(got, expect(c, V, np.float32))
    if kind == "float":
        want = expect(c, V, np.float64)
        count = c["frequency"].max() * (hist_hi + 64) + np.abs(c["presence"]).max() + 8
        ok = np.isfinite(want)
        assert np.array_equal(got[~ok], want[~ok])
        size = np.abs(want[ok]) + 2 * np.abs(c["logits"][:, :V][ok].astype(np.float64)) + count
        assert (np.abs(got[ok] - want[ok]) <= 2.0 ** -21 * size).all()


def test_each_part_alone():
    rng = np.random.default_rng(1)
    whole = case(rng, [1, 1, 1], 999, 50, 50, biases=30, grammar=1.0, fresh=True)
    base = ("logits", "row_start", "history", "hist_len")
    for part in (("repetition",), ("presence",), ("frequency", "prompt_len"), ("biases",), ("mask", "mask_row"), ("slot", "repetition"), ("fresh", "presence"), ()):
        c = {k: whole[k] for k in base + part}
        got, st = run(c, 999, torch.float32)
        assert st == 0
        same(got, expect(c, 999, np.float32))
    c = {k: whole[k] for k in base + ("mask", "fresh", "frequency")}
    del c["row_start"]  # a row a request, masks by row
    got, st = run(c, 999, torch.float16)
    c["row_start"] = whole["row_start"]
    assert st == 0
    same(got, expect(c, 999, np.float32))


def test_what_is_not_finite_and_rows_without_a_token():
    rng = np.random.default_rng(2)
    c = case(rng, [1, 1, 1, 1], 500, 30, 30, grammar=1.0)
    c["mask_row"][:] = [0, 1, 2, -1]
    c["mask"][1], c["mask"][2] = 0, -1  # nothing is left; everything is
    c["logits"][:, ::5] = np.nan
    c["logits"][:, 1::5] = np.inf
    c["logits"][:, 2::5] = -np.inf
    c["logits"][3, :4] = [65504, -65504, 6e-8, -0.0]
    got, st = run(c, 500, torch.float16)
    assert st == 0 and (got[1] == -np.inf).all()
    same(got, expect(c, 500, np.float32))
    bits = np.unpackbits(c["mask"][0].view(np.uint8), bitorder="little")[:500]
    assert (got[0][bits == 0] == -np.inf).all()


def test_a_token_listed_twice_takes_the_last_bias():
    rng = np.random.default_rng(3)
    c = case(rng, [1, 1], 700, 10, 10)
    c["biases"] = [[(5, 1.0), (9, 2.0), (5, -3.0), (5, 0.25)] + [(600, float(i)) for i in range(300)], [(5, 7.0), (5, float("-inf"))]]
    got, st = run(c, 700, torch.float32)
    assert st == 0
    same(got, expect(c, 700, np.float32))


def test_counts_above_sixteen_bits():
    V, n = 1000, 200000
    h = np.full((1, n), 7, dtype=np.int32)
    h[0, ::2] = 8
    c = dict(logits=np.ones((1, V), dtype=np.float16), row_start=np.array([0, 1], dtype=np.int32), history=h, hist_len=np.array([n], dtype=np.int32),
             prompt_len=np.array([3], dtype=np.int32), frequency=np.array([0.125], dtype=np.float32))
    got, st = run(c, V, torch.float32)
    assert st == 0 and got[0, 7] == 1 - 0.125 * (n // 2 - 1) and got[0, 8] == 1 - 0.125 * (n // 2 - 2) and got[0, 9] == 1


@pytest.mark.parametrize("V,biased", [(300007, 0), (40000, 40000), (248320, 5000)])
def test_every_token_in_the_history(V, biased):
    """More different tokens than the tables of a request's CTAs take at once."""
    rng = np.random.default_rng(V)
    c = case(rng, [2, 1], V, 2 * V, 1, fresh=True)
    for r in range(c["history"].shape[0]):
        c["history"][r] = rng.permutation(np.concatenate([np.arange(V), rng.integers(0, V, V)]))
    c["hist_len"][:] = [2 * V, V + V // 2]
    c["prompt_len"][:] = [V // 3, V]
    if biased:
        c["biases"] = [[(int(v), float(i % 7) - 3) for i, v in enumerate(rng.permutation(V)[:biased])], []]
    got, st = run(c, V, torch.float32)
    assert st == 0
    same(got, expect(c, V, np.float32))


def test_what_does_not_fit_is_left_out_and_flagged():
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(4)

    def flagged(want, change, same_as=None, **kw):
        c = case(rng, [1, 1, 1], 300, 20, 20, **kw)
        c["hist_len"][:] = [20, 7, 0]
        c["prompt_len"][:] = [3, 7, 0]
        clean = {k: v.copy() for k, v in c.items()}
        change(c)
        if same_as:
            same_as(clean)
        got, st = run(c, 300, torch.float32)
        assert st == want
        same(got, expect(clean, 300, np.float32))

    def put(name, at, value):
        return lambda c: c[name].__setitem__(at, value)

    def history(at, value):  # in the first request's row
        return lambda c: c["history"].__setitem__((c["slot"][0], at), value)

    flagged(0, history(4, -1), history(4, -1))  # padding
    flagged(tb.TB_DEV_BAD_ID, history(4, 300), history(4, -1))
    flagged(tb.TB_DEV_BAD_ID, put("slot", 1, 5), put("hist_len", 1, 0))
    flagged(0, put("slot", 0, -1), put("slot", 0, -1))
    flagged(tb.TB_DEV_BAD_LEN, put("hist_len", 0, 21), put("hist_len", 0, 20))
    flagged(tb.TB_DEV_BAD_LEN, put("hist_len", 1, -5), put("hist_len", 1, 0))
    flagged(tb.TB_DEV_BAD_LEN, put("prompt_len", 1, 9), put("prompt_len", 1, 7))
    flagged(tb.TB_DEV_BAD_LEN, put("prompt_len", 0, -2), put("prompt_len", 0, 0))
    flagged(tb.TB_DEV_BAD_ID, put("mask_row", 1, 3), put("mask_row", 1, -1), grammar=0.5)
    flagged(tb.TB_DEV_BAD_ID, put("fresh", 0, 300), put("fresh", 0, -1), fresh=True)
    flagged(tb.TB_DEV_BAD_ID, lambda c: c["biases"].__setitem__(0, [(300, 1.0), (4, 1.0), (-1, 2.0)]), lambda c: c["biases"].__setitem__(0, [(4, 1.0)]), biases=3)


def test_row_starts_that_do_not_fit():
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(5)
    for rows, live in (([2, 5, 7], range(2, 7)), ([0, 9, 7], []), ([-4, 3, 8], range(3, 8)), ([0, 3, 200], range(0, 3)), ([0, 2 ** 31 - 1, -2 ** 31], [])):
        c = case(rng, [4, 4], 100, 20, 20, fresh=True)
        c["row_start"] = np.array(rows, dtype=np.int32)
        got, st = run(c, 100, torch.float32)
        assert st == (0 if rows[0] == 2 else tb.TB_DEV_BAD_LEN)
        rest = [t for t in range(8) if t not in live]
        assert (got[rest] == 77).all()
        for b in range(2):
            r = [t for t in live if rows[b] <= t < rows[b + 1]]
            if r:
                one = {k: v for k, v in c.items() if k != "row_start"}
                for k in ("hist_len", "slot", "prompt_len", "repetition", "presence", "frequency"):
                    one[k] = one[k][b: b + 1]
                one["logits"], one["fresh"], one["row_start"] = one["logits"][r], one["fresh"][r], np.array([0, len(r)])
                same(got[r], expect(one, 100, np.float32))


def test_more_than_sixty_four_fresh_tokens():
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(6)
    c = case(rng, [70], 400, 20, 20, fresh=True)
    got, st = run(c, 400, torch.float32)
    assert st == tb.TB_DEV_BAD_LEN
    c["fresh"][64:] = -1
    same(got, expect(c, 400, np.float32))


def test_graph_and_stream():
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(7)
    V = 20000
    c = case(rng, [1, 1], V, 64, 64)
    d = {k: torch.from_numpy(v).cuda() for k, v in c.items()}
    x, out = d.pop("logits"), torch.empty(2, V, device="cuda")
    h, n = d.pop("history"), d.pop("hist_len")
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        tb.tb_logits_adjust(x, out, h, n, **d)
    for _ in range(2):
        c["hist_len"] = rng.integers(0, 65, 2).astype(np.int32)
        c["prompt_len"] = np.zeros(2, dtype=np.int32)
        n.copy_(torch.from_numpy(c["hist_len"]))
        d["prompt_len"].zero_()
        g.replay()
        torch.cuda.synchronize()
        same(out.cpu().numpy(), expect(c, V, np.float32))


def test_rows_past_two_to_the_31_elements():
    import ternary_hadamard_rotated_gb300 as tb

    T, V = 8700, 248320  # 4.3 GB
    x = torch.zeros(T, V, dtype=torch.float16, device="cuda")
    x[-1] = 1
    h = torch.tensor([[5, V - 1, 5]], dtype=torch.int32, device="cuda")
    row_start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    tb.tb_logits_adjust(x, x, h, torch.tensor([3], dtype=torch.int32, device="cuda"), row_start=row_start, frequency=torch.tensor([0.25], device="cuda"))
    want = torch.ones(V)
    want[5], want[V - 1] = 0.5, 0.75
    assert torch.equal(x[-1].cpu().float(), want) and float(x[0, 5]) == -0.5
