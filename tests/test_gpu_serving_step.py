"""The operators around the linears together, as a decode step uses them: a packed linear with adapters beside it, the
positions on the way to the cache, attention over the cache, the linears behind it, and the logits.

Each stage is looked at from its own inputs in 64 bits, with the tolerance of its own tests, and the captured step gives
what the calls one by one give, bit by bit, for other tokens, adapters and histories too."""
import os
import importlib.util

import numpy as np
import pytest

from oracle import mixers, serving

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def hybrid():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layers.py")
    spec = importlib.util.spec_from_file_location("hybrid_layers", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


B, HIDDEN, HQ, HK, D, ROT, PAGE, N_ADAPT, RANK, VOCAB = 5, 1024, 8, 2, 64, 32, 16, 3, 16, 3000


class DecodeStep:
    """One token for each of B requests through an attention layer and the lm_head, in buffers of its own."""

    def __init__(self, seed):
        import ternary_hadamard_rotated_gb300 as tb

        h = hybrid()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.tb = tb
        self.qkv, self.out = h.Linear(HIDDEN, (HQ + 2 * HK) * D, gen, N_ADAPT, RANK), h.Linear(1024, HIDDEN, gen, N_ADAPT, RANK)
        self.head = h.Linear(HIDDEN, VOCAB, gen)
        self.mix = (torch.randn(HQ * D, 1024, generator=gen, device="cuda") * 0.05).half()  # (the heads' 512 to a folded width)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.x = torch.randn(B, HIDDEN, generator=gen, device="cuda").half()
        self.adapter, self.rows = i32(B), torch.arange(B + 1, dtype=torch.int32, device="cuda")
        self.cached, self.fresh = torch.tensor([0, 31, 16, 200, 5], dtype=torch.int32, device="cuda"), i32(B) + 1
        pages = 40
        perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        self.table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(self.cached.tolist()):
            n = -(-c // PAGE)
            self.table[b, :n] = perm[at: at + n]
            at += n
        self.free = perm[at:].contiguous()
        self.k_cache, self.v_cache = (torch.randn(pages, HK, PAGE, D, generator=gen, device="cuda").half() for _ in range(2))
        self.slots, self.total, self.starts = torch.zeros(B, dtype=torch.int64, device="cuda"), i32(B), i32(B + 1)
        self.rotary = torch.empty(tb.tb_rotary_plan_size(ROT), dtype=torch.uint8, device="cuda")
        tb.tb_rotary_plan(self.rotary, ROT, base=1e6, scaling=tb.TB_ROTARY_PARTS, factor=4.0, original=64.0)
        self.plan = torch.empty(tb.tb_adapter_plan_size(B, N_ADAPT), dtype=torch.uint8, device="cuda")
        self.history = torch.from_numpy(rng.integers(0, VOCAB, (B, 50)).astype(np.int32)).cuda()
        self.hist_len, self.prompt_len = i32(B) + 50, i32(B) + 20
        self.repetition, self.presence = torch.full((B,), 1.2, device="cuda"), torch.full((B,), 0.5, device="cuda")
        self.mask = torch.from_numpy(rng.integers(0, 2 ** 32, (2, -(-VOCAB // 32)), dtype=np.uint32).view(np.int32)).cuda()
        self.mask_row = torch.tensor([-1, 0, -1, 1, 0], dtype=torch.int32, device="cuda")
        self.status = i32(1)
        self.y, self.o = torch.empty(B, (HQ + 2 * HK) * D, dtype=torch.float16, device="cuda"), torch.empty(B, HQ, D, dtype=torch.float16, device="cuda")
        self.h, self.logits = torch.empty(B, HIDDEN, dtype=torch.float16, device="cuda"), torch.empty(B, VOCAB, dtype=torch.float16, device="cuda")
        self.raw, self.adjusted = torch.empty_like(self.logits), torch.empty(B, VOCAB, device="cuda")
        self.plain_y, self.turned = torch.empty_like(self.y), torch.empty(B, HQ, D, dtype=torch.float16, device="cuda")
        ws = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws_linear = {m: ws(tb.tb_packed_linear_workspace_size(B, m.K, m.N)) for m in (self.qkv, self.out, self.head)}
        self.ws_adapter = ws(max(tb.tb_adapter_linear_workspace_size(B, N_ADAPT, m.K, m.N, RANK) for m in (self.qkv, self.out)))
        self.ws_attn = ws(tb.tb_tree_attention_workspace_size(B, B, 1, HQ, HK, D))

    def linear(self, m, x, y):
        self.tb.tb_packed_linear(x, m.signs, 1024, m.w, m.scales, m.biases, y, self.ws_linear[m])

    def run(self):
        tb, st = self.tb, self.status
        tb.tb_adapter_plan(self.rows, self.adapter, B, N_ADAPT, self.plan, st)
        self.linear(self.qkv, self.x, self.plain_y)
        tb.tb_adapter_linear(self.x, self.qkv.a, self.qkv.b, self.qkv.adapter_scales, self.plan, self.plain_y, self.ws_adapter, out=self.y, dev_status=st)
        q, k, v = (t.unflatten(1, (-1, D)) for t in self.y.split([HQ * D, HK * D, HK * D], 1))
        tb.tb_cache_plan(self.cached, self.fresh, PAGE, self.free, self.table, self.slots, self.starts, self.total, dev_status=st)
        tb.tb_rotary_cache_write(q, k, v, self.cached, self.slots, self.rotary, ROT, tb.TB_ROTARY_PAIRS, self.turned, self.k_cache, self.v_cache, dev_status=st)
        tb.tb_tree_attention(self.turned, self.k_cache, self.v_cache, self.table, self.total, self.starts, 1, self.o, self.ws_attn, dev_status=st)
        self.wide = torch.matmul(self.o.flatten(1), self.mix)
        self.linear(self.out, self.wide, self.h)
        self.h0 = self.h.clone()
        tb.tb_adapter_linear(self.wide, self.out.a, self.out.b, self.out.adapter_scales, self.plan, self.h, self.ws_adapter, dev_status=st)  # in place
        self.linear(self.head, self.h, self.raw)
        tb.tb_logits_adjust(self.raw, self.adjusted, self.history, self.hist_len, self.prompt_len, repetition=self.repetition, presence=self.presence, mask=self.mask,
                            mask_row=self.mask_row, dev_status=st)
        return self.y, self.turned, self.o, self.h, self.raw, self.adjusted


def numpy(t):
    return t.detach().cpu().numpy()


def adapters_close(got, x, m, adapter, y):
    want, S, H = serving.adapter_linear(numpy(x), numpy(m.a), numpy(m.b), numpy(m.adapter_scales), None, list(range(B + 1)), adapter, numpy(y))
    tol = (m.K / 8 + RANK / 8 + 80) * 2.0 ** -23 * S + 2.0 ** -21 * H + 2.0 ** -11 * np.abs(want) + 2.0 ** -25  # as in the adapters' tests
    assert (np.abs(numpy(got).astype(np.float64) - want) <= tol).all()


def test_decode_step():
    s = DecodeStep(3)
    adapter = [0, 2, -1, 2, 1]
    s.adapter.copy_(torch.tensor(adapter, dtype=torch.int32))
    before = numpy(s.k_cache), numpy(s.v_cache)
    s.run()
    torch.cuda.synchronize()
    assert int(s.status) == 0
    adapters_close(s.y, s.x, s.qkv, adapter, s.plain_y)
    # positions and cache
    f, amp = serving.rotary_freqs(ROT, 1e6, "parts", 4.0, 64.0)
    y = numpy(s.y).reshape(B, HQ + 2 * HK, D)
    pos = numpy(s.cached)
    for part, got in ((y[:, :HQ], numpy(s.turned)), (y[:, HQ: HQ + HK], None)):
        want, size = serving.rotary(part, pos, f, amp, ROT, True)
        if got is None:
            kc = numpy(s.k_cache)
            got = np.stack([kc[i // PAGE, :, i % PAGE] for i in numpy(s.slots)])
            turned_k = got
        assert (np.abs(got.astype(np.float64) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -20 * size).all()  # as in the positions' tests
    kc, vc = mixers.cache_write(turned_k, y[:, HQ + HK:], numpy(s.slots), *before)
    assert np.array_equal(kc, numpy(s.k_cache)) and np.array_equal(vc, numpy(s.v_cache))
    # attention's own tests hold its tolerance; here: a softmax over the right keys (fp16 output, weights of 11 bits)
    o, _ = mixers.tree_attention(numpy(s.turned).astype(np.float64), kc.astype(np.float64), vc.astype(np.float64), numpy(s.table), numpy(s.total), list(range(B + 1)), None, D ** -0.5)
    assert np.abs(numpy(s.o) - o).max() <= 2.0 ** -8 * np.abs(vc).max()
    adapters_close(s.h, s.wide, s.out, adapter, s.h0)
    # logits: the same steps in fp32 give the same bits
    want = serving.logits_adjust(numpy(s.raw), list(range(B + 1)), numpy(s.history), numpy(s.hist_len), numpy(s.prompt_len), repetition=numpy(s.repetition),
                                 presence=numpy(s.presence), mask=numpy(s.mask), mask_row=numpy(s.mask_row), dtype=np.float32)
    assert np.array_equal(numpy(s.adjusted), want)


def test_decode_step_in_a_graph():
    s, other = DecodeStep(5), DecodeStep(5)
    s.run()  # (the library's first calls on a device)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    rng = np.random.default_rng(1)
    for step in range(3):
        new = [int(v) for v in rng.integers(-1, N_ADAPT, B)]
        for t in (s, other):
            t.adapter.copy_(torch.tensor(new, dtype=torch.int32))
            t.x.copy_(torch.from_numpy(np.random.default_rng(step).standard_normal((B, HIDDEN)).astype(np.float16)))
            t.history.copy_(torch.from_numpy(np.random.default_rng(step + 9).integers(0, VOCAB, (B, 50)).astype(np.int32)))
            t.hist_len.fill_(step * 20)
            t.prompt_len.fill_(step)
        g.replay()
        want = other.run()
        torch.cuda.synchronize()
        for a, b in zip((s.y, s.turned, s.o, s.h, s.raw, s.adjusted), want):
            assert torch.equal(a, b)
        assert torch.equal(s.k_cache, other.k_cache) and torch.equal(s.v_cache, other.v_cache)
    assert int(s.status) == 0 and int(other.status) == 0


def test_example_logits():
    """The example's rows of drafts against the same tokens put into the history."""
    h = hybrid()
    layers = h.HybridLayers(hidden=1024, key_heads=2, value_heads=8, heads=8, kv_heads=2, dim=128, page=16, pages=16, max_pages=8, requests=2, vocab=777)
    x = torch.randn(5, 1024, device="cuda").half()
    history = [[1, 5, 5, 700], [3]]
    parents = [[-1, 0, 0], [-1, 0]]
    drafts = [[9, 5, 12], [3, 3]]
    pen = dict(repetition=torch.tensor([1.5, 1.0], device="cuda"), frequency=torch.tensor([0.5, 0.25], device="cuda"))
    got = layers.next_logits(x, history, [2, 1], lens=[3, 2], fresh=sum(drafts, []), tree=h.tree_words(parents), **pen)
    assert int(layers.status) == 0
    row = 0
    for b, p in enumerate(parents):
        for i in range(len(p)):
            path, q = [], i
            while q >= 0:
                path.insert(0, drafts[b][q])
                q = p[q]
            one = layers.next_logits(x, [history[b] + path], [[2, 1][b]], lens=[5], **{k: v[b: b + 1] for k, v in pen.items()})
            assert torch.equal(one[row], got[row])
            row += 1


def test_two_calls_at_once_on_two_streams():
    """Each operator on two streams at a time, with outputs and workspaces of their own and the same plans."""
    import ternary_hadamard_rotated_gb300 as tb

    gen = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()  # noqa: E731
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    T, K, N, R, V = 900, 640, 512, 64, 50000
    turns = torch.empty(tb.tb_rotary_plan_size(64), dtype=torch.uint8, device="cuda")
    tb.tb_rotary_plan(turns, 64)
    grouped = torch.empty(tb.tb_adapter_plan_size(T, 3), dtype=torch.uint8, device="cuda")
    tb.tb_adapter_plan(ints(0, 300, 700, 900), ints(2, 0, 1), T, 3, grouped)
    q, k, pos = randn(T, 8, 128), randn(T, 2, 128), torch.arange(T, dtype=torch.int32, device="cuda")
    x, y, a, b, scale = randn(T, K), randn(T, N), randn(3, R, K) * 0.05, randn(3, N, R), torch.ones(3, device="cuda")
    logits, history = randn(20, V), torch.randint(0, V, (20, 9000), generator=gen, dtype=torch.int32, device="cuda")
    lengths, rate = torch.full((20,), 9000, dtype=torch.int32, device="cuda"), torch.rand(20, generator=gen, device="cuda")
    outs = []
    for _ in range(3):
        ws = torch.empty(tb.tb_adapter_linear_workspace_size(T, 3, K, N, R), dtype=torch.uint8, device="cuda")
        outs.append((torch.empty_like(q), torch.empty_like(k), torch.empty_like(y), torch.empty(20, V, device="cuda"), ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), None]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        if s is None:
            torch.cuda.synchronize()  # the last by itself
        tb.tb_adapter_linear(x, a, b, scale, grouped, y, o[4], out=o[2], stream=s)
        tb.tb_logits_adjust(logits, o[3], history, lengths, frequency=rate, stream=s)
        tb.tb_rotary(q, k, pos, turns, 64, tb.TB_ROTARY_HALF, o[0], o[1], stream=s)
    torch.cuda.synchronize()
    for o in outs[:2]:
        for mine, alone in zip(o[:4], outs[2]):
            assert torch.equal(mine, alone)


def test_calls_behind_copies_kernels_and_other_streams():
    """Each first launch may be set up before what is in front of it is over: its inputs are written by a copy, by a kernel, by
    a kernel of another stream that is waited for, and by the operators themselves, one after another and in a graph."""
    import ternary_hadamard_rotated_gb300 as tb

    gen = torch.Generator(device="cuda").manual_seed(4)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda").half()  # noqa: E731
    T, K, N, R, V = 300, 512, 4096, 16, 4096
    turns = torch.empty(tb.tb_rotary_plan_size(64), dtype=torch.uint8, device="cuda")
    tb.tb_rotary_plan(turns, 64)
    a, b, scale = randn(3, R, K) * 0.05, randn(3, N, R), torch.ones(3, device="cuda")
    rows = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    history, lengths = torch.randint(0, V, (T, 50), generator=gen, dtype=torch.int32, device="cuda"), torch.full((T,), 50, dtype=torch.int32, device="cuda")
    rate = torch.rand(T, generator=gen, device="cuda")
    sources = [(randn(T, K), randn(T, N), torch.tensor(ids, dtype=torch.int32, device="cuda"), torch.randint(0, 9999, (T,), generator=gen, dtype=torch.int32, device="cuda"))
               for ids in ([0, 1, 2], [2, -1, 0], [1, 1, -1], [0, 2, 0])]
    x, y, ids, pos = (torch.zeros_like(m) for m in sources[0])
    plan = torch.empty(tb.tb_adapter_plan_size(T, 3), dtype=torch.uint8, device="cuda")
    ws = torch.empty(tb.tb_adapter_linear_workspace_size(T, 3, K, N, R), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def step(source, out, settle):
        now = torch.cuda.current_stream()
        x.copy_(source[0])
        torch.add(source[1], 0, out=y)
        side.wait_stream(now)
        with torch.cuda.stream(side):
            pos.copy_(source[3])
            torch.add(source[2], 0, out=ids)
        now.wait_stream(side)
        settle()
        tb.tb_adapter_plan(rows, ids, T, 3, plan)
        settle()
        tb.tb_adapter_linear(x, a, b, scale, plan, y, ws)
        settle()
        q = y.view(T, N // 128, 128)
        tb.tb_rotary(q, None, pos, turns, 64, tb.TB_ROTARY_HALF, q, None)
        settle()
        tb.tb_logits_adjust(y[:, :V], out, history, lengths, frequency=rate)

    alone = [torch.empty(T, V, device="cuda") for _ in sources]
    for s, o in zip(sources, alone):
        step(s, o, torch.cuda.synchronize)
    torch.cuda.synchronize()
    row = [torch.empty(T, V, device="cuda") for _ in sources * 5]
    for i, o in enumerate(row):
        step(sources[i % 4], o, lambda: None)
    torch.cuda.synchronize()
    assert all(torch.equal(o, alone[i % 4]) for i, o in enumerate(row))
    captured = [torch.empty(T, V, device="cuda") for _ in sources]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for s, o in zip(sources, captured):
            step(s, o, lambda: None)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(captured, alone))
