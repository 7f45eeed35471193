"""The operators around the packed linears of a serving step, case by case: rotary positions on the way to the
cache, low-rank adapters of many requests, and the logits' penalties, biases and grammar masks.

``listed()`` gives the cases that are timed, ``draw(rng)`` more of the same ranges, ``prepare`` the tensors a
serving program holds before the call, ``run`` one pass, ``work`` the bytes and operations that the pass cannot
do without, and ``exact`` the outputs in 64 bits.  With ``own`` set, ``run`` calls the library; otherwise it
computes the operator from elementary torch operations in 32 bits (angles in 64), rounded once at the end.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    full = dict(op="rotary", heads=24, kv_heads=4, dim=256, rot=64, layout="half", base=1e7, page=64, inverse=False)  # the hybrid model's attention layer
    return [
        # one user, one token: q turned, k turned into its slot, v beside it
        dict(full, name="rotary-one", cache=True, tokens=1, run=1, past=4097, scaling="none", factor=1.0, mix=1),
        # one token for each of 64 requests far into contexts that were scaled by parts
        dict(full, name="rotary-decode", cache=True, tokens=64, run=1, past=260000, scaling="parts", factor=8.0, mix=2),
        # packed prompts on their way to prompt attention and the cache
        dict(full, name="rotary-prompts", cache=True, tokens=12289, run=1777, past=0, scaling="none", factor=1.0, mix=3),
        # whole heads in pairs of neighbours, without a cache
        dict(full, name="rotary-long", cache=False, heads=32, kv_heads=8, dim=128, rot=128, layout="pairs", tokens=40001, run=40001, past=0, scaling="linear",
             factor=4.0, mix=4),
        # one user's adapter beside the gate projection
        dict(name="adapter-one", op="adapter", batch=1, q_lo=1, q_hi=1, adapters=1, bare=0.0, shapes=1, k0=5120, n0=17408, rank=16, ranks=False, plan=False, mix=5),
        # one token for each of 64 requests, most with an adapter of their own
        dict(name="adapter-decode", op="adapter", batch=64, q_lo=1, q_hi=1, adapters=100, bare=0.1, shapes=1, k0=5120, n0=17408, rank=32, ranks=True, plan=False, mix=6),
        # verification of drafts, few adapters: the step's plan and every linear of one layer
        dict(name="adapter-layer", op="adapter", batch=24, q_lo=3, q_hi=8, adapters=7, bare=0.2, shapes=4, k0=5120, n0=8192, k1=6144, n1=5120, k2=5120, n2=34816,
             k3=17408, n3=5120, rank=16, ranks=False, plan=True, mix=7),
        # packed prompts of mixed lengths, each with its adapter
        dict(name="adapter-prompts", op="adapter", batch=13, q_lo=20, q_hi=1500, adapters=9, bare=0.1, shapes=1, k0=5120, n0=17408, rank=64, ranks=True, plan=False,
             mix=8),
        # one long prompt
        dict(name="adapter-long", op="adapter", batch=1, q_lo=8192, q_hi=8192, adapters=3, bare=0.0, shapes=1, k0=17408, n0=5120, rank=16, ranks=False, plan=False, mix=9),
        # one user's next token: penalties over a short conversation
        dict(name="logits-one", op="logits", batch=1, q_lo=1, q_hi=1, vocab=248320, pad=0, hist_lo=700, hist_hi=700, biases=0, grammar=0.0, wide=False, tree=False, mix=10),
        # a decoding batch, a third of it under grammars, some with biased tokens
        dict(name="logits-decode", op="logits", batch=64, q_lo=1, q_hi=1, vocab=248320, pad=0, hist_lo=30, hist_hi=8000, biases=300, grammar=0.3, wide=True, tree=False,
             mix=11),
        # verification of drafted trees over long conversations
        dict(name="logits-verify", op="logits", batch=9, q_lo=5, q_hi=16, vocab=248320, pad=0, hist_lo=2000, hist_hi=30000, biases=0, grammar=0.3, wide=False, tree=True,
             mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "adapter", "logits"])
    mix = rng.randrange(1 << 30)
    if op == "rotary":
        kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        scaling = rng.choice(["none", "linear", "base", "parts"]) if rot >= 8 else rng.choice(["none", "linear"])
        group = rng.choice([1, 3, 4, 6])
        tokens = min(_log(rng, 1, 40000), 150_000_000 // (kv * (group + 2) * dim))
        return dict(op=op, cache=rng.random() < 0.6, tokens=tokens, run=_log(rng, 1, 3000), past=rng.choice([0, 500, 100000]), heads=kv * group, kv_heads=kv, dim=dim,
                    rot=rot, layout=rng.choice(["half", "pairs"]), base=rng.choice([1e4, 5e5, 1e7]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 32.0]), page=rng.choice([16, 32, 64, 128, 256]), inverse=rng.random() < 0.25, mix=mix)
    if op == "adapter":
        long = rng.random() < 0.5
        batch, k, n = _log(rng, 1, 12 if long else 80), 8 * _log(rng, 16, 2176), 8 * _log(rng, 16, 2176)
        q_hi = min(_log(rng, 30, 8000), max(30, 150_000_000 // (batch * (k + n)))) if long else rng.choice([1, 1, 2, 9])
        return dict(op=op, batch=batch, q_lo=1, q_hi=q_hi, adapters=_log(rng, 1, 64), bare=rng.choice([0.0, 0.2]), shapes=1, k0=k, n0=n, rank=8 * rng.choice([1, 2, 2, 3, 4, 8, 8, 16]),
                    ranks=rng.random() < 0.5, plan=False, mix=mix)
    tree = rng.random() < 0.4
    return dict(op=op, batch=_log(rng, 1, 6 if tree else 48), q_lo=1, q_hi=_log(rng, 2, 20) if tree else 1, vocab=_log(rng, 1000, 248320), pad=rng.choice([0, 0, 5, 64]),
                hist_lo=0, hist_hi=_log(rng, 10, 30000), biases=rng.choice([0, 0, 7, 300]), grammar=rng.choice([0.0, 0.5, 1.0]), wide=rng.random() < 0.5, tree=tree, mix=mix)


def _lengths(case, name, salt=0):
    """The requests' lengths: spread over the logarithm between the case's bounds, the same in every pass."""
    rng = random.Random(case["mix"] * 8 + salt)
    lo, hi = case[name + "_lo"], case[name + "_hi"]
    return [lo if lo == hi else _log(rng, lo + 1, hi + 1) - 1 for _ in range(case["batch"])]


def _sums(values):
    out = [0]
    for v in values:
        out.append(out[-1] + v)
    return out


def _up(n, page):
    return -(-n // page)


def _adapters_of(case):
    """The requests' adapters (-1: none), and the adapters' ranks."""
    rng = random.Random(case["mix"] * 8 + 5)
    ids = [-1 if rng.random() < case["bare"] else rng.randrange(case["adapters"]) for _ in range(case["batch"])]
    ranks = [rng.choice([case["rank"], case["rank"] // 2, rng.randint(1, case["rank"])]) if case["ranks"] else case["rank"] for _ in range(case["adapters"])]
    return ids, ranks


def _masked(case):
    """Which rows are under a grammar: their rows of the mask, or -1."""
    rng = random.Random(case["mix"] * 8 + 6)
    rows, n = [], 0
    for f in _lengths(case, "q"):
        under = rng.random() < case["grammar"]
        rows += [n + i if under else -1 for i in range(f)]
        n += f if under else 0
    return rows, n


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).half()


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device=DEV)


def prepare(case, seed):
    return {"rotary": _prepare_rotary, "adapter": _prepare_adapter, "logits": _prepare_logits}[case["op"]](case, _gen(seed))


ORIGINAL = 8192  # context of the model before its positions were scaled


def _frequencies(case):
    """Radians a position of each pair, and the rotation's amplitude."""
    R, base, s = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "base":
        base = base * s ** (R / (R - 2))
    f = np.float64(base) ** (-2.0 * np.arange(R // 2) / R)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "parts":
        # the pair that turns `beta` times over the original context
        pair = lambda beta: R * math.log(ORIGINAL / (beta * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), R - 1)
        ramp = np.clip((np.arange(R // 2) - low) / max(high - low, 1e-3), 0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1.0
    return f, 1.0


def _prepare_rotary(case, gen):
    T, Hq, Hk, D, page, run_ = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"], case["run"]
    qkv = _randn(gen, T, (Hq + 2 * Hk) * D)  # the three projections side by side, as one packed linear leaves them
    q, k, v = (x.view(T, -1, D) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    t = torch.arange(T, device=DEV)
    begin = torch.randint(0, case["past"] + 1, (_up(T, run_),), generator=gen, device=DEV)
    pos = begin[t // run_] + t % run_
    f, amplitude = _frequencies(case)
    new = lambda like: torch.zeros(like.shape, dtype=torch.float16, device=DEV)  # noqa: E731
    state = dict(case=case, q=q, k=k, v=v, pos=pos.to(torch.int32), freq=torch.from_numpy(f).to(DEV), amplitude=amplitude, q_out=new(q))
    prompts = run_ > 1  # prompt attention reads k beside the cache
    state["k_out"] = new(k) if prompts or not case["cache"] else None
    if case["cache"]:
        per = _up(run_ + page - 1, page)
        pool = _up(T, run_) * per + 5
        first = torch.randint(0, page, (_up(T, run_),), generator=gen, device=DEV)
        at = first[t // run_] + t % run_
        state["slots"] = torch.randperm(pool, generator=gen, device=DEV)[t // run_ * per + at // page] * page + at % page
        state["k_cache"], state["v_cache"] = (torch.zeros(pool, Hk, page, D, dtype=torch.float16, device=DEV) for _ in range(2))
    if own:
        import ternary_hadamard_rotated_gb300 as tb
        kind = {"none": tb.TB_ROTARY_NONE, "linear": tb.TB_ROTARY_LINEAR, "base": tb.TB_ROTARY_BASE, "parts": tb.TB_ROTARY_PARTS}[case["scaling"]]
        state["layout"] = tb.TB_ROTARY_HALF if case["layout"] == "half" else tb.TB_ROTARY_PAIRS
        state["plan"] = torch.empty(tb.tb_rotary_plan_size(case["rot"]), dtype=torch.uint8, device=DEV)
        tb.tb_rotary_plan(state["plan"], case["rot"], base=case["base"], scaling=kind, factor=case["factor"], original=ORIGINAL)
    return state


def _shapes(case):
    return [(case["k%d" % i], case["n%d" % i]) for i in range(case["shapes"])]


def _prepare_adapter(case, gen):
    lens = _lengths(case, "q")
    ids, ranks = _adapters_of(case)
    T, n, R = sum(lens), case["adapters"], case["rank"]
    state = dict(case=case, tokens=T, lens=lens, ids=ids, ranks=ranks, row_start=_ints(_sums(lens)), adapter=_ints(ids), rank=_ints(ranks) if case["ranks"] else None,
                 scale=0.5 + 1.5 * _rand(gen, n), linears=[])
    for K, N in _shapes(case):
        a, b = _randn(gen, n, R, K, scale=K ** -0.5), _randn(gen, n, N, R, scale=0.3 * R ** -0.5)
        state["linears"].append(dict(a=a, b=b, x=_randn(gen, T, K), y=_randn(gen, T, N), out=torch.zeros(T, N, dtype=torch.float16, device=DEV)))
    if own:
        import ternary_hadamard_rotated_gb300 as tb
        state["plan"] = torch.empty(tb.tb_adapter_plan_size(T, n), dtype=torch.uint8, device=DEV)
        size = max(tb.tb_adapter_linear_workspace_size(T, n, K, N, R) for K, N in _shapes(case))
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        tb.tb_adapter_plan(state["row_start"], state["adapter"], T, n, state["plan"])  # once a step, for all its linears
    return state


def _prepare_logits(case, gen):
    fresh, hist = _lengths(case, "q"), _lengths(case, "hist", 1)
    B, V, T = case["batch"], case["vocab"], sum(fresh)
    words = lambda *shape: torch.exp(_rand(gen, *shape) * math.log(V)).long().clamp(1, V).sub(1).to(torch.int32)  # noqa: E731  frequent tokens have low numbers
    rng = random.Random(case["mix"] * 8 + 7)
    wide = _randn(gen, T, V + case["pad"], scale=3.0)
    state = dict(case=case, fresh_lens=fresh, logits=wide[:, :V], row_start=_ints(_sums(fresh)), history=words(B + 2, max(hist) + 1),
                 slot=torch.randperm(B + 2, generator=gen, device=DEV)[:B].to(torch.int32), hist_len=_ints(hist), prompt_len=_ints([rng.randint(0, h) for h in hist]),
                 repetition=torch.where(_rand(gen, B) < 0.3, 1.0, 1.0 + 0.3 * _rand(gen, B)), presence=_rand(gen, B), frequency=0.3 * _rand(gen, B),
                 drafts=None, words=None, bias_start=None, bias_ids=None, bias_values=None, mask=None, mask_row=None,
                 out=torch.zeros(T, V + case["pad"], dtype=torch.float32 if case["wide"] else torch.float16, device=DEV)[:, :V])
    if case["tree"]:
        state["drafts"], state["words"] = words(T), _trees(gen, fresh)
    if case["biases"]:
        lens = [rng.choice([0, 1, case["biases"]]) for _ in range(B)]
        n = sum(lens)
        i = _ints([j for m in lens for j in range(m)], torch.int64)
        off = torch.randint(0, V, (B,), generator=gen, device=DEV)[_ints([b for b, m in enumerate(lens) for _ in range(m)], torch.int64)]
        state["bias_start"], state["bias_ids"] = _ints(_sums(lens)), ((off + i * (V // case["biases"])) % V).to(torch.int32)  # no token twice in a request
        state["bias_values"] = torch.where(_rand(gen, n) < 0.1, -100.0, 4 * _rand(gen, n) - 2)
    rows, n = _masked(case)
    if n:
        # a grammar leaves a handful of tokens, half of them, or nearly all
        keep = _ints([rng.choice([1e-4, 0.5, 0.999]) for _ in range(n)], torch.float32)
        m = torch.empty(n, _up(V, 32), dtype=torch.int32, device=DEV)
        for r in range(n):
            bits = (_rand(gen, _up(V, 32) * 32) < keep[r]).view(-1, 32).long()
            m[r] = (bits << torch.arange(32, device=DEV)).sum(1).to(torch.int32)
        state["mask"], state["mask_row"] = m, _ints(rows)
    return state


def _trees(gen, fresh):
    """A random tree of drafted tokens for each request: bit j of a token's word says that token j of its request is on its path (itself included)."""
    n = max(fresh)
    parent = (torch.rand(len(fresh), n, generator=gen, device=DEV) * (torch.arange(n, device=DEV) + 1)).long() - 1  # -1: hangs on the last token of the history
    words = torch.zeros(len(fresh), n + 1, dtype=torch.int64, device=DEV)
    for i in range(n):
        words[:, i] = (1 << i if i < 63 else -(1 << 63)) | torch.where(parent[:, i] >= 0, words.gather(1, parent[:, i: i + 1].clamp(min=0))[:, 0], 0)
    return torch.cat([words[b, :f] for b, f in enumerate(fresh)])


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "adapter": _own_adapter, "logits": _own_logits}[op](s)
    return {"rotary": _plain_rotary, "adapter": _plain_adapter, "logits": _plain_logits}[op](s)


def _rotary_outputs(s):
    return tuple(s[x] for x in ("q_out", "k_out", "k_cache", "v_cache") if s.get(x) is not None)


def _own_rotary(s):
    import ternary_hadamard_rotated_gb300 as tb
    c = s["case"]
    if c["cache"]:
        tb.tb_rotary_cache_write(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["plan"], c["rot"], s["layout"], s["q_out"], s["k_cache"], s["v_cache"], k_out=s["k_out"],
                                 inverse=c["inverse"])
    else:
        tb.tb_rotary(s["q"], s["k"], s["pos"], s["plan"], c["rot"], s["layout"], s["q_out"], s["k_out"], inverse=c["inverse"])
    return _rotary_outputs(s)


def _own_adapter(s):
    import ternary_hadamard_rotated_gb300 as tb
    if s["case"]["plan"]:
        tb.tb_adapter_plan(s["row_start"], s["adapter"], s["tokens"], s["case"]["adapters"], s["plan"])
    for m in s["linears"]:
        tb.tb_adapter_linear(m["x"], m["a"], m["b"], s["scale"], s["plan"], m["y"], s["workspace"], out=m["out"], rank=s["rank"])
    return [m["out"] for m in s["linears"]]


def _own_logits(s):
    import ternary_hadamard_rotated_gb300 as tb
    tb.tb_logits_adjust(s["logits"], s["out"], s["history"], s["hist_len"], s["prompt_len"], row_start=s["row_start"] if s["case"]["tree"] else None, slot=s["slot"],
                        fresh=s["drafts"], tree=s["words"], repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], bias_start=s["bias_start"],
                        bias_ids=s["bias_ids"], bias_values=s["bias_values"], mask=s["mask"], mask_row=s["mask_row"])
    return s["out"]


def _plain_rotary(s):
    c = s["case"]
    R, n = c["rot"], c["rot"] // 2
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = (s["amplitude"] * torch.cos(angle)).float()[:, None], (s["amplitude"] * torch.sin(angle)).float()[:, None]
    if c["inverse"]:
        sin = -sin

    def turn(x, out):
        f = x.float()
        a, b = (f[..., :n], f[..., n:R]) if c["layout"] == "half" else (f[..., 0:R:2], f[..., 1:R:2])
        a, b = a * cos - b * sin, a * sin + b * cos
        out[..., :R] = (torch.cat([a, b], -1) if c["layout"] == "half" else torch.stack([a, b], -1).flatten(-2)).half()
        out[..., R:] = x[..., R:]

    turn(s["q"], s["q_out"])
    k = s["k_out"] if s["k_out"] is not None else torch.empty_like(s["k"])
    turn(s["k"], k)
    if c["cache"]:
        p, i = s["slots"] // c["page"], s["slots"] % c["page"]
        s["k_cache"][p, :, i] = k
        s["v_cache"][p, :, i] = s["v"]
    return _rotary_outputs(s)


def _plain_adapter(s):
    live = torch.arange(s["case"]["rank"], device=DEV)
    for m in s["linears"]:
        t = 0
        for n, g in zip(s["lens"], s["ids"]):
            y = m["y"][t: t + n]
            if g >= 0:
                h = torch.matmul(m["x"][t: t + n].float(), m["a"][g].float().t())
                h = torch.where(live < s["ranks"][g], h, 0.0)
                y = (y.float() + s["scale"][g] * torch.matmul(h, m["b"][g].float().t())).half()
            m["out"][t: t + n] = y
            t += n
    return [m["out"] for m in s["linears"]]


def _plain_logits(s):
    V, T = s["case"]["vocab"], s["logits"].shape[0]
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(s["row_start"][1:], t.to(torch.int32), right=True)
    L = s["history"].shape[1]
    ids, place = s["history"][s["slot"].long()[b]].long(), torch.arange(L, device=DEV)
    here = place < s["hist_len"][b][:, None]
    said = here & (place >= s["prompt_len"][b][:, None])
    zeros = lambda: torch.zeros(T, V, dtype=torch.int32, device=DEV)  # noqa: E731
    seen = zeros().scatter_add_(1, ids, here.to(torch.int32))
    count = zeros().scatter_add_(1, ids, said.to(torch.int32))
    if s["drafts"] is not None:
        j = torch.arange(max(s["fresh_lens"]), device=DEV)
        path = ((s["words"][:, None] >> j) & 1).to(torch.int32)
        drafts = s["drafts"].long()[(s["row_start"].long()[b][:, None] + j).clamp(max=T - 1)]
        seen.scatter_add_(1, drafts, path)
        count.scatter_add_(1, drafts, path)
    x, rho = s["logits"].float(), s["repetition"][b][:, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rho, x * rho), x)
    x = torch.where(count > 0, x - s["frequency"][b][:, None] * count.float() - s["presence"][b][:, None], x)
    if s["bias_ids"] is not None:
        n = s["bias_start"][1:] - s["bias_start"][:-1]
        owner = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n.long(), output_size=s["bias_ids"].numel())
        bias = torch.zeros(n.numel(), V, device=DEV)
        bias[owner, s["bias_ids"].long()] = s["bias_values"]
        x = x + bias[b]
    if s["mask"] is not None:
        bits = (s["mask"][s["mask_row"].long().clamp(min=0)][:, :, None] >> torch.arange(32, dtype=torch.int32, device=DEV)) & 1
        x = torch.where((bits.flatten(1)[:, :V] == 1) | (s["mask_row"] < 0)[:, None], x, -torch.inf)
    s["out"].copy_(x)
    return s["out"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "rotary":
        T, D, Hq, Hk = case["tokens"], case["dim"], case["heads"], case["kv_heads"]
        copies = (2 if case["run"] > 1 else 1) if case["cache"] else 1  # of k that are written
        return {"bytes": T * (2 * D * (2 * Hq + Hk * (1 + copies) + (2 * Hk if case["cache"] else 0)) + 4 + (8 if case["cache"] else 0)), "flops": 3 * T * (Hq + Hk) * case["rot"]}
    if op == "adapter":
        lens = _lengths(case, "q")
        ids, ranks = _adapters_of(case)
        bytes_, flops = 0, 0
        for K, N in _shapes(case):
            bytes_ += sum(4 * N * n + (2 * K * n if g >= 0 else 0) for n, g in zip(lens, ids)) + sum(2 * ranks[g] * (K + N) for g in set(ids) if g >= 0)
            flops += sum(2 * n * ranks[g] * (K + N) for n, g in zip(lens, ids) if g >= 0)
        return {"bytes": bytes_, "flops": flops}
    fresh, hist = _lengths(case, "q"), _lengths(case, "hist", 1)
    V, T, masked = case["vocab"], sum(fresh), _masked(case)[1]
    return {"bytes": T * V * (6 if case["wide"] else 4) + 4 * sum(hist) + masked * _up(V, 32) * 4, "flops": 4 * (sum(h * f for h, f in zip(hist, fresh)))}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "adapter": _exact_adapter, "logits": _exact_logits}[case["op"]](s)


def _exact_rotary(s):
    """Pairs as complex numbers, times the unit number of their angle."""
    c = s["case"]
    T, R = c["tokens"], c["rot"]
    even = torch.arange(0, R, 2, device=DEV)
    first, second = (even // 2, even // 2 + R // 2) if c["layout"] == "half" else (even, even + 1)
    angle = torch.outer(s["pos"].double(), s["freq"]) * (-1.0 if c["inverse"] else 1.0)
    unit = torch.polar(torch.full_like(angle, s["amplitude"]), angle)[:, None]

    def turned(x):
        y = x.double()
        z = torch.complex(y[..., first], y[..., second]) * unit
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def cached(x):
        P, H, page, D = s["k_cache"].shape
        rows = torch.zeros(P * page, H, D, dtype=torch.float64, device=DEV).index_copy_(0, s["slots"], x.double())
        return rows.view(P, page, H, D).transpose(1, 2).contiguous()

    k = turned(s["k"])
    out = [turned(s["q"])]
    if s["k_out"] is not None:
        out.append(k)
    if c["cache"]:
        out += [cached(k), cached(s["v"])]
    return tuple(out)


def _exact_adapter(s):
    out = []
    starts = _sums(s["lens"])
    for m in s["linears"]:
        z = m["y"].double()
        for g in sorted(set(s["ids"]) - {-1}):  # all rows of an adapter at once
            rows = torch.cat([torch.arange(starts[i], starts[i + 1], device=DEV) for i, x in enumerate(s["ids"]) if x == g])
            r = s["ranks"][g]
            z[rows] += float(s["scale"][g]) * (m["x"][rows].double() @ m["a"][g, :r].double().t() @ m["b"][g, :, :r].double().t())
        out.append(z)
    return out


def _exact_logits(s):
    """Row by row, on the host."""
    V = s["case"]["vocab"]
    host = {k: v.cpu().numpy() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("out", "logits")}
    out = np.empty((s["logits"].shape[0], V))
    t = 0
    for b, n in enumerate(s["fresh_lens"]):
        past = host["history"][host["slot"][b], : host["hist_len"][b]]
        for i in range(n):
            path = [host["drafts"][t - i + j] for j in range(n) if int(host["words"][t]) >> j & 1] if s["drafts"] is not None else []
            path = np.array(path, dtype=past.dtype)
            x = s["logits"][t].double().cpu().numpy()
            known = np.unique(np.concatenate([past, path]))
            x[known] = np.where(x[known] > 0, x[known] / float(host["repetition"][b]), x[known] * float(host["repetition"][b]))
            said, times = np.unique(np.concatenate([past[host["prompt_len"][b]:], path]), return_counts=True)
            x[said] -= float(host["frequency"][b]) * times + float(host["presence"][b])
            if s["bias_ids"] is not None:
                at = slice(host["bias_start"][b], host["bias_start"][b + 1])
                x[host["bias_ids"][at]] += host["bias_values"][at].astype(np.float64)
            if s["mask"] is not None and host["mask_row"][t] >= 0:
                words = host["mask"][host["mask_row"][t]].view(np.uint32)
                x[np.unpackbits(words.view(np.uint8), bitorder="little")[:V] == 0] = -np.inf
            out[t] = x
            t += 1
    return torch.from_numpy(out).to(DEV)
