"""The operators between the packed linears, case by case: the paged cache's plan and writes, attention
over that cache and over whole prompts, and the gated delta rule.

``listed()`` gives the cases that are timed, ``draw(rng)`` more of the same ranges, ``prepare`` the tensors a
serving program holds before the call, ``run`` one pass, ``work`` the bytes and operations that the pass cannot
do without, and ``exact`` the outputs in 64 bits.  With ``own`` set, ``run`` calls the library; otherwise it
computes the operator from elementary torch operations in 32 bits, rounded once at the end.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
HEAD = 128  # head width of the gated delta rule


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one scheduler step of a decoding server: every request gets one token, a few need a page
        dict(name="plan-decode", op="plan", batch=256, page=64, cached_lo=1, cached_hi=32768, fresh_lo=1, fresh_hi=1, mix=1),
        # admission of many prompts at once, chunked prefills of requests that are part-way in among them
        dict(name="plan-prefill", op="plan", batch=500, page=16, cached_lo=1, cached_hi=9000, fresh_lo=1, fresh_hi=8191, mix=2),
        # K and V of one decoded token for each of 64 requests
        dict(name="write-decode", op="write", tokens=64, run=1, heads=4, dim=256, page=64, mix=3),
        # K and V of long prompts, page after page
        dict(name="write-prefill", op="write", tokens=40001, run=1777, heads=4, dim=256, page=64, mix=4),
        # one user, one token, a context of a few thousand tokens: latency counts
        dict(name="decode-one", op="tree", batch=1, q_lo=1, q_hi=1, len_lo=4097, len_hi=4097, tree=False, heads=24, kv_heads=4, dim=256, page=64, mix=5),
        # verification of up to 16 drafted tokens for a small batch
        dict(name="tree-verify", op="tree", batch=9, q_lo=5, q_hi=16, len_lo=300, len_hi=9000, tree=True, heads=24, kv_heads=4, dim=256, page=64, mix=6),
        # decode of a full batch over long, ragged contexts: bandwidth counts
        dict(name="decode-batch", op="tree", batch=64, q_lo=1, q_hi=1, len_lo=2000, len_hi=30000, tree=False, heads=24, kv_heads=4, dim=256, page=64, mix=7),
        # packed prompts of mixed lengths, some with earlier tokens before them
        dict(name="prompt-ragged", op="prompt", batch=13, q_lo=1, q_hi=1999, past_lo=0, past_hi=700, heads=24, kv_heads=4, dim=256, mix=8),
        # one long prompt
        dict(name="prompt-long", op="prompt", batch=1, q_lo=12289, q_hi=12289, past_lo=0, past_hi=0, heads=24, kv_heads=4, dim=256, mix=9),
        # one decoded token for each of 64 requests: the states are read and written once
        dict(name="delta-step", op="delta", batch=64, len_lo=1, len_hi=1, key_heads=16, value_heads=48, norm=True, mix=10),
        # packed prompts of mixed lengths
        dict(name="delta-ragged", op="delta", batch=12, len_lo=1, len_hi=1500, key_heads=16, value_heads=48, norm=True, mix=11),
        # one long prompt
        dict(name="delta-long", op="delta", batch=1, len_lo=8192, len_hi=8192, key_heads=16, value_heads=48, norm=True, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "tree", "prompt", "delta"])
    mix = rng.randrange(1 << 30)
    if op == "plan":
        many = rng.random() < 0.5
        batch = _log(rng, 1, 300 if many else 2000)
        return dict(op=op, batch=batch, page=rng.choice([16, 32, 64, 128, 256]), cached_lo=1, cached_hi=_log(rng, 16, 9000),
                    fresh_lo=1, fresh_hi=_log(rng, 64, 8191) if many else rng.randint(1, 8), mix=mix)
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 30000), run=_log(rng, 1, 2000), heads=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 256]),
                    page=rng.choice([16, 32, 64, 128, 256]), mix=mix)
    if op == "tree":
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 3, 4, 6, 8])
        tree = rng.random() < 0.5
        q_hi = _log(rng, 2, 64) if tree else 1
        return dict(op=op, batch=_log(rng, 1, 24), q_lo=1, q_hi=q_hi, len_lo=q_hi, len_hi=_log(rng, max(q_hi, 100), 16000), tree=tree, heads=kv * group,
                    kv_heads=kv, dim=rng.choice([64, 128, 256]), page=rng.choice([16, 32, 64, 128, 256]), mix=mix)
    if op == "prompt":
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, batch=_log(rng, 1, 10), q_lo=1, q_hi=_log(rng, 20, 4000), past_lo=0, past_hi=rng.choice([0, 100, 1000]),
                    heads=kv * rng.choice([1, 2, 4, 6]), kv_heads=kv, dim=rng.choice([64, 128, 256]), mix=mix)
    kh = rng.choice([2, 4, 8, 16])
    long = rng.random() < 0.6
    return dict(op=op, batch=_log(rng, 1, 8 if long else 60), len_lo=1, len_hi=_log(rng, 20, 2500) if long else rng.randint(1, 6), key_heads=kh,
                value_heads=kh * rng.choice([1, 2, 3]), norm=rng.random() < 0.7, mix=mix)


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


def _tree_lengths(case):
    fresh = _lengths(case, "q")
    return fresh, [max(n, f) for n, f in zip(_lengths(case, "len", 1), fresh)]


def _prompt_lengths(case):
    q = _lengths(case, "q")
    return q, [a + b for a, b in zip(q, _lengths(case, "past", 1))]


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _randn(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).half()


def prepare(case, seed):
    return {"plan": _prepare_plan, "write": _prepare_write, "tree": _prepare_tree, "prompt": _prepare_prompt, "delta": _prepare_delta}[case["op"]](case, _gen(seed))


def _prepare_plan(case, gen):
    B, page = case["batch"], case["page"]
    cached, fresh = _lengths(case, "cached"), _lengths(case, "fresh", 1)
    have = [_up(c, page) for c in cached]
    need = [_up(c + f, page) for c, f in zip(cached, fresh)]
    held, wanted = sum(have), sum(need) - sum(have)
    pages = torch.randperm(held + 2 * wanted + 8, generator=gen, device=DEV).to(torch.int32)  # the pool in the order of use
    width = max(need) + 3
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    first = _ints(_sums(have)[:-1])
    col = torch.arange(width, device=DEV)[None, :]
    inside = col < _ints(have)[:, None]
    table = torch.where(inside, pages[(first[:, None] + col).clamp(max=max(held - 1, 0))], table)
    T = sum(fresh)
    return dict(case=case, cached=_ints(cached), fresh=_ints(fresh), free=pages[held:].clone(), table=table, tokens=T,
                slots=torch.empty(T, dtype=torch.int64, device=DEV), row_start=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                total=torch.empty(B, dtype=torch.int32, device=DEV), used=torch.empty(1, dtype=torch.int32, device=DEV))


def _prepare_write(case, gen):
    T, H, D, page, run_ = case["tokens"], case["heads"], case["dim"], case["page"], case["run"]
    # requests of `run` tokens that begin somewhere in a page; a request's pages lie anywhere in the pool
    reqs = _up(T, run_)
    per = _up(run_ + page - 1, page)
    pool = reqs * per + 5
    t = torch.arange(T, device=DEV)
    r = t // run_
    begin = torch.randint(0, page, (reqs,), generator=gen, device=DEV)
    pos = begin[r] + t - r * run_
    pages = torch.randperm(pool, generator=gen, device=DEV)
    slots = pages[r * per + pos // page] * page + pos % page
    kv = _randn(gen, T, 2 * H * D)  # the two projections side by side, as one packed linear leaves them
    k, v = kv[:, : H * D].view(T, H, D), kv[:, H * D:].view(T, H, D)
    return dict(case=case, k=k, v=v, slots=slots, k_cache=torch.zeros(pool, H, page, D, dtype=torch.float16, device=DEV),
                v_cache=torch.zeros(pool, H, page, D, dtype=torch.float16, device=DEV))


def _trees(gen, fresh):
    """A random tree of drafted tokens for each request: bit j of a token's word says that it sees token j of its request (its ancestors and itself)."""
    n = max(fresh)
    parent = (torch.rand(len(fresh), n, generator=gen, device=DEV) * (torch.arange(n, device=DEV) + 1)).long() - 1  # -1: hangs on the last cached token
    words = torch.zeros(len(fresh), n + 1, dtype=torch.int64, device=DEV)
    for i in range(n):
        words[:, i] = (1 << i if i < 63 else -(1 << 63)) | torch.where(parent[:, i] >= 0, words.gather(1, parent[:, i: i + 1].clamp(min=0))[:, 0], 0)
    return torch.cat([words[b, :f] for b, f in enumerate(fresh)])


def _prepare_tree(case, gen):
    B, Hq, Hk, D, page = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    fresh, total = _tree_lengths(case)
    T = sum(fresh)
    pages = [_up(n, page) for n in total]
    pool = sum(pages) + 3
    perm = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    width = max(pages)
    col = torch.arange(width, device=DEV)[None, :]
    table = torch.where(col < _ints(pages)[:, None], perm[(_ints(_sums(pages)[:-1])[:, None] + col).clamp(max=pool - 1)], -1)
    q = _randn(gen, T, (Hq + 2 * Hk) * D, scale=1.5)[:, : Hq * D].view(T, Hq, D)  # a slice of the fused projection
    state = dict(case=case, q=q, k_cache=_randn(gen, pool, Hk, page, D), v_cache=_randn(gen, pool, Hk, page, D), table=table, total=_ints(total),
                 row_start=_ints(_sums(fresh)), tree=_trees(gen, fresh) if case["tree"] else None, max_q=max(fresh), max_len=max(total),
                 o=torch.empty(T, Hq, D, dtype=torch.float16, device=DEV))
    if own:
        import ternary_hadamard_rotated_gb300 as tb
        state["workspace"] = torch.zeros(tb.tb_tree_attention_workspace_size(B, T, max(fresh), Hq, Hk, D), dtype=torch.uint8, device=DEV)
    return state


def _prepare_prompt(case, gen):
    Hq, Hk, D = case["heads"], case["kv_heads"], case["dim"]
    ql, kl = _prompt_lengths(case)
    if ql == kl:  # the three are slices of the fused projection
        qkv = _randn(gen, sum(ql), (Hq + 2 * Hk) * D)
        q, k, v = (x.view(sum(ql), -1, D) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    else:
        q, k, v = _randn(gen, sum(ql), Hq, D), _randn(gen, sum(kl), Hk, D), _randn(gen, sum(kl), Hk, D)
    return dict(case=case, q=q, k=k, v=v, ql=ql, kl=kl, q_start=_ints(_sums(ql)), k_start=_ints(_sums(kl)),
                o=torch.empty(sum(ql), Hq, D, dtype=torch.float16, device=DEV))


def _prepare_delta(case, gen):
    B, Hk, Hv = case["batch"], case["key_heads"], case["value_heads"]
    lens = _lengths(case, "len")
    T = sum(lens)
    qkv = _randn(gen, T, (2 * Hk + Hv) * HEAD)  # the fused projection after its convolution
    q, k, v = (x.view(T, -1, HEAD) for x in qkv.split([Hk * HEAD, Hk * HEAD, Hv * HEAD], 1))
    if not case["norm"]:  # the caller has normalised them
        q, k = ((x.float() / x.float().norm(dim=-1, keepdim=True)).half() for x in (q, k))
    # decays from nearly 1 to a tenth, as a head's learned rate and step give them
    rate = torch.exp(torch.linspace(-6, 0.5, Hv, device=DEV))
    g = -rate * torch.nn.functional.softplus(torch.randn(T, Hv, generator=gen, device=DEV))
    beta = torch.sigmoid(torch.randn(T, Hv, generator=gen, device=DEV))
    state = dict(case=case, q=q, k=k, v=v, g=g, beta=beta, lens=lens, row_start=_ints(_sums(lens)), max_len=max(lens),
                 state_in=torch.randn(B, Hv, HEAD, HEAD, generator=gen, device=DEV) * 0.3, state_out=torch.empty(B, Hv, HEAD, HEAD, device=DEV),
                 o=torch.empty(T, Hv, HEAD, dtype=torch.float16, device=DEV))
    if own:
        import ternary_hadamard_rotated_gb300 as tb
        state["workspace"] = torch.zeros(tb.tb_gated_delta_workspace_size(T, B, max(lens), Hk, Hv), dtype=torch.uint8, device=DEV)
    return state


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"plan": _plain_plan, "write": _plain_write, "tree": _plain_tree, "prompt": _plain_prompt, "delta": _plain_delta}[s["case"]["op"]](s)


def _run_own(s):
    import ternary_hadamard_rotated_gb300 as tb
    op = s["case"]["op"]
    if op == "plan":
        tb.tb_cache_plan(s["cached"], s["fresh"], s["case"]["page"], s["free"], s["table"], s["slots"], s["row_start"], s["total"], s["used"])
        return s["table"], s["slots"], s["row_start"], s["total"], s["used"]
    if op == "write":
        tb.tb_cache_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return s["k_cache"], s["v_cache"]
    if op == "tree":
        tb.tb_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["total"], s["row_start"], s["max_q"], s["o"], s["workspace"], tree=s["tree"])
        return s["o"]
    if op == "prompt":
        tb.tb_prompt_attention(s["q"], s["k"], s["v"], s["q_start"], s["k_start"], s["o"])
        return s["o"]
    tb.tb_gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["row_start"], s["max_len"], s["o"], s["workspace"], state_in=s["state_in"],
                      state_out=s["state_out"], normalise=s["case"]["norm"])
    return s["o"], s["state_out"]


def _plain_plan(s):
    page, cached, fresh, T = s["case"]["page"], s["cached"], s["fresh"], s["tokens"]
    have = (cached + page - 1) // page
    need = (cached + fresh + page - 1) // page
    ends = torch.cumsum(need - have, 0)
    first = ends - (need - have)
    col = torch.arange(s["table"].shape[1], device=DEV)[None, :]
    taken = (first - have)[:, None] + col
    new = (col >= have[:, None]) & (col < need[:, None])
    table = torch.where(new, s["free"][taken.clamp(0, s["free"].numel() - 1)], s["table"])
    sums = torch.cumsum(fresh, 0)
    row_start = torch.nn.functional.pad(sums, (1, 0)).to(torch.int32)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(sums, t, right=True)
    pos = cached[b] + t - row_start[b]
    slots = table[b, pos // page].to(torch.int64) * page + pos % page
    return table, slots, row_start, cached + fresh, ends[-1:].to(torch.int32)


def _plain_write(s):
    page = s["case"]["page"]
    p, i = s["slots"] // page, s["slots"] % page
    s["k_cache"][p, :, i] = s["k"]
    s["v_cache"][p, :, i] = s["v"]
    return s["k_cache"], s["v_cache"]


def _plain_tree(s):
    c = s["case"]
    B, Hq, Hk, D, page, n = c["batch"], c["heads"], c["kv_heads"], c["dim"], c["page"], s["max_q"]
    T, G, L = s["q"].shape[0], Hq // Hk, s["table"].shape[1] * page
    start = s["row_start"].long()
    fresh = start[1:] - start[:-1]
    row = (start[:-1, None] + torch.arange(n, device=DEV)).clamp(max=T - 1)  # [B, n], the padded rows unused
    q = s["q"][row].float().view(B, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, D)
    pages = s["table"].long().clamp(min=0)
    k = s["k_cache"][pages].float().permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hk, G, n, L) * D ** -0.5
    del k
    prefix = (s["total"] - fresh)[:, None]
    j = torch.arange(L, device=DEV)[None, :] - prefix  # the key's number among the drafted tokens, below 0 in the prefix
    i = torch.arange(n, device=DEV)
    if s["tree"] is None:
        seen = j[:, None, :] <= i[None, :, None]
    else:
        seen = ((s["tree"][row][:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1).bool() | (j < 0)[:, None, :]
    seen = seen & (j < fresh[:, None])[:, None, :]
    x = torch.where(seen[:, None, None], x, -torch.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    v = s["v_cache"][pages].float().permute(0, 2, 1, 3, 4).reshape(B, Hk, L, D)
    o = torch.matmul(x.view(B, Hk, G * n, L), v).view(B, Hk, G, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, Hq, D)
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:], t, right=True)
    return o[b * n + t - start[b]].half()


def _plain_prompt(s):
    Hq, Hk, D = s["case"]["heads"], s["case"]["kv_heads"], s["case"]["dim"]
    G, out, a, b = Hq // Hk, torch.empty_like(s["o"]), 0, 0
    for lq, lk in zip(s["ql"], s["kl"]):
        seen = torch.arange(lk, device=DEV)[None, :] <= torch.arange(lq, device=DEV)[:, None] + (lk - lq)
        for h in range(Hk):
            q = s["q"][a: a + lq, h * G: (h + 1) * G].float().transpose(0, 1)
            x = torch.matmul(q, s["k"][b: b + lk, h].float().t()) * D ** -0.5
            x = torch.where(seen, x, -torch.inf)
            x = torch.exp(x - x.amax(-1, keepdim=True))
            x = x / x.sum(-1, keepdim=True)
            out[a: a + lq, h * G: (h + 1) * G] = torch.matmul(x, s["v"][b: b + lk, h].float()).transpose(0, 1).half()
        a, b = a + lq, b + lk
    return out


def _plain_delta(s):
    """The chunked form: inside a chunk the recurrence is a triangular system, between chunks the state is carried."""
    Hk, Hv = s["case"]["key_heads"], s["case"]["value_heads"]
    B, L = s["case"]["batch"], s["max_len"]
    C = min(64, L)
    N = _up(L, C)
    start = s["row_start"].long()
    t = torch.arange(N * C, device=DEV)
    inside = t[None, :] < (start[1:] - start[:-1])[:, None]  # [B, N * C]
    row = (start[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)

    def chunks(x, heads):  # [T, H, ...] -> [B, Hv, N, C, ...], zero past a request's end
        x = torch.where(inside.view(B, N * C, *[1] * (x.dim() - 1)), x[row].float(), 0.0)
        x = x.repeat_interleave(Hv // heads, 2)
        return x.view(B, N, C, *x.shape[2:]).movedim(3, 1)

    q, k, v, g, beta = chunks(s["q"], Hk), chunks(s["k"], Hk), chunks(s["v"], Hv), chunks(s["g"], Hv), chunks(s["beta"], Hv)
    if s["case"]["norm"]:
        q, k = (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
    q = q * HEAD ** -0.5
    gs = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=DEV).tril()
    decay = torch.exp(torch.where(low, gs[..., :, None] - gs[..., None, :], -torch.inf))
    A = (beta[..., None] * torch.matmul(k, k.transpose(-1, -2)) * decay).tril(-1)
    inv = torch.eye(C, device=DEV).expand_as(A).clone()
    for i in range(1, C):  # row i of (I + A)^-1 from the rows above it
        inv[..., i, :i] = -torch.matmul(A[..., i: i + 1, :i], inv[..., :i, :i])[..., 0, :]
    u = torch.matmul(inv, beta[..., None] * v)
    w = torch.matmul(inv, (beta * torch.exp(gs))[..., None] * k)
    p = torch.matmul(q, k.transpose(-1, -2)) * decay
    qs = q * torch.exp(gs)[..., None]
    ks = k * torch.exp(gs[..., -1:] - gs)[..., None]
    S, o = s["state_in"], torch.empty_like(v)
    for c in range(N):
        x = u[:, :, c] - torch.matmul(w[:, :, c], S)
        o[:, :, c] = torch.matmul(qs[:, :, c], S) + torch.matmul(p[:, :, c], x)
        S = S * torch.exp(gs[:, :, c, -1])[..., None, None] + torch.matmul(ks[:, :, c].transpose(-1, -2), x)
    T = s["q"].shape[0]
    n = torch.arange(T, device=DEV)
    b = torch.searchsorted(start[1:], n, right=True)
    return o.movedim(1, 3).reshape(B * N * C, Hv, HEAD)[b * (N * C) + n - start[b]].half(), S


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "plan":
        page = case["page"]
        cached, fresh = _lengths(case, "cached"), _lengths(case, "fresh", 1)
        new = sum(_up(c + f, page) - _up(c, page) for c, f in zip(cached, fresh))
        return {"bytes": 16 * case["batch"] + 8 * new + 8 * sum(fresh), "flops": 0}
    if op == "write":
        return {"bytes": case["tokens"] * (8 * case["heads"] * case["dim"] + 8), "flops": 0}
    if op == "tree":
        fresh, total = _tree_lengths(case)
        D, Hq = case["dim"], case["heads"]
        return {"bytes": 4 * D * case["kv_heads"] * sum(total) + 4 * D * Hq * sum(fresh), "flops": 4 * D * Hq * sum(f * n for f, n in zip(fresh, total))}
    if op == "prompt":
        ql, kl = _prompt_lengths(case)
        D, Hq = case["dim"], case["heads"]
        pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(ql, kl))
        return {"bytes": 4 * D * Hq * sum(ql) + 4 * D * case["kv_heads"] * sum(kl), "flops": 4 * D * Hq * pairs}
    lens = _lengths(case, "len")
    Hk, Hv, T = case["key_heads"], case["value_heads"], sum(lens)
    return {"bytes": T * (4 * HEAD * (Hk + Hv) + 8 * Hv) + 8 * HEAD * HEAD * Hv * case["batch"], "flops": 6 * HEAD * HEAD * Hv * T}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "plan":  # whole numbers only
        return None
    s = prepare(case, seed)
    return {"write": _exact_write, "tree": _exact_tree, "prompt": _exact_prompt, "delta": _exact_delta}[case["op"]](s)


def _exact_write(s):
    out = []
    for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        P, H, page, D = cache.shape
        rows = torch.zeros(P * page, H, D, dtype=torch.float64, device=DEV).index_copy_(0, s["slots"], x.double())
        out.append(rows.view(P, page, H, D).transpose(1, 2).contiguous())
    return tuple(out)


def _softmax_rows(q, k, v, seen):
    """q [n, D], k and v [L, D], seen [n, L]: each row's weighted mean of v."""
    x = (q @ k.t()) / math.sqrt(q.shape[1])
    x = x.masked_fill(~seen, -math.inf)
    w = torch.softmax(x, -1)
    return w @ v


def _exact_tree(s):
    c = s["case"]
    fresh, total = _tree_lengths(c)
    G, page = c["heads"] // c["kv_heads"], c["page"]
    out = torch.empty(s["o"].shape, dtype=torch.float64, device=DEV)
    a = 0
    for b, (n, L) in enumerate(zip(fresh, total)):
        pos = torch.arange(L, device=DEV)
        at = s["table"][b, : _up(L, page)].long()[pos // page]
        seen = torch.ones(n, L, dtype=torch.bool, device=DEV)
        for i in range(n):
            word = (1 << (i + 1)) - 1 if s["tree"] is None else int(s["tree"][a + i])
            seen[i, L - n:] = torch.tensor([bool(word >> j & 1) for j in range(n)], device=DEV)
        for h in range(c["kv_heads"]):
            k, v = (x[at, h, pos % page].double() for x in (s["k_cache"], s["v_cache"]))
            for g in range(h * G, (h + 1) * G):
                out[a: a + n, g] = _softmax_rows(s["q"][a: a + n, g].double(), k, v, seen)
        a += n
    return out


def _exact_prompt(s):
    c = s["case"]
    G = c["heads"] // c["kv_heads"]
    out = torch.empty(s["o"].shape, dtype=torch.float64, device=DEV)
    a = b = 0
    for lq, lk in zip(s["ql"], s["kl"]):
        for i in range(0, lq, 2048):
            n = min(2048, lq - i)
            end = lk - lq + i + n  # no row of this block sees a key past it
            seen = torch.arange(end, device=DEV)[None, :] <= torch.arange(i, i + n, device=DEV)[:, None] + (lk - lq)
            for h in range(c["heads"]):
                k, v = (x[b: b + end, h // G].double() for x in (s["k"], s["v"]))
                out[a + i: a + i + n, h] = _softmax_rows(s["q"][a + i: a + i + n, h].double(), k, v, seen)
        a, b = a + lq, b + lk
    return out


def _exact_delta(s):
    """The recurrence, token by token, all requests and heads at once."""
    c = s["case"]
    G = c["value_heads"] // c["key_heads"]
    lens = s["lens"]
    S = s["state_in"].double()
    out = torch.empty(s["o"].shape, dtype=torch.float64, device=DEV)
    order = sorted(range(len(lens)), key=lambda b: -lens[b])  # the requests that still run are the first ones
    S = S[order]
    start = _sums(lens)
    first = _ints([start[b] for b in order], torch.int64)
    for t in range(max(lens)):
        n = sum(x > t for x in lens)
        row = first[:n] + t
        q, k, v = (s[x][row].double() for x in "qkv")
        if c["norm"]:
            q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + 1e-6) for x in (q, k))
        q, k = (x.repeat_interleave(G, 1) for x in (q, k))
        R = S[:n] * torch.exp(s["g"][row].double())[..., None, None]
        u = s["beta"][row].double()[..., None] * (v - torch.einsum("bhk,bhkv->bhv", k, R))
        R = R + k[..., :, None] * u[..., None, :]
        out[row] = torch.einsum("bhk,bhkv->bhv", q, R) / math.sqrt(HEAD)
        S[:n] = R
    back = torch.empty_like(S)
    back[order] = S
    return out, back
