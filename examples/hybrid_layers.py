"""A linear-attention layer and a full-attention layer of the hybrid model, on the library's calls.

Each layer is the pack's linears (tb_packed_linear) around its mixer: the gated delta rule with a pool of
fp32 states, or attention with a paged K/V cache.  The three phases of serving run through both:

  prefill  packed prompts of different lengths   tb_gated_delta (chunks), tb_prompt_attention
  decode   one token per request                 tb_gated_delta (steps), tb_tree_attention
  verify   a tree of drafted tokens per request  tb_gated_delta (a run per path), tb_tree_attention

tb_cache_plan and tb_cache_write keep the cache in each.  Weights are random ternary codes; what lies
outside the library here (norms, the short convolution, gates, the token loop) is left out or done in
torch.  ``python examples/hybrid_layers.py`` runs the phases at the 27B model's sizes and prints how far
decoding is from one prompt of the same tokens.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ternary_hadamard_rotated_gb300 as tb  # noqa: E402

DEV = "cuda"
D_DELTA = 128


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _starts(lens):
    return _i32([sum(lens[:i]) for i in range(len(lens) + 1)])


class Linear:
    """A packed linear with random ternary weights: y = fwht(x) . W^T."""

    def __init__(self, K, N, gen):
        codes = torch.randint(-1, 2, (N, K), dtype=torch.int8, device=DEV, generator=gen)
        self.K, self.N = K, N
        self.scales = torch.full((N, K // 128), 1.2 * K ** -0.5, dtype=torch.float16, device=DEV)
        self.w = torch.empty((N, K // 16), dtype=torch.int32, device=DEV)
        self.biases = torch.empty_like(self.scales)
        self.signs = (torch.randint(0, 2, (K,), device=DEV, dtype=torch.int8, generator=gen) * 2 - 1).contiguous()
        tb.tb_pack_w2(codes, self.scales, self.w, self.biases)
        self.workspace = {}

    def __call__(self, x):
        M = x.shape[0]
        if M not in self.workspace:
            self.workspace[M] = torch.zeros(tb.tb_packed_linear_workspace_size(M, self.K, self.N), dtype=torch.uint8, device=DEV)
        y = torch.empty(M, self.N, dtype=torch.float16, device=DEV)
        tb.tb_packed_linear(x, self.signs, 1024, self.w, self.scales, self.biases, y, self.workspace[M])
        return y


class HybridLayers:
    def __init__(self, hidden=5120, key_heads=16, value_heads=48, heads=24, kv_heads=4, dim=256, requests=4, pages=256, page=64,
                 max_pages=64, seed=0):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.kh, self.vh, self.h, self.kvh, self.dim, self.page = key_heads, value_heads, heads, kv_heads, dim, page
        # the linear-attention layer, its small unquantised projection of decays and steps, and its states
        self.delta_in = Linear(hidden, (2 * key_heads + value_heads) * D_DELTA, gen)
        self.delta_out = Linear(value_heads * D_DELTA, hidden, gen)
        self.gates = torch.randn(hidden, 2 * value_heads, generator=gen, device=DEV) * hidden ** -0.5
        self.states = torch.zeros(requests, value_heads, D_DELTA, D_DELTA, device=DEV)
        # the full-attention layer and its cache
        self.attn_in = Linear(hidden, (heads + 2 * kv_heads) * dim, gen)
        self.attn_out = Linear(heads * dim, hidden, gen)
        self.k_cache = torch.empty(pages, kv_heads, page, dim, dtype=torch.float16, device=DEV)
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.full((requests, max_pages), -1, dtype=torch.int32, device=DEV)
        self.free = list(range(pages))
        self.cached = [0] * requests
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    # ---- the mixers' inputs

    def _delta(self, x, lens, slot_in, slot_out):
        """The linear-attention layer over packed requests, states from and to the pool's rows."""
        T, B, Hk, Hv = x.shape[0], len(lens), self.kh, self.vh
        q, k, v = (y.unflatten(1, (-1, D_DELTA)) for y in self.delta_in(x).split([Hk * D_DELTA, Hk * D_DELTA, Hv * D_DELTA], 1))
        a, b = (x.float() @ self.gates).chunk(2, 1)
        g, beta = (-torch.nn.functional.softplus(a) * 0.2).contiguous(), torch.sigmoid(b).contiguous()
        o = torch.empty(T, Hv, D_DELTA, dtype=torch.float16, device=DEV)
        n = max(lens)
        ws = torch.empty(tb.tb_gated_delta_workspace_size(T, B, n, Hk, Hv), dtype=torch.uint8, device=DEV)
        tb.tb_gated_delta(q, k, v, g, beta, _starts(lens), n, o, ws, state_in=self.states, state_out=self.states, slot_in=_i32(slot_in),
                          slot_out=_i32(slot_out), normalise=True, dev_status=self.status)
        return x + self.delta_out(o.flatten(1))

    def _qkv(self, x):
        y = self.attn_in(x)
        return (t.unflatten(1, (-1, self.dim)) for t in y.split([self.h * self.dim, self.kvh * self.dim, self.kvh * self.dim], 1))

    def _append(self, k, v, lens):
        """Pages and slots for the new tokens of every request, and their K and V written there."""
        B = len(lens)
        cached = self.cached
        slots = torch.empty(sum(lens), dtype=torch.int64, device=DEV)
        rows, total = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
        need = sum(-(-(c + n) // self.page) - -(-c // self.page) for c, n in zip(cached, lens))
        tb.tb_cache_plan(_i32(cached), _i32(lens), self.page, _i32(self.free[:need]), self.table, slots, rows, total, dev_status=self.status)
        tb.tb_cache_write(k, v, slots, self.k_cache, self.v_cache, self.status)
        return rows, total, need

    def _over_cache(self, q, rows, total, max_q, tree=None):
        T, H, D = q.shape
        o = torch.empty(T, H, D, dtype=torch.float16, device=DEV)
        ws = torch.empty(tb.tb_tree_attention_workspace_size(total.numel(), T, max_q, H, self.kvh, D), dtype=torch.uint8, device=DEV)
        tb.tb_tree_attention(q, self.k_cache, self.v_cache, self.table, total, rows, max_q, o, ws, tree=tree, dev_status=self.status)
        return o

    # ---- the phases

    def prefill(self, x, lens):
        """Packed prompts, one per request: hidden states after both layers."""
        here = list(range(len(lens)))
        x = self._delta(x, lens, [-1] * len(lens), here)  # from no state, to the request's row
        q, k, v = self._qkv(x)
        self.cached = [0] * len(lens)
        rows, _, need = self._append(k, v, lens)
        del self.free[:need]
        o = torch.empty(q.shape, dtype=torch.float16, device=DEV)
        tb.tb_prompt_attention(q, k, v, rows, rows, o, dev_status=self.status)
        self.cached = list(lens)
        return x + self.attn_out(o.flatten(1))

    def decode(self, x):
        """One token per request."""
        B = x.shape[0]
        here = list(range(B))
        x = self._delta(x, [1] * B, here, here)
        q, k, v = self._qkv(x)
        rows, total, need = self._append(k, v, [1] * B)
        del self.free[:need]
        o = self._over_cache(q, rows, total, 1)
        self.cached = [c + 1 for c in self.cached]
        return x + self.attn_out(o.flatten(1))

    def verify(self, x, parents):
        """A tree of drafted tokens per request: parents[b][i] is the draft before draft i, or -1 for the last
        accepted token.  Nothing is kept: the states' rows are read only, the cache's tokens not counted."""
        lens = [len(p) for p in parents]
        first = [sum(lens[:b]) for b in range(len(lens))]
        # the linear layer runs each path from a root to a leaf as a request of its own, from the same row
        paths = []
        for b, p in enumerate(parents):
            for leaf in (i for i in range(len(p)) if i not in p):
                path = [leaf]
                while p[path[0]] >= 0:
                    path.insert(0, p[path[0]])
                paths.append((b, path))
        at = torch.tensor([first[b] + i for b, path in paths for i in path], device=DEV)
        y = self._delta(x[at], [len(path) for _, path in paths], [b for b, _ in paths], [-1] * len(paths))
        x = torch.empty_like(x).index_copy_(0, at, y)  # (a draft on several paths is the same on each)
        # the attention layer takes the whole tree: each draft sees itself and its ancestors
        words = []
        for p in parents:
            own = []
            for i, q in enumerate(p):
                own.append((1 << i) | (own[q] if q >= 0 else 0))
            words += own
        q, k, v = self._qkv(x)
        rows, total, _ = self._append(k, v, lens)
        tree = torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device=DEV)
        o = self._over_cache(q, rows, total, max(lens), tree)
        return x + self.attn_out(o.flatten(1))


def run(lens, steps, parents, **sizes):
    """Prefill, decode and verify; returns the largest relative errors (2-norm) of the decoded and of the
    verified hidden states against one prompt of the same tokens."""
    B = len(lens)
    layers = HybridLayers(requests=B, **sizes)
    hidden = layers.delta_in.K
    gen = torch.Generator(device=DEV).manual_seed(7)
    rand = lambda n: torch.randn(n, hidden, generator=gen, device=DEV).half()  # noqa: E731
    prompts, later = [rand(n) for n in lens], [rand(steps) for _ in lens]
    drafts = [rand(len(p)) for p in parents]
    layers.prefill(torch.cat(prompts), lens)
    decoded = torch.stack([layers.decode(torch.cat([y[i: i + 1] for y in later])) for i in range(steps)], 1)
    verified = layers.verify(torch.cat(drafts), parents)
    assert int(layers.status) == 0
    far = lambda a, b: float((a.float() - b.float()).norm() / b.float().norm())  # noqa: E731
    worst, worst_draft, at = 0.0, 0.0, 0
    for b in range(B):
        other = HybridLayers(requests=1, **sizes)  # the same weights, an empty cache
        whole = other.prefill(torch.cat([prompts[b], later[b]]), [lens[b] + steps])
        worst = max(worst, far(decoded[b], whole[lens[b]:]))
        for i, p in enumerate(parents[b]):  # each draft as the last token of its own path
            path = [i]
            while parents[b][path[0]] >= 0:
                path.insert(0, parents[b][path[0]])
            other = HybridLayers(requests=1, **sizes)
            whole = other.prefill(torch.cat([prompts[b], later[b], drafts[b][path]]), [lens[b] + steps + len(path)])
            worst_draft = max(worst_draft, far(verified[at + i], whole[-1]))
        at += len(parents[b])
    return worst, worst_draft


if __name__ == "__main__":
    print("relative error of decoded and of verified tokens against one prompt: %.1e, %.1e"
          % run([700, 1, 130], 5, [[-1, 0, 0, 1, 1, 2], [-1, -1], [-1, 0, 1, 2]]))
