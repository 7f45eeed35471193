"""GPU parity of attention over packed prompts and over the paged cache against float64; the tolerance
of each element is derived in oracle.mixers.attention_tolerance."""
import numpy as np
import pytest

from oracle import mixers

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def close(got, want, tol, what=""):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bad = np.abs(got - want) > tol
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], tol[bad][:4])


def starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def guarded(T, H, D):
    o = torch.full((T + 2, H, D), 7.0, dtype=torch.float16, device="cuda")
    return o, o[:T]


# ---------------------------------------------------------------- prompts

def prompt_case(seed, ql, kl, Hq, Hkv, D, fused, scale=None, peak=1.0):
    import ternary_hadamard_rotated_gb300 as tb

    rng = torch.Generator().manual_seed(seed)
    Tq, Tk = sum(ql), sum(kl)
    if fused:  # slices of one projection, with room between the tokens
        qkv = torch.randn(Tq, (Hq + 2 * Hkv) * D + 24, generator=rng).half().cuda()
        q = qkv[:, 8: 8 + Hq * D].unflatten(1, (Hq, D))
        k = qkv[:, 8 + Hq * D: 8 + (Hq + Hkv) * D].unflatten(1, (Hkv, D))
        v = qkv[:, 8 + (Hq + Hkv) * D: 8 + (Hq + 2 * Hkv) * D].unflatten(1, (Hkv, D))
    else:
        q, k, v = (torch.randn(T, H, D, generator=rng).half().cuda() for T, H in ((Tq, Hq), (Tk, Hkv), (Tk, Hkv)))
    if peak != 1.0:
        q.mul_(peak)
    full, o = guarded(Tq, Hq, D)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tb.tb_prompt_attention(q, k, v, starts(ql), starts(kl), o, scale=scale, dev_status=st)
    torch.cuda.synchronize()
    assert (full[Tq:] == 7.0).all()
    assert int(st) == 0
    want, tol = mixers.prompt_attention(q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), starts(ql).tolist(),
                                        starts(kl).tolist(), D ** -0.5 if scale is None else scale)
    close(o, want, tol, (ql, kl, Hq, Hkv, D))
    return q, k, v, o


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ql", [[1], [2], [15, 1, 17], [64], [127], [128], [129], [255, 0, 257], [1, 300, 3, 0, 0, 63]])
def test_prompt_lengths(D, ql):
    prompt_case(D + len(ql), ql, ql, 6, 2, D, fused=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (24, 4), (5, 1), (8, 8), (32, 2)])
def test_prompt_heads(D, Hq, Hkv):
    prompt_case(Hq, [70, 1, 33], [70, 1, 33], Hq, Hkv, D, fused=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ql,kl", [([1], [200]), ([3, 70, 1], [130, 391, 128]), ([128, 5], [256, 5]), ([130], [129 + 130]),
                                   ([64, 200, 0, 7], [3, 64, 40, 0]), ([300], [1])])
def test_prompt_with_earlier_keys_and_with_too_few(D, ql, kl):
    """More keys than queries (a prompt's later part), and fewer (the first rows see nothing: zeros)."""
    q, k, v, o = prompt_case(5, ql, kl, 4, 2, D, fused=False)
    a = 0
    for lq, lk in zip(ql, kl):
        if lk < lq:
            assert (o[a: a + lq - lk] == 0).all()
        a += lq


@pytest.mark.parametrize("B", [31, 100, 128, 129, 400])
def test_prompt_many_requests(B):
    rng = np.random.default_rng(B)
    ql = rng.integers(0, 70, B).tolist()
    kl = [q + int(rng.integers(-3, 60)) if q else int(rng.integers(0, 9)) for q in ql]
    prompt_case(B, ql, [max(0, k) for k in kl], 3, 1, 64 if B == 100 else 128, fused=False)


@pytest.mark.parametrize("D", [128, 256])
def test_prompt_long(D):
    prompt_case(9, [1500, 700], [1500, 700], 3, 1, D, fused=True)


@pytest.mark.parametrize("D", [64, 256])
def test_prompt_peaked_and_flat(D):
    prompt_case(2, [260], [260], 2, 1, D, fused=False, peak=20.0)
    prompt_case(3, [260], [260], 2, 1, D, fused=False, scale=1e-4)


def test_prompt_rising_scores():
    """Scores that grow along the keys: the running maximum moves in every tile."""
    import ternary_hadamard_rotated_gb300 as tb

    D, L = 256, 700
    gen = torch.Generator().manual_seed(1)
    q = torch.ones(L, 1, D).half()
    k = (torch.linspace(0, 40, L)[:, None, None] / 16 + torch.randn(L, 1, D, generator=gen) * 0.1).half()
    v = torch.randn(L, 1, D, generator=gen).half()
    o = torch.empty(L, 1, D, dtype=torch.float16, device="cuda")
    for kk in (k, k.flip(0).contiguous(), -k):
        tb.tb_prompt_attention(q.cuda(), kk.cuda(), v.cuda(), starts([L]), starts([L]), o)
        want, tol = mixers.prompt_attention(q.numpy(), kk.numpy(), v.numpy(), [0, L], [0, L], D ** -0.5)
        close(o, want, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prompt_what_is_not_seen_does_not_reach_a_row(D, bad):
    """A token whose K and V are not finite: the rows before it, and the other requests, are as without it."""
    import ternary_hadamard_rotated_gb300 as tb

    gen = torch.Generator().manual_seed(4)
    lens = [150, 90, 140]
    T = sum(lens)
    q, k, v = (torch.randn(T, 2, D, generator=gen).half().cuda() for _ in range(3))
    ref = torch.empty_like(q)
    tb.tb_prompt_attention(q, k, v, starts(lens), starts(lens), ref)
    at = lens[0] + 50
    k2, v2 = k.clone(), v.clone()
    k2[at], v2[at] = bad, bad
    o = torch.empty_like(q)
    tb.tb_prompt_attention(q, k2, v2, starts(lens), starts(lens), o)
    torch.cuda.synchronize()
    keep = torch.ones(T, dtype=torch.bool)
    keep[at: lens[0] + lens[1]] = False
    want, tol = mixers.prompt_attention(q.cpu().numpy(), k.cpu().numpy(), v.cpu().numpy(), starts(lens).tolist(),
                                        starts(lens).tolist(), D ** -0.5)
    close(o[keep], want[keep.numpy()], tol[keep.numpy()])
    if bad != bad:
        assert torch.isnan(o[at: lens[0] + lens[1]]).all()


def test_prompt_flags_row_starts_that_do_not_fit():
    import ternary_hadamard_rotated_gb300 as tb

    q = torch.randn(40, 2, 64, device="cuda").half()
    i32 = dict(dtype=torch.int32, device="cuda")
    for qs, ks in (([0, 41], [0, 40]), ([0, 40], [0, 41]), ([0, 40], [10, 5]), ([-3, 40], [0, 40])):
        o = torch.full((42, 2, 64), 7.0, dtype=torch.float16, device="cuda")
        st = torch.zeros(1, **i32)
        tb.tb_prompt_attention(q, q, q, torch.tensor(qs, **i32), torch.tensor(ks, **i32), o[:40], dev_status=st)
        torch.cuda.synchronize()
        assert int(st) == tb.TB_DEV_BAD_LEN
        assert (o[40:] == 7.0).all()


# ---------------------------------------------------------------- the paged cache

def tree_words(rng, fresh):
    words = []
    for n in fresh:
        w = []
        for i in range(n):
            p = rng.integers(-1, i) if i else -1
            w.append((1 << i) | (w[p] if p >= 0 else 0))
        words += w
    return words


def as_int64(words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def tree_case(seed, fresh, total, Hq, Hkv, D, page, tree, spare=3, poison=True, words=None, peak=1.0):
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(seed)
    B, T = len(fresh), sum(fresh)
    need = [-(-n // page) for n in total]
    pages = sum(need) + spare
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((B, max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    kc = rng.standard_normal((pages, Hkv, page, D)).astype(np.float16)
    vc = rng.standard_normal((pages, Hkv, page, D)).astype(np.float16)
    if poison:  # what lies behind a request's last token, and in pages of nobody, is not finite
        kp, vp = np.full_like(kc, np.nan), np.full_like(vc, np.inf)
    else:
        kp, vp = kc.copy(), vc.copy()
    for b in range(B):
        table[b, : need[b]] = perm[at: at + need[b]]
        for j in range(need[b]):
            n = min(page, total[b] - j * page)
            kp[table[b, j], :, :n] = kc[table[b, j], :, :n]
            vp[table[b, j], :, :n] = vc[table[b, j], :, :n]
        at += need[b]
    if tree and words is None:
        words = tree_words(rng, fresh)
    wide = torch.from_numpy((rng.standard_normal((T, (Hq + 2) * D)) * peak).astype(np.float16)).cuda()
    q = wide[:, D: (Hq + 1) * D].unflatten(1, (Hq, D))
    full, o = guarded(T, Hq, D)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq = max(fresh)
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(B, T, mq, Hq, Hkv, D) + 64, dtype=torch.uint8, device="cuda")
    args = (q, torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda(), torch.from_numpy(table).cuda(),
            torch.tensor(total, dtype=torch.int32, device="cuda"), starts(fresh), mq, o, ws[: ws.numel() - 64])
    for _ in range(2):  # the second call on the same workspace
        o.fill_(3.0)
        tb.tb_tree_attention(*args, tree=as_int64(words) if words is not None else None, dev_status=st)
        torch.cuda.synchronize()
        first = o.clone() if _ == 0 else first
    assert torch.equal(first, o)
    assert (full[T:] == 7.0).all() and (ws[ws.numel() - 64:] == 0).all()
    assert int(st) == 0
    want, tol = mixers.tree_attention(q.cpu().numpy(), kc, vc, table, total, starts(fresh).tolist(), words, D ** -0.5)
    close(o, want, tol, (fresh, total, Hq, Hkv, D, page))
    return o


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("total", [[1], [2], [16], [17], [255], [1000], [3000, 1, 77], [129, 640, 31, 64, 65]])
def test_decode_lengths(D, page, total):
    tree_case(D + page + len(total), [1] * len(total), total, 6, 1, D, page, tree=False)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (24, 4), (4, 4), (8, 1), (16, 1), (40, 2), (9, 3)])
@pytest.mark.parametrize("n", [1, 3])
def test_decode_heads(Hq, Hkv, n):
    tree_case(Hq, [n, n], [333, 90], Hq, Hkv, 256, 64, tree=False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fresh,total", [([2], [2]), ([5], [400]), ([8, 16], [1000, 16]), ([64], [64]), ([64, 1, 0, 33], [700, 50, 9, 1300]),
                                         ([17, 31], [18, 5000]), ([63], [64])])
def test_tree(D, fresh, total):
    tree_case(len(fresh) + D, fresh, total, 6, 2, D, 32, tree=True)
    tree_case(len(fresh) + D, fresh, total, 6, 2, D, 128, tree=False)


def test_tree_full_heads_and_many_requests():
    rng = np.random.default_rng(8)
    fresh = rng.integers(0, 20, 40).tolist()
    total = [int(f + rng.integers(0, 600)) for f in fresh]
    fresh[3], total[3] = 0, 0
    tree_case(1, fresh, total, 24, 4, 256, 64, tree=True)
    tree_case(2, [1] * 200, rng.integers(1, 900, 200).tolist(), 24, 4, 128, 16, tree=False)


def test_tree_peaked():
    tree_case(4, [4], [900], 4, 1, 256, 64, tree=True, peak=20.0)


def test_tree_rows_that_see_nothing():
    """A drafted token with an empty word and no prefix before its request's newest tokens: zeros."""
    o = tree_case(6, [4, 3], [4, 40], 6, 1, 128, 16, tree=True, words=[1, 0, 0b0010, 1 << 63, 1, 0, 0b111])
    assert (o[1] == 0).all() and (o[3] == 0).all() and (o[5] != 0).any()


@pytest.mark.parametrize("n", [1, 8, 40])
def test_tree_unseen_drafts_do_not_reach_a_row(n):
    """Siblings whose K and V are not finite: only the rows that see them change."""
    import ternary_hadamard_rotated_gb300 as tb

    D, page, L = 256, 32, 300 + n
    gen = torch.Generator().manual_seed(1)
    pages = -(-L // page)
    kc, vc = (torch.randn(pages, 2, page, D, generator=gen).half() for _ in range(2))
    q = torch.randn(n + 1, 6, D, generator=gen).half().cuda()
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    total = torch.tensor([L + 1], dtype=torch.int32, device="cuda")
    if (L + 1) > pages * page:
        pytest.skip("needs room for the last draft")
    words = [1 << i for i in range(n)] + [1 << n]
    kp, vp = kc.clone(), vc.clone()
    pos = L  # the last draft
    kp[pos // page, :, pos % page], vp[pos // page, :, pos % page] = float("nan"), float("inf")
    o = torch.empty_like(q)
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(1, n + 1, n + 1, 6, 2, D), dtype=torch.uint8, device="cuda")
    tb.tb_tree_attention(q, kp.cuda(), vp.cuda(), table, total, starts([n + 1]), n + 1, o, ws, tree=as_int64(words))
    torch.cuda.synchronize()
    want, tol = mixers.tree_attention(q.cpu().numpy(), kc.numpy(), vc.numpy(), table.cpu().numpy(), [L + 1], [0, n + 1], words, D ** -0.5)
    close(o[:n], want[:n], tol[:n])
    assert not torch.isfinite(o[n]).any()


def test_tree_flags():
    import ternary_hadamard_rotated_gb300 as tb

    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.randn(6, 2, 16, 64, device="cuda").half()
    q = torch.randn(5, 4, 64, device="cuda").half()
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(2, 5, 4, 4, 2, 64), dtype=torch.uint8, device="cuda")

    def call(total, table, rows, mq=4):
        o = torch.full((5, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        st = torch.zeros(1, **i32)
        tb.tb_tree_attention(q, kc, kc, torch.tensor(table, **i32), torch.tensor(total, **i32), torch.tensor(rows, **i32), mq, o, ws, dev_status=st)
        torch.cuda.synchronize()
        return o, int(st)

    good = [[0, 1], [2, 3]]
    assert call([20, 30], good, [0, 1, 5])[1] == 0
    o, st = call([20, 3], good, [0, 1, 5])  # fewer cached tokens than queries
    assert st == tb.TB_DEV_BAD_LEN and (o[1:] == 0).all() and (o[0] != 0).any()
    o, st = call([20, 33], good, [0, 1, 5])  # past the table's row
    assert st == tb.TB_DEV_BAD_LEN and (o[1:] == 0).all()
    o, st = call([20, 30], good, [0, 1, 5], mq=3)  # more queries than max_q
    assert st == tb.TB_DEV_BAD_LEN and (o[1:] == 0).all()
    o, st = call([20, 30], [[0, 6], [2, -1]], [0, 1, 5])  # pages outside the cache: their tokens are left out
    assert st == tb.TB_DEV_BAD_SLOT
    want, tol = mixers.tree_attention(q.cpu().numpy(), kc.cpu().numpy(), kc.cpu().numpy(), [[0, 6], [2, -1]], [20, 30], [0, 1, 5], None, 0.125)
    close(o, want, tol)


def test_tree_cache_past_two_to_the_31_elements():
    import ternary_hadamard_rotated_gb300 as tb

    pages, H, page, D = 2 ** 31 // (4 * 64 * 256) + 40, 4, 64, 256
    gen = torch.Generator(device="cuda").manual_seed(1)
    kc = torch.zeros((pages, H, page, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    used = [pages - 1, 3, pages - 17]
    for p in used:
        kc[p] = torch.randn(H, page, D, generator=gen, device="cuda").half()
        vc[p] = torch.randn(H, page, D, generator=gen, device="cuda").half()
    q = torch.randn(2, 24, D, generator=gen, device="cuda").half()
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    total = torch.tensor([150], dtype=torch.int32, device="cuda")
    o = torch.empty_like(q)
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(1, 2, 2, 24, H, D), dtype=torch.uint8, device="cuda")
    tb.tb_tree_attention(q, kc, vc, table, total, starts([2]), 2, o, ws)
    torch.cuda.synchronize()
    want, tol = mixers.tree_attention(q.cpu().numpy(), kc[used].cpu().numpy(), vc[used].cpu().numpy(), [[0, 1, 2]], [150], [0, 2], None, D ** -0.5)
    close(o, want, tol)


def test_other_stream():
    import ternary_hadamard_rotated_gb300 as tb

    s = torch.cuda.Stream()
    q = torch.randn(200, 4, 128, device="cuda").half()
    k = torch.randn(200, 2, 128, device="cuda").half()
    a, b = torch.empty_like(q), torch.empty_like(q)
    tb.tb_prompt_attention(q, k, k, starts([200]), starts([200]), a)
    torch.cuda.synchronize()
    tb.tb_prompt_attention(q, k, k, starts([200]), starts([200]), b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,Hkv,D,max_q,n", [(6, 2, 128, 1, 5), (6, 2, 64, 3, 130), (1, 1, 64, 1, 20000), (4, 2, 256, 64, 65)])
@pytest.mark.parametrize("why", ["rows", "short", "long"])
def test_tree_lengths_that_do_not_fit_among_others_that_do(Hq, Hkv, D, max_q, n, why):
    """A request of more rows than max_q, or whose length does not fit, before requests whose keys are spread over
    many CTAs and between them: zeros for it, the others as ever, and nothing written past the workspace."""
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(n)
    page, width = 64, 100
    bad = n if why == "rows" else max_q
    fresh = [bad, max_q, bad, 1, bad]
    wrong = {"rows": max(n, 70) if n < 6400 else 6400, "short": max_q - 1, "long": width * page + 1}[why]
    total = [wrong, 6000, wrong, 3000, wrong]
    table = np.full((5, width), -1, dtype=np.int32)
    table[1], table[3] = rng.permutation(width), rng.permutation(width)
    kc, vc = (rng.standard_normal((width, Hkv, page, D)).astype(np.float16) for _ in range(2))
    T, i32 = sum(fresh), dict(dtype=torch.int32, device="cuda")
    q = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(n)).half().cuda()
    full, o = guarded(T, Hq, D)
    size = tb.tb_tree_attention_workspace_size(5, T, max_q, Hq, Hkv, D)
    ws = torch.full((size + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, **i32)
    tb.tb_tree_attention(q, torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda(), torch.from_numpy(table).cuda(), torch.tensor(total, **i32),
                         starts(fresh), max_q, o, ws[:size], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == tb.TB_DEV_BAD_LEN
    assert (ws[size:] == 0xA5).all() and (full[T:] == 7.0).all()
    row = starts(fresh).tolist()
    for b in (0, 2, 4):
        assert (o[row[b]: row[b + 1]] == 0).all(), b
    for b in (1, 3):
        part = slice(row[b], row[b + 1])
        want, tol = mixers.tree_attention(q[part].cpu().numpy(), kc, vc, table[b: b + 1], [total[b]], [0, fresh[b]], None, D ** -0.5)
        close(o[part], want, tol, (b, why))


def attend_on_gpu(q, k, v, seen, scale):
    """Rows q [n, D] of one head over k, v [L, D] in 64 bits, seen [n, L], and their tolerance."""
    q, k, v = q.double(), k.double(), v.double()
    s = (q @ k.T * scale).masked_fill(~seen, -float("inf"))
    w = torch.exp(s - s.amax(1, keepdim=True))
    l = w.sum(1, keepdim=True)
    o, wv, tail = w @ v / l, w @ v.abs() / l, seen.double() @ v.abs() / l
    sterm = (q.abs() @ k.abs().T * scale).amax(1, keepdim=True)
    parts = [x.cpu().numpy() for x in (o, wv, tail, sterm)]
    return parts[0], mixers.attention_tolerance(*parts, q.shape[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prompt_one_bad_value_early_in_a_very_long_context(bad):
    """Every row of the long request has to be made again from 160000 keys, which takes longer than any wait inside
    the pipeline may last; the other columns of these rows and the other request stay right."""
    import ternary_hadamard_rotated_gb300 as tb

    D, H, ql, kl = 64, 6, [21, 60], [160000, 60]
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(sum(ql), H, D, generator=gen).half().cuda()
    k, v = (torch.randn(sum(kl), 1, D, generator=gen).half().cuda() for _ in range(2))
    at, col = 5, 3
    v[at, 0, col] = bad
    o = torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tb.tb_prompt_attention(q, k, v, starts(ql), starts(kl), o, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    clean = v.clone()
    clean[at, 0, col] = 0
    for a, b, x, y in ((0, 21, 0, 160000), (21, 81, 160000, 160060)):
        n, L = b - a, y - x
        seen = torch.arange(L, device="cuda")[None, :] <= torch.arange(n, device="cuda")[:, None] + L - n
        for h in range(H):
            want, tol = attend_on_gpu(q[a:b, h], k[x:y, 0], clean[x:y, 0], seen, D ** -0.5)
            keep = [c for c in range(D) if a or c != col]
            close(o[a:b, h][:, keep], want[:, keep], tol[:, keep], (a, h))
    got = o[:21, :, col]
    assert torch.isnan(got).all() if bad != bad else (got == bad).all()


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("others", [0, 300])
def test_tree_one_bad_value_early_in_a_very_long_context(n, others):
    """The same over the paged cache, alone (rows joined from parts) and among requests enough that many rows are
    finished by one CTA, every fifth of these with a bad value too."""
    import ternary_hadamard_rotated_gb300 as tb

    D, H, page = 128, 6, 64
    fresh, total = [n] + [1] * others, [160000] + [257] * others
    need = [-(-t // page) for t in total]
    gen = torch.Generator().manual_seed(6)
    kc, vc = (torch.randn(sum(need), 1, page, D, generator=gen).half().cuda() for _ in range(2))
    table = torch.full((len(fresh), max(need)), -1, dtype=torch.int32)
    first = np.concatenate([[0], np.cumsum(need)])
    for b, c in enumerate(need):
        table[b, :c] = torch.arange(first[b], first[b] + c)
    q = torch.randn(sum(fresh), H, D, generator=gen).half().cuda()
    clean = vc.clone()
    hit = [b for b in range(len(fresh)) if b % 5 == 0]
    for b in hit:
        vc[first[b], 0, 7, 11] = float("nan")
        clean[first[b], 0, 7, 11] = 0
    o = torch.empty_like(q)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(len(fresh), sum(fresh), n, H, 1, D), dtype=torch.uint8, device="cuda")
    tb.tb_tree_attention(q, kc, vc, table.cuda(), torch.tensor(total, dtype=torch.int32, device="cuda"), starts(fresh), n, o, ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    row = starts(fresh).tolist()
    for b in range(len(fresh)):
        k, v = (x[first[b]: first[b] + need[b], 0].reshape(-1, D)[: total[b]] for x in (kc, clean))
        seen = torch.arange(total[b], device="cuda")[None, :] <= torch.arange(fresh[b], device="cuda")[:, None] + total[b] - fresh[b]
        part = slice(row[b], row[b + 1])
        keep = [c for c in range(D) if b not in hit or c != 11]
        for h in range(H):
            want, tol = attend_on_gpu(q[part, h], k, v, seen, D ** -0.5)
            close(o[part, h][:, keep], want[:, keep], tol[:, keep], (b, h))
        if b in hit:
            assert torch.isnan(o[part, :, 11]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_score_of_minus_infinity_weighs_nothing(D):
    """Keys of -infinity: rows of nothing else give zeros, whatever their values; beside other keys their weight
    is 0, which leaves a finite value out."""
    import ternary_hadamard_rotated_gb300 as tb

    gen = torch.Generator().manual_seed(7)
    L, page = 200, 16
    q = torch.rand(L, 2, D, generator=gen).half().cuda() + 0.5
    k, v = (torch.randn(L, 1, D, generator=gen).half().cuda() for _ in range(2))
    k[:70] = -float("inf")
    v[3, 0, 5] = float("inf")
    o = torch.empty_like(q)
    tb.tb_prompt_attention(q, k, v, starts([L]), starts([L]), o)
    kc, vc = (torch.cat([x, x[:8]]).view(-1, page, 1, D).transpose(1, 2).contiguous() for x in (k, v))
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    n = 64
    for total in (66, L):
        p = torch.empty(n, 2, D, dtype=torch.float16, device="cuda")
        ws = torch.zeros(tb.tb_tree_attention_workspace_size(1, n, n, 2, 1, D), dtype=torch.uint8, device="cuda")
        tb.tb_tree_attention(q[total - n: total].contiguous(), kc, vc, table, torch.tensor([total], dtype=torch.int32, device="cuda"), starts([n]), n, p, ws)
        for got, lo in ((o, 0), (p, total - n)):
            for h in range(2):
                rows = got[:, h]
                pos = torch.arange(lo, lo + rows.shape[0])
                assert (rows[pos < 70] == 0).all()
                seen = (torch.arange(L)[None, :] <= pos[pos >= 70][:, None]) & (torch.arange(L)[None, :] >= 70)
                if seen.shape[0]:
                    at = pos[pos >= 70].cuda()
                    # (a key of -infinity is as one that is not there)
                    want, tol = attend_on_gpu(q[at, h], k[70:, 0], v[70:, 0], seen[:, 70:].cuda(), D ** -0.5)
                    keep = [c for c in range(D) if c != 5]
                    close(rows[pos >= 70][:, keep], want[:, keep], tol[:, keep], (lo, h))
                    assert torch.isnan(rows[pos >= 70][:, 5]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rate", [0.002, 0.2])
def test_values_that_are_not_finite_reach_the_columns_of_the_rows_that_see_them(D, rate):
    """NaN and infinities strewn over V: each output is NaN, infinite or finite as its own sum is."""
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(int(1 / rate))
    lens, H, page = [150, 1, 260], 3, 32
    T = sum(lens)
    q, k, v = (rng.standard_normal((T, h, D)).astype(np.float16) for h in (H, 1, 1))
    kinds = np.array([np.nan, np.inf, -np.inf], dtype=np.float16)
    hit = rng.random(v.shape) < rate
    v[hit] = kinds[rng.integers(0, 3, int(hit.sum()))]
    cuda = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    o = torch.empty(T, H, D, dtype=torch.float16, device="cuda")
    tb.tb_prompt_attention(cuda(q), cuda(k), cuda(v), starts(lens), starts(lens), o)
    with np.errstate(invalid="ignore"):
        want, tol = mixers.prompt_attention(q, k, v, starts(lens).tolist(), starts(lens).tolist(), D ** -0.5)

    def same(got, want, tol):
        got = got.double().cpu().numpy()
        fin = np.isfinite(want)
        assert not fin.all() and (fin.any() or rate > 0.1)  # (what the case is to hold)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
        assert (np.abs(got[fin] - want[fin]) <= tol[fin]).all()

    same(o, want, tol)
    # the last 40 tokens of the last request over the paged cache
    n, L = 40, lens[2]
    need = -(-L // page)
    kc, vc = (np.zeros((need, 1, page, D), dtype=np.float16) for _ in range(2))
    for j in range(L):
        kc[j // page, 0, j % page], vc[j // page, 0, j % page] = k[151 + j, 0], v[151 + j, 0]
    p = torch.empty(n, H, D, dtype=torch.float16, device="cuda")
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(1, n, n, H, 1, D), dtype=torch.uint8, device="cuda")
    tb.tb_tree_attention(cuda(q[-n:]), cuda(kc), cuda(vc), torch.arange(need, dtype=torch.int32, device="cuda")[None],
                         torch.tensor([L], dtype=torch.int32, device="cuda"), starts([n]), n, p, ws)
    same(p, want[-n:], tol[-n:])


def flat_tail(D, n, drop):
    """A query, one key of the largest score and n whose weights are 2^-drop of it each: k [n + 1, 1, D], with
    values of 0 and 1, so that the output is the tail's share."""
    q = torch.zeros(1, 1, D)
    q[..., 0] = D ** 0.5
    k = torch.zeros(n + 1, 1, D)
    k[n // 3, 0, 0] = drop * float(np.log(2.0))
    v = torch.ones(n + 1, 1, D)
    v[n // 3] = 0
    return q.half().cuda(), k.half().cuda(), v.half().cuda()


@pytest.mark.parametrize("drop", [16.0, 22.0, 24.6, 25.5, 27.0])
@pytest.mark.parametrize("D", [64, 256])
def test_many_small_weights_beside_a_large_one(D, drop):
    """n weights far below the largest.  The weights are fp16 operands with the largest one at 2^7 or more, so
    that a weight below 2^-14 of that is rounded by at most 2^-25 / 2^7 of the largest; scores and sums are exact
    here up to fp32's 2^-20 (24 bits less those of a score of 19)."""
    import ternary_hadamard_rotated_gb300 as tb

    n = 2 ** 18 - 1
    q, k, v = flat_tail(D, n, drop)
    w = float(np.exp2(-(k[n // 3, 0, 0].double() * q[0, 0, 0].double()).item() * D ** -0.5 / np.log(2.0)))
    want = n * w / (1 + n * w)
    tol = 2.0 ** -11 * want + (2.0 ** -11 + 2.0 ** -20) * want + n * 2.0 ** -32 + 2.0 ** -25
    o = torch.empty_like(q)
    tb.tb_prompt_attention(q, k, v, starts([1]), starts([n + 1]), o)
    assert (o.double() - want).abs().max().item() <= tol
    page = 256
    kc, vc = (x.view(-1, page, 1, D).transpose(1, 2).contiguous() for x in (k, v))
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    ws = torch.zeros(tb.tb_tree_attention_workspace_size(1, 1, 1, 1, 1, D), dtype=torch.uint8, device="cuda")
    tb.tb_tree_attention(q, kc, vc, table, torch.tensor([n + 1], dtype=torch.int32, device="cuda"), starts([1]), 1, o, ws)
    assert (o.double() - want).abs().max().item() <= tol


def test_prompt_row_starts_that_go_back():
    """Requests 0, 2, 4, .. all of the rows [0, T), more than 2^31 tiles together.  Nothing is computed."""
    import ternary_hadamard_rotated_gb300 as tb

    T, B = 1 << 20, 600001
    q = torch.zeros(T, 1, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(1, 1, 64, dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, T], dtype=torch.int32, device="cuda").repeat((B + 1) // 2)
    assert rows.numel() == B + 1
    o = torch.full_like(q, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tb.tb_prompt_attention(q, k, k, rows, torch.zeros_like(rows), o, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == tb.TB_DEV_BAD_LEN and (o == 7.0).all()


def test_prompt_of_very_many_requests():
    """A call whose work is counted in 64 bits first; requests of one token: their own value."""
    import ternary_hadamard_rotated_gb300 as tb

    T, B = 1 << 19, 600001
    rows = torch.arange(B + 1, device="cuda").clamp(max=T).int()
    q = torch.zeros(T, 1, 64, dtype=torch.float16, device="cuda")
    v = torch.randn(T, 1, 64, device="cuda").half()
    o = torch.full_like(q, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tb.tb_prompt_attention(q, v, v, rows, rows, o, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0 and torch.equal(o, v)
