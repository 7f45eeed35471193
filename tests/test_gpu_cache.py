"""GPU parity of the paged cache's plan and writes: whole numbers and copies, so every element is equal."""
import numpy as np
import pytest

from oracle import mixers

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def plan(cached, fresh, page, free, table, T, guard=3):
    """One call; outputs have guard elements behind them that must stay as they were."""
    import ternary_hadamard_rotated_gb300 as tb

    B, width = table.shape
    dev = dict(device="cuda")
    c, f = torch.tensor(cached, dtype=torch.int32, **dev), torch.tensor(fresh, dtype=torch.int32, **dev)
    fr = torch.tensor(free, dtype=torch.int32, **dev)
    tab = torch.full((B + 1, width), -77, dtype=torch.int32, **dev)
    tab[:B] = torch.from_numpy(table)
    slots = torch.full((T + guard,), -77, dtype=torch.int64, **dev)
    rows = torch.full((B + 1 + guard,), -77, dtype=torch.int32, **dev)
    total = torch.full((B + guard,), -77, dtype=torch.int32, **dev)
    used = torch.full((1 + guard,), -77, dtype=torch.int32, **dev)
    st = torch.zeros(1, dtype=torch.int32, **dev)
    tb.tb_cache_plan(c, f, page, fr, tab[:B], slots[:T], rows[: B + 1], total[:B], used[:1], st)
    torch.cuda.synchronize()
    assert (tab[B] == -77).all() and (slots[T:] == -77).all() and (rows[B + 1:] == -77).all()
    assert (total[B:] == -77).all() and (used[1:] == -77).all()
    return (tab[:B].cpu().numpy(), slots[:T].cpu().numpy(), rows[: B + 1].cpu().numpy(), total[:B].cpu().numpy(),
            int(used[0])), int(st)


def requests(rng, B, page, cached_hi, fresh_hi, spare=5):
    cached, fresh = rng.integers(0, cached_hi + 1, B), rng.integers(0, fresh_hi + 1, B)
    have, need = -(-cached // page), -(-(cached + fresh) // page)
    width = int(max(need.max(), 1)) + 2
    pages = rng.permutation(int(need.sum()) + spare)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, : have[b]] = pages[at: at + have[b]]
        at += have[b]
    return cached, fresh, pages[at:].astype(np.int32), table


@pytest.mark.parametrize("B,page,cached_hi,fresh_hi", [
    (1, 16, 0, 1), (1, 256, 700, 1), (7, 64, 100, 0), (3, 64, 200, 130), (31, 16, 90, 5), (33, 32, 64, 64),
    (511, 128, 300, 1), (513, 16, 40, 40), (2000, 64, 500, 3), (5, 16, 0, 20000), (16384, 16, 30, 2)])
def test_plan_matches(B, page, cached_hi, fresh_hi):
    rng = np.random.default_rng(B * 1000 + page)
    cached, fresh, free, table = requests(rng, B, page, cached_hi, fresh_hi)
    T = int(fresh.sum()) + 11  # room past the last token: padding
    got, st = plan(cached, fresh, page, free, table, T)
    want = mixers.cache_plan(cached, fresh, page, free, table, T)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert st == 0
    again, _ = plan(cached, fresh, page, free, got[0], T)  # on its own table: the same once more
    for g, w in zip(again, want):
        assert np.array_equal(g, w)


def test_plan_without_enough_pages():
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(3)
    cached, fresh, free, table = requests(rng, 40, 16, 50, 60)
    need = int((-(-(cached + fresh) // 16) + (-cached // 16)).sum())
    T = int(fresh.sum())
    for n in (0, 1, need - 1):
        got, st = plan(cached, fresh, 16, free[:n], table, T)
        want = mixers.cache_plan(cached, fresh, 16, free[:n], table, T)
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
        assert st == tb.TB_DEV_NO_PAGE and got[4] == n
    got, st = plan(cached, fresh, 16, free[:need], table, T)
    assert st == 0 and got[4] == need
    # rows of the table too short for some requests
    short = table[:, :4].copy()
    keep = cached <= 64
    got, st = plan(cached[keep], fresh[keep], 16, free, short[keep], T)
    want = mixers.cache_plan(cached[keep], fresh[keep], 16, free, short[keep], T)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert st == tb.TB_DEV_NO_PAGE


def test_plan_flags_lengths_that_do_not_fit():
    import ternary_hadamard_rotated_gb300 as tb

    table = np.full((3, 4), -1, dtype=np.int32)
    table[0, 0] = 9
    got, st = plan([5, 0, 0], [2, -4, 3], 16, np.arange(4, dtype=np.int32), table, 8)
    assert st == tb.TB_DEV_BAD_LEN
    want = mixers.cache_plan([5, 0, 0], [2, 0, 3], 16, np.arange(4), table, 8)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    _, st = plan([5, 0, 0], [2, 4, 3], 16, np.arange(4, dtype=np.int32), table, 8)  # 9 tokens, room for 8
    assert st == tb.TB_DEV_BAD_LEN
    got, st = plan([17, 0, 0], [2, 0, 0], 16, np.arange(4, dtype=np.int32), table, 8)  # a held page without a number
    assert st == tb.TB_DEV_BAD_SLOT
    assert (got[1] == -1).all()


@pytest.mark.parametrize("T,H,D,page,split", [(1, 1, 64, 16, False), (37, 4, 256, 64, True), (300, 2, 128, 256, True),
                                              (1000, 8, 64, 32, False), (5, 3, 8, 128, True), (4001, 4, 256, 16, True)])
def test_write_matches(T, H, D, page, split):
    import ternary_hadamard_rotated_gb300 as tb

    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 3
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[rng.random(T) < 0.2] = -1
    kv = rng.standard_normal((T, 2 * H * D + (16 if split else 0))).astype(np.float16)
    kv[0, 0], kv[-1, -17] = np.inf, np.nan
    kc = rng.standard_normal((pages, H, page, D)).astype(np.float16)
    vc = rng.standard_normal((pages, H, page, D)).astype(np.float16)
    x = torch.from_numpy(kv).cuda()
    if split:
        k, v = x[:, 8: 8 + H * D].view(T, H, D), x[:, 8 + H * D: 8 + 2 * H * D].view(T, H, D)
        kn, vn = kv[:, 8: 8 + H * D].reshape(T, H, D), kv[:, 8 + H * D: 8 + 2 * H * D].reshape(T, H, D)
    else:
        k, v = x[:, : H * D].contiguous().view(T, H, D), x[:, H * D:].contiguous().view(T, H, D)
        kn, vn = kv[:, : H * D].reshape(T, H, D), kv[:, H * D:].reshape(T, H, D)
    kd, vd = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tb.tb_cache_write(k, v, torch.from_numpy(slots).cuda(), kd, vd, st)
    torch.cuda.synchronize()
    wk, wv = mixers.cache_write(kn, vn, slots, kc, vc)
    assert np.array_equal(kd.cpu().numpy().view(np.uint16), wk.view(np.uint16))
    assert np.array_equal(vd.cpu().numpy().view(np.uint16), wv.view(np.uint16))
    assert int(st) == 0
    slots[-1] = pages * page  # just past the cache
    tb.tb_cache_write(k, v, torch.from_numpy(slots).cuda(), kd, vd, st)
    torch.cuda.synchronize()
    assert int(st) == tb.TB_DEV_BAD_SLOT


def test_write_past_two_to_the_31_elements():
    """A cache whose offsets pass 32 bits: the last page of a 9 GB pair."""
    import ternary_hadamard_rotated_gb300 as tb

    pages, H, page, D = 2 ** 31 // (4 * 64 * 256) + 40, 4, 64, 256
    kc = torch.zeros((pages, H, page, D), dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.randn(3, H, D, device="cuda").half()
    v = torch.randn(3, H, D, device="cuda").half()
    slots = torch.tensor([pages * page - 1, 0, (pages - 2) * page], device="cuda")
    tb.tb_cache_write(k, v, slots, kc, vc)
    torch.cuda.synchronize()
    for c, x in ((kc, k), (vc, v)):
        for t, s in enumerate(slots.tolist()):
            assert torch.equal(c[s // page, :, s % page], x[t])
        assert int((c != 0).sum()) == int((x != 0).sum())
