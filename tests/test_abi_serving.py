"""Host-side refusals of the operators around the linears, and the binding's checks (no GPU needed)."""
import os

import pytest

P = 0x1000  # a 16-byte aligned non-null placeholder; never dereferenced by these calls
Q = 0x2000


@pytest.fixture(scope="module")
def lib():
    import ternary_hadamard_rotated_gb300 as tb
    from ternary_hadamard_rotated_gb300 import build as tbbuild

    if not os.path.exists(tb.LIB_PATH):
        tbbuild.build()
    return tb.load()


def caller(fn, names, **ok):
    def call(**kw):
        a = {**ok, **kw}
        return fn(*[a[n] for n in names.split()])
    return call


def test_rotary_plan_refuses(lib):
    call = caller(lib.tb_rotary_plan, "plan size R base kind factor original fast slow amp freqs st s", plan=P, size=1 << 20, R=64, base=1e4, kind=0, factor=1.0,
                  original=4096.0, fast=32.0, slow=1.0, amp=0.0, freqs=None, st=None, s=None)
    nan, inf = float("nan"), float("inf")
    for R in (0, -2, 63, 1, 1026):
        assert call(R=R) == -2 and lib.tb_rotary_plan_size(R) == 0
    assert call(kind=4) == call(kind=-1) == -3
    assert call(plan=None) == -1
    assert call(plan=P + 8) == call(freqs=P + 4) == -6
    assert call(size=lib.tb_rotary_plan_size(64) - 1) == -7
    assert call(amp=-1.0) == call(amp=nan) == call(amp=inf) == call(amp=1e39) == -4
    assert call(base=1.0) == call(base=nan) == call(base=inf) == -4
    for kind in (1, 2, 3):
        assert call(kind=kind, factor=0.0) == call(kind=kind, factor=-2.0) == call(kind=kind, factor=nan) == call(kind=kind, factor=inf) == -4
        assert call(kind=kind, freqs=P) == -4
    assert call(kind=2, factor=2.0, R=2) == -4
    part = dict(kind=3, factor=2.0)
    assert call(**part, original=0.0) == call(**part, original=inf) == call(**part, slow=0.0) == call(**part, fast=1.0) == call(**part, fast=nan) == -4


ROTARY = dict(q=P, ldq=4096, Hq=16, k=P, ldk=1024, Hk=4, T=7, D=256, pos=P, plan=P, R=64, layout=0, inv=0, qo=Q, ldqo=4096, ko=Q, ldko=1024, st=None, s=None)


def test_rotary_refuses(lib):
    call = caller(lib.tb_rotary, "q ldq Hq k ldk Hk T D pos plan R layout inv qo ldqo ko ldko st s", **ROTARY)
    for name in ("q", "k", "pos", "plan", "qo", "ko"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    for bad in (dict(R=0), dict(R=63), dict(R=258), dict(D=252), dict(D=1032, ldq=1 << 20, ldqo=1 << 20, ldk=1 << 20, ldko=1 << 20), dict(Hq=0), dict(Hq=1025), dict(Hk=-1),
                dict(T=-1), dict(T=2 ** 31), dict(ldq=4088), dict(ldq=4100), dict(ldqo=4088), dict(ldk=1016), dict(ldk=1028), dict(ldko=1016), dict(ldko=1030)):
        assert call(**bad) == -2, bad
    assert call(qo=P, ldqo=4104) == call(ko=P, ldko=2048) == -2  # in place at another distance
    assert call(layout=2) == call(layout=-1) == -3
    assert call(T=0, q=None, k=None) == 0


def test_rotary_cache_write_refuses(lib):
    call = caller(lib.tb_rotary_cache_write, "q ldq Hq k ldk v ldv Hk T D pos slots plan R layout inv qo ldqo ko ldko kc vc pages page st s",
                  **ROTARY, v=P, ldv=1024, slots=P, kc=Q, vc=Q, pages=9, page=64)
    for name in ("q", "k", "v", "pos", "slots", "plan", "qo", "kc", "vc"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(slots=P + 4) == call(ko=Q + 2) == -6
    assert call(Hk=0) == call(ldv=1016) == call(ldv=1020) == call(pages=0) == call(pages=2 ** 31) == call(R=66, D=64) == -2
    assert call(page=48) == call(layout=7) == -3
    assert call(T=0, v=None) == 0


def test_adapter_plan_refuses(lib):
    size = lib.tb_adapter_plan_size(100, 5)
    assert size > 0 and lib.tb_adapter_plan_size(-1, 5) == lib.tb_adapter_plan_size(9, 0) == lib.tb_adapter_plan_size(9, 16385) == 0
    call = caller(lib.tb_adapter_plan, "row ad B T n plan size st s", row=P, ad=P, B=4, T=100, n=5, plan=P, size=size, st=None, s=None)
    for name in ("row", "ad", "plan"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(plan=P + 8) == -6
    assert call(B=0) == call(T=-1) == call(T=2 ** 30 + 1) == call(n=0) == -2
    assert call(B=16385) == call(n=16385) == -8
    assert call(size=size - 1) == -7


def test_adapter_linear_refuses(lib):
    need = lib.tb_adapter_linear_workspace_size(9, 5, 1024, 512, 16)
    call = caller(lib.tb_adapter_linear, "x ldx T K a b n R N rank scale plan y ldy out ldo ws size st s", x=P, ldx=1024, T=9, K=1024, a=P, b=P, n=5, R=16, N=512,
                  rank=None, scale=P, plan=P, y=P, ldy=512, out=Q, ldo=512, ws=P, size=need, st=None, s=None)
    for name in ("x", "a", "b", "scale", "plan", "y", "out"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(rank=P + 2) == call(ws=P + 8) == -6
    for bad in (dict(K=0), dict(K=1020), dict(K=1 << 21, ldx=1 << 21), dict(N=508), dict(N=0), dict(R=0), dict(R=12), dict(n=0), dict(T=-1), dict(ldx=1016), dict(ldx=1028),
                dict(ldy=504), dict(ldo=516)):
        assert call(**bad) == -2, bad
    assert call(out=P, ldo=520) == -2  # in place at another distance
    assert call(R=264) == -3
    assert call(n=16385) == -8
    assert call(size=need - 1) == call(ws=None) == -7
    assert call(T=0, x=None) == 0
    for bad in ((-1, 5, 1024, 512, 16), (9, 0, 1024, 512, 16), (9, 5, 0, 512, 16), (9, 5, 1024, 512, 264)):
        assert lib.tb_adapter_linear_workspace_size(*bad) == 0


def test_logits_adjust_refuses(lib):
    call = caller(lib.tb_logits_adjust, "x ld T V row B hist nh ldh slot hl pl fresh tree rep pres freq bs bi bv nb mask mr mrow out ldo kind st s", x=P, ld=1000, T=6, V=1000,
                  row=P, B=4, hist=P, nh=9, ldh=50, slot=P, hl=P, pl=P, fresh=P, tree=P, rep=P, pres=P, freq=P, bs=P, bi=P, bv=P, nb=3, mask=P, mr=2, mrow=P, out=Q, ldo=1000,
                  kind=0, st=None, s=None)
    for name in ("x", "out", "hist", "hl", "bs", "bi", "bv"):
        assert call(**{name: None}) == -1, name
    assert call(fresh=None) == -1  # a tree of nothing
    for name in ("x", "row", "hist", "slot", "hl", "pl", "fresh", "rep", "pres", "freq", "bs", "bi", "bv", "mask", "mrow", "out"):
        assert call(**{name: P + 2}) == -6, name
    assert call(x=P + 8) == call(out=Q + 8) == call(tree=P + 4) == -6
    for bad in (dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25, ldo=1 << 25), dict(ld=999), dict(ldo=999), dict(T=-1), dict(B=0), dict(nh=0), dict(ldh=-1), dict(ldh=(1 << 28) + 1), dict(nb=-1), dict(mr=-1),
                dict(row=None), dict(slot=None, nh=3), dict(mrow=None)):
        assert call(**bad) == -2, bad
    assert call(out=P, kind=1) == call(out=P, ldo=1008) == -2  # in place at another type or distance
    assert call(kind=2) == -3
    assert call(T=65536) == call(B=65536) == -8
    assert call(T=0, x=None) == 0


def test_binding_refuses_what_it_cannot_pass_on():
    import torch

    import ternary_hadamard_rotated_gb300 as tb

    f16, i32 = torch.float16, torch.int32
    q, k, pos, plan = torch.zeros(4, 2, 64, dtype=f16), torch.zeros(4, 1, 64, dtype=f16), torch.zeros(4, dtype=i32), torch.zeros(tb.tb_rotary_plan_size(64), dtype=torch.uint8)
    c = torch.zeros(3, 1, 16, 64, dtype=f16)
    bad = [lambda: tb.tb_rotary(q.float(), k, pos, plan, 64, 0, q, k), lambda: tb.tb_rotary(q, k, pos.long(), plan, 64, 0, q, k), lambda: tb.tb_rotary(q, k, pos, plan, 64, 0, q[:3], k),
           lambda: tb.tb_rotary(q, k, pos[:3], plan, 64, 0, q, k), lambda: tb.tb_rotary(q, k[:3], pos, plan, 64, 0, q, k), lambda: tb.tb_rotary(q, k, pos, plan, 64, 0, q, q),
           lambda: tb.tb_rotary_cache_write(q, k, k, pos, pos, plan, 64, 0, q, c, c), lambda: tb.tb_rotary_cache_write(q, k, q, pos, pos.long(), plan, 64, 0, q, c, c),
           lambda: tb.tb_rotary_cache_write(q, k, k, pos, pos.long(), plan, 64, 0, q, c, c, k_out=q),
           lambda: tb.tb_rotary_cache_write(q, k, k, pos, pos.long(), plan, 64, 0, q, c, c[:2]),
           lambda: tb.tb_rotary(q, k, pos, plan, 64, 0, q, k)]  # not on a GPU
    x, y, a, b, s = torch.zeros(4, 16, dtype=f16), torch.zeros(4, 24, dtype=f16), torch.zeros(2, 8, 16, dtype=f16), torch.zeros(2, 24, 8, dtype=f16), torch.zeros(2)
    bad += [lambda: tb.tb_adapter_linear(x.float(), a, b, s, plan, y, plan), lambda: tb.tb_adapter_linear(x.t().contiguous().t(), a, b, s, plan, y, plan),
            lambda: tb.tb_adapter_linear(x, a, b[:, :16], s, plan, y, plan), lambda: tb.tb_adapter_linear(x, a, b, s[:1], plan, y, plan),
            lambda: tb.tb_adapter_linear(x, a, b, s, plan, y[:3], plan), lambda: tb.tb_adapter_linear(x, a, b, s, plan, y, plan, out=y.float()),
            lambda: tb.tb_adapter_linear(x, a, b, s, plan, y, plan, rank=s), lambda: tb.tb_adapter_linear(x, a, b, s, plan, y, plan),
            lambda: tb.tb_adapter_plan(pos, pos, 4, 2, plan), lambda: tb.tb_adapter_plan(torch.zeros(5, dtype=i32), pos, 4, 2, plan)]
    h, n = torch.zeros(4, 9, dtype=i32), torch.zeros(4, dtype=i32)
    bad += [lambda: tb.tb_logits_adjust(y.float(), y, h, n), lambda: tb.tb_logits_adjust(y, y[:, :23], h, n), lambda: tb.tb_logits_adjust(y, y.double(), h, n),
            lambda: tb.tb_logits_adjust(y, y, h.long(), n), lambda: tb.tb_logits_adjust(y, y, h, n, prompt_len=n[:2]), lambda: tb.tb_logits_adjust(y, y, h, n, tree=n),
            lambda: tb.tb_logits_adjust(y, y, h, n, mask=h), lambda: tb.tb_logits_adjust(y, y, h, n, repetition=n), lambda: tb.tb_logits_adjust(y, y, h[:, ::2], n),
            lambda: tb.tb_logits_adjust(y, y, h, n)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)


def test_rotary_of_k_needs_a_place_for_it():
    import ternary_hadamard_rotated_gb300 as tb

    torch = pytest.importorskip("torch")
    q = torch.zeros(2, 4, 64, dtype=torch.float16)
    pos, plan = torch.zeros(2, dtype=torch.int32), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_out"):
        tb.tb_rotary(q, q, pos, plan, 64, tb.TB_ROTARY_HALF, q, None)
