"""Host-side refusals of the mixers' entry points, and the binding's checks (no GPU needed)."""
import os

import pytest

P = 0x1000  # a 16-byte aligned non-null placeholder; never dereferenced by these calls


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
        return fn(*[a[n] for n in names])
    return call


def test_cache_plan_refuses(lib):
    call = caller(lib.tb_cache_plan, ["cached", "fresh", "B", "page", "free", "n_free", "table", "max_pages", "slots", "T", "row", "total", "used", "st", "s"],
                  cached=P, fresh=P, B=4, page=64, free=P, n_free=9, table=P, max_pages=8, slots=P, T=10, row=P, total=P, used=None, st=None, s=None)
    for name in ("cached", "fresh", "free", "table", "slots", "row", "total"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(slots=P + 4) == -6
    assert call(used=P + 1) == -6
    assert call(B=0) == call(T=-1) == call(max_pages=0) == call(n_free=-1) == call(T=2 ** 31) == -2
    for page in (0, 8, 24, 48, 512, -64):
        assert call(page=page) == -3
    assert call(B=16385) == -8


def test_cache_write_refuses(lib):
    call = caller(lib.tb_cache_write, ["k", "ldk", "v", "ldv", "slots", "T", "H", "D", "kc", "vc", "pages", "page", "st", "s"],
                  k=P, ldk=1024, v=P, ldv=1024, slots=P, T=5, H=4, D=256, kc=P, vc=P, pages=9, page=64, st=None, s=None)
    for name in ("k", "v", "slots", "kc", "vc"):
        assert call(**{name: None}) == -1
        assert call(**{name: P + 2}) == -6
    assert call(ldk=1016) == call(ldv=1028) == call(H=0) == call(D=100) == call(D=1032, ldk=8192, ldv=8192) == call(pages=0) == call(T=-1) == -2
    assert call(page=40) == -3
    assert call(T=0, k=None, v=None) == 0


def test_tree_attention_refuses(lib):
    call = caller(lib.tb_tree_attention, ["q", "ldq", "T", "Hq", "Hkv", "D", "kc", "vc", "pages", "page", "table", "mp", "total", "row", "B", "mq", "tree", "scale",
                                          "o", "ws", "wsb", "st", "s"],
                  q=P, ldq=6144, T=8, Hq=24, Hkv=4, D=256, kc=P, vc=P, pages=9, page=64, table=P, mp=8, total=P, row=P, B=4, mq=2, tree=None, scale=0.0625,
                  o=P, ws=P, wsb=1 << 40, st=None, s=None)
    for name in ("q", "kc", "vc", "table", "total", "row", "o"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(tree=P + 4) == call(ws=P + 8) == -6
    assert call(Hq=22) == call(Hq=0) == call(Hkv=0) == call(ldq=6143) == call(ldq=6140) == call(B=0) == call(T=-1) == call(mq=0) == call(mp=0) == call(pages=0) == -2
    assert call(D=96, ldq=8192) == call(D=512, ldq=16384) == call(page=65) == -3
    assert call(mq=65) == -8
    assert call(scale=0.0) == call(scale=-1.0) == call(scale=float("nan")) == call(scale=float("inf")) == -4
    assert call(T=0) == 0
    need = lib.tb_tree_attention_workspace_size(4, 8, 2, 24, 4, 256)
    if need:
        assert call(wsb=need - 1) == call(ws=None, wsb=0) == -7


def test_prompt_attention_refuses(lib):
    call = caller(lib.tb_prompt_attention, ["q", "ldq", "k", "ldk", "v", "ldv", "Tq", "Tk", "Hq", "Hkv", "D", "qs", "ks", "B", "scale", "o", "st", "s"],
                  q=P, ldq=6144, k=P, ldk=1024, v=P, ldv=1024, Tq=8, Tk=9, Hq=24, Hkv=4, D=256, qs=P, ks=P, B=2, scale=0.0625, o=P, st=None, s=None)
    for name in ("q", "k", "v", "qs", "ks", "o"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(Hq=22) == call(ldq=6136) == call(ldk=1016) == call(ldv=1020) == call(B=0) == call(Tq=-1) == call(Tk=-1) == call(Hkv=0) == -2
    assert call(D=80) == -3
    assert call(scale=0.0) == call(scale=float("inf")) == -4
    assert call(Tq=0) == 0


def test_gated_delta_refuses(lib):
    call = caller(lib.tb_gated_delta, ["q", "ldq", "k", "ldk", "v", "ldv", "g", "beta", "T", "Hk", "Hv", "D", "row", "B", "ml", "norm", "scale", "si", "xi", "ni", "so",
                                       "xo", "no", "o", "ws", "wsb", "st", "s"],
                  q=P, ldq=2048, k=P, ldk=2048, v=P, ldv=6144, g=P, beta=P, T=70, Hk=16, Hv=48, D=128, row=P, B=2, ml=64, norm=1, scale=0.1, si=P, xi=None, ni=2,
                  so=P, xo=None, no=2, o=P, ws=P, wsb=1 << 40, st=None, s=None)
    for name in ("q", "k", "v", "g", "beta", "row", "o"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P + 2}) == -6, name
    assert call(si=P + 4) == call(so=P + 8) == call(xi=P + 1) == call(xo=P + 2) == call(ws=P + 4) == -6
    assert call(Hv=40) == call(Hk=0) == call(ldq=2040) == call(ldk=2052) == call(ldv=6136) == call(B=0) == call(T=-1) == call(ml=-1) == -2
    assert call(ni=1) == call(no=1) == call(ni=0, xi=P) == -2  # without slots each request needs a row of its own
    assert call(D=64) == call(D=256, ldq=8192, ldk=8192, ldv=16384) == -3
    assert call(scale=float("nan")) == call(scale=float("-inf")) == -4
    need = lib.tb_gated_delta_workspace_size(70, 2, 64, 16, 48)
    if need:
        assert call(wsb=need - 1) == -7


def test_binding_refuses_layouts_it_cannot_pass_on():
    import torch

    import ternary_hadamard_rotated_gb300 as tb

    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    for bad in (q.float(), q.transpose(0, 1).contiguous().transpose(0, 1), torch.zeros(4, 2, 128, dtype=torch.float16)[..., ::2], q.flatten(1)):
        with pytest.raises(ValueError):
            tb.tb_prompt_attention(bad, q, q, i, i, q)
    with pytest.raises(ValueError):
        tb.tb_prompt_attention(q, q, q, i.long(), i, q)
    with pytest.raises(ValueError):
        tb.tb_prompt_attention(q, q, q, i, i, q[:3])
    with pytest.raises(ValueError):
        tb.tb_prompt_attention(q, q, q[:3], i, i, q)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        tb.tb_cache_write(q, q, torch.zeros(4, dtype=torch.int32), c, c)
    with pytest.raises(ValueError):
        tb.tb_cache_write(q, q, torch.zeros(4, dtype=torch.int64), c, c.transpose(1, 2).contiguous())
    with pytest.raises(ValueError):
        tb.tb_tree_attention(q, c, c, i[None], i[:1], i, 4, q, tree=torch.zeros(4, dtype=torch.int32))
    g = torch.zeros(4, 2)
    with pytest.raises(ValueError):
        tb.tb_gated_delta(q, q, q, g.half(), g, i, 4, q)


@pytest.mark.parametrize("ml", [1, 64])
def test_gated_delta_refuses_tokens_too_far_apart(lib, ml):
    """More than 2^31 elements between two tokens: refused for q, k and v alike, on both of its paths."""
    call = caller(lib.tb_gated_delta, ["q", "ldq", "k", "ldk", "v", "ldv", "g", "beta", "T", "Hk", "Hv", "D", "row", "B", "ml", "norm", "scale", "si", "xi", "ni", "so",
                                       "xo", "no", "o", "ws", "wsb", "st", "s"],
                  q=P, ldq=2048, k=P, ldk=2048, v=P, ldv=6144, g=P, beta=P, T=70, Hk=16, Hv=48, D=128, row=P, B=2, ml=ml, norm=1, scale=0.1, si=P, xi=None, ni=2,
                  so=P, xo=None, no=2, o=None, ws=P, wsb=1 << 40, st=None, s=None)
    assert call() == -1  # everything is looked at but o
    for name in ("ldq", "ldk", "ldv"):
        assert call(**{name: 2 ** 31}) == -1
        assert call(**{name: 2 ** 31 + 8}) == -2, name


def test_binding_takes_one_token_of_any_row_length():
    """The distance of two tokens means nothing where there is one, as in a decode step's slice of a projection."""
    import torch

    import ternary_hadamard_rotated_gb300 as tb

    f16 = torch.float16
    wide = torch.zeros(3, 515, dtype=f16)
    all3 = wide[:, :512].unflatten(1, (2, 256))
    one = all3[1:2]
    assert one.stride(0) == 515 and tb._tokens("q", one, f16) == 512
    assert tb._tokens("q", all3[1:1], f16) == 512
    assert tb._tokens("q", all3, f16) == 515  # (which the calls refuse)
