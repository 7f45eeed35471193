"""What the logits' call reports of requests that have no rows in a step (finished, or waiting, beside those that decode)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind", ["half", "float", "in place"])
@pytest.mark.parametrize("wrong,flag", [
    ({}, 0), (dict(slot=4), "TB_DEV_BAD_ID"), (dict(slot=2 ** 31 - 1), "TB_DEV_BAD_ID"), (dict(hist_len=-1), "TB_DEV_BAD_LEN"), (dict(hist_len=21), "TB_DEV_BAD_LEN"),
    (dict(prompt_len=8), "TB_DEV_BAD_LEN"), (dict(prompt_len=-1), "TB_DEV_BAD_LEN"), (dict(bias_start=9), "TB_DEV_BAD_LEN"), (dict(slot=-1), 0)])
def test_a_request_without_rows(kind, wrong, flag):
    import ternary_hadamard_rotated_gb300 as tb

    V = 300
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(2, V, device="cuda").half()
    a = dict(row_start=ints(0, 1, 1, 2), slot=ints(0, 1, 2), hist_len=ints(20, 7, 3), prompt_len=ints(3, 7, 0), bias_start=ints(0, 1, 2, 3), bias_ids=ints(5, 6, 7),
             bias_values=torch.ones(3, device="cuda"), presence=torch.ones(3, device="cuda"))
    history = torch.randint(8, V, (4, 20), dtype=torch.int32, device="cuda")

    def run(**changed):
        out = x.clone() if kind == "in place" else torch.empty(2, V, dtype=torch.float16 if kind == "half" else torch.float32, device="cuda")
        st = ints(0)
        args = {k: v.clone() for k, v in a.items()}
        for k, v in changed.items():
            args[k][1] = v
        tb.tb_logits_adjust(out if kind == "in place" else x, out, history, dev_status=st, **args)
        return out, int(st)

    want, st = run()
    assert st == 0
    got, st = run(**wrong)
    assert st == (getattr(tb, flag) if flag else 0)
    if "bias_start" in wrong:  # (where the first request's list ends, too: it is taken as empty)
        assert torch.equal(got[1], want[1])
    else:
        assert torch.equal(got, want)
