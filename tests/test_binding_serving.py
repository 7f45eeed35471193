"""What the binding of the operators around the linears refuses before the library is reached, argument by argument."""
import pytest

torch = pytest.importorskip("torch")

F16, F32, I32, I64, F64 = torch.float16, torch.float32, torch.int32, torch.int64, torch.float64


def calls():
    """(function, its arguments by name): each one right, but that all tensors lie on the CPU."""
    import ternary_hadamard_rotated_gb300 as tb

    z = lambda *s, t=F16: torch.zeros(*s, dtype=t)  # noqa: E731
    byte = lambda n: z(n, t=torch.uint8)  # noqa: E731
    st = z(1, t=I32)
    turns, grouped = byte(tb.tb_rotary_plan_size(64)), byte(tb.tb_adapter_plan_size(4, 2))
    turn = dict(q=z(4, 2, 64), k=z(4, 1, 64), pos=z(4, t=I32), plan=turns, R=64, layout=0, q_out=z(4, 2, 64), k_out=z(4, 1, 64), dev_status=st)
    return {
        "tb_rotary_plan": dict(plan=turns, R=64, freqs=z(32, t=F64), dev_status=st),
        "tb_rotary": turn,
        "tb_rotary_cache_write": dict(turn, v=z(4, 1, 64), slots=z(4, t=I64), k_cache=z(3, 1, 16, 64), v_cache=z(3, 1, 16, 64)),
        "tb_adapter_plan": dict(row_start=z(5, t=I32), adapter=z(4, t=I32), T=4, n=2, plan=grouped, dev_status=st),
        "tb_adapter_linear": dict(x=z(4, 16), a=z(2, 8, 16), b=z(2, 24, 8), scale=z(2, t=F32), plan=grouped, y=z(4, 24), out=z(4, 24), rank=z(2, t=I32),
                                  workspace=byte(4096), dev_status=st),
        "tb_logits_adjust": dict(logits=z(4, 100), out=z(4, 100), history=z(4, 9, t=I32), hist_len=z(4, t=I32), prompt_len=z(4, t=I32), row_start=z(5, t=I32),
                                 slot=z(4, t=I32), fresh=z(4, t=I32), tree=z(4, t=I64), repetition=z(4, t=F32), presence=z(4, t=F32), frequency=z(4, t=F32),
                                 bias_start=z(5, t=I32), bias_ids=z(3, t=I32), bias_values=z(3, t=F32), mask=z(2, 4, t=I32), mask_row=z(4, t=I32), dev_status=st),
    }


NAMES = {"tb_rotary_plan": "plan freqs dev_status", "tb_rotary": "q k pos plan q_out k_out dev_status",
         "tb_rotary_cache_write": "q k v pos slots plan q_out k_out k_cache v_cache dev_status", "tb_adapter_plan": "plan row_start adapter dev_status",
         "tb_adapter_linear": "x a b scale plan y out rank workspace dev_status",
         "tb_logits_adjust": "logits out history hist_len prompt_len row_start slot fresh tree repetition presence frequency bias_start bias_ids bias_values mask "
                             "mask_row dev_status"}
PAIRS = [(fn, name) for fn, names in NAMES.items() for name in names.split()]


def test_every_tensor_of_every_call_is_named_here():
    for fn, args in calls().items():
        assert sorted(NAMES[fn].split()) == sorted(k for k, v in args.items() if isinstance(v, torch.Tensor))


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 1


@pytest.fixture
def no_library(monkeypatch):
    """The binding with a library whose calls fail the test."""
    import ternary_hadamard_rotated_gb300 as tb

    class Library:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(f"{name} was reached")

    args = calls()
    monkeypatch.setattr(tb, "_lib", Library())
    return tb, args


@pytest.mark.parametrize("fn", list(NAMES))
def test_tensors_off_the_gpu(no_library, fn):
    tb, args = no_library
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        getattr(tb, fn)(**args[fn])


@pytest.mark.parametrize("fn,name", PAIRS)
def test_a_tensor_on_another_device(no_library, fn, name):
    tb, args = no_library
    if name == NAMES[fn].split()[0]:  # the first one says where the others have to lie
        other = NAMES[fn].split()[1]
        with pytest.raises(ValueError, match=rf"^{'q_out|k' if fn.startswith('tb_rotary') and name == 'q' else 'y' if name == 'x' else other} lies on cpu, .* cuda:1$"):
            getattr(tb, fn)(**dict(args[fn], **{name: args[fn][name].as_subclass(Elsewhere)}))
        return
    with pytest.raises(ValueError, match=rf"^{name} lies on .*, the call's first tensor on cpu$"):
        getattr(tb, fn)(**dict(args[fn], **{name: args[fn][name].as_subclass(Elsewhere)}))


@pytest.mark.parametrize("fn,size", [("tb_rotary", 271), ("tb_rotary_cache_write", 271), ("tb_adapter_linear", 31)])
def test_plans_and_workspaces_that_are_no_buffers(no_library, fn, size):
    tb, args = no_library
    with pytest.raises(ValueError, match="^plan must hold at least"):
        getattr(tb, fn)(**dict(args[fn], plan=torch.zeros(size, dtype=torch.uint8)))
    with pytest.raises(ValueError, match="^plan must be contiguous"):
        getattr(tb, fn)(**dict(args[fn], plan=torch.zeros(1, dtype=torch.uint8).expand(4096)))
    if fn == "tb_adapter_linear":
        with pytest.raises(ValueError, match="^workspace must be contiguous"):
            tb.tb_adapter_linear(**dict(args[fn], workspace=torch.zeros(1, dtype=torch.uint8).expand(1 << 20)))


@pytest.mark.gpu
@pytest.mark.parametrize("fn,name", PAIRS)
def test_one_tensor_left_on_the_host(no_library, fn, name):
    tb, args = no_library
    own = {k: v.cuda() if isinstance(v, torch.Tensor) and k != name else v for k, v in args[fn].items()}
    for stream in (None, torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
        with pytest.raises(ValueError, match="lies on c|must be a CUDA tensor"):
            getattr(tb, fn)(**own, stream=stream)


# Types, shapes and strides, argument by argument.  The name of the refused argument begins the message.

def first_lines(t):
    return t[: t.shape[0] - 1]


def strided(t):
    return torch.stack([t, t], -1)[..., 0]


ANY_SIZE = {"plan", "workspace", "dev_status", "bias_ids", "history"}  # (their number of elements is their own)
FROM_THE_FIRST = {"q", "x", "logits", "adapter", "hist_len"}  # (they say how many there have to be: another argument is refused)


@pytest.mark.parametrize("fn,name", [p for p in PAIRS if p[1] not in ("plan", "workspace", "dev_status")])
def test_a_tensor_of_another_type(no_library, fn, name):
    tb, args = no_library
    other = F64 if args[fn][name].dtype is not F64 else F32
    with pytest.raises(ValueError, match=rf"^{name} must be .* got {other}"):
        getattr(tb, fn)(**dict(args[fn], **{name: args[fn][name].to(other)}))
    if fn == "tb_logits_adjust" and name == "out":
        return  # (fp32 is a type of its own there)
    near = {F16: F32, F32: F16, I32: I64, I64: I32, F64: F32}[args[fn][name].dtype]
    with pytest.raises(ValueError, match=rf"^{name} must be "):
        getattr(tb, fn)(**dict(args[fn], **{name: args[fn][name].to(near)}))


@pytest.mark.parametrize("fn,name", [p for p in PAIRS if p[1] not in ANY_SIZE | FROM_THE_FIRST])
def test_a_tensor_of_another_length(no_library, fn, name):
    tb, args = no_library
    refused = {"a": "b", "k_cache": "v_cache"}.get(name, name)  # (the first of two that have to agree says how many)
    changed = args[fn][name][:, 1:].contiguous() if name == "mask" else first_lines(args[fn][name])
    with pytest.raises(ValueError, match=rf"^{refused} (must|and)"):
        getattr(tb, fn)(**dict(args[fn], **{name: changed}))


@pytest.mark.parametrize("fn,name", [("tb_rotary", "q"), ("tb_rotary_cache_write", "q"), ("tb_adapter_plan", "adapter"), ("tb_logits_adjust", "hist_len"),
                                     ("tb_adapter_linear", "x"), ("tb_logits_adjust", "logits")])
def test_the_tensor_that_says_how_many(no_library, fn, name):
    tb, args = no_library
    refused = {"q": "(k|q_out)", "adapter": "row_start", "hist_len": "row_start", "x": "y", "logits": "out"}[name]
    with pytest.raises(ValueError, match=rf"^{refused} (must|and)"):
        getattr(tb, fn)(**dict(args[fn], **{name: first_lines(args[fn][name])}))
    if name == "hist_len":
        with pytest.raises(ValueError, match="^bias_values must"):
            tb.tb_logits_adjust(**dict(args[fn], bias_ids=first_lines(args[fn]["bias_ids"])))


@pytest.mark.parametrize("fn,name", [p for p in PAIRS if p[1] not in ("plan", "workspace", "dev_status")])
def test_a_tensor_with_gaps(no_library, fn, name):
    tb, args = no_library
    with pytest.raises(ValueError, match=rf"^{name}(:| must be contiguous)"):
        getattr(tb, fn)(**dict(args[fn], **{name: strided(args[fn][name])}))


def test_more_shapes(no_library):
    tb, args = no_library
    z = lambda *s: torch.zeros(*s, dtype=F16)  # noqa: E731
    for fn, name, value, refused in [
            ("tb_rotary", "k", z(4, 1, 72), "k and q"), ("tb_rotary", "k_out", z(4, 2, 64), "k_out and k"), ("tb_rotary", "q_out", z(4, 2, 72), "q_out and q"),
            ("tb_rotary", "q", z(4, 128), "q must"), ("tb_rotary_cache_write", "v", z(4, 2, 64), "v and k"), ("tb_rotary_cache_write", "v_cache", z(3, 1, 32, 64), "v_cache must"),
            ("tb_rotary_cache_write", "k_cache", z(3, 2, 16, 64), "k_cache must"), ("tb_rotary_cache_write", "k_cache", z(3, 1, 16, 72), "k_cache must"),
            ("tb_adapter_linear", "a", z(2, 8, 24), "a must"), ("tb_adapter_linear", "a", z(2, 16, 16), "b must"), ("tb_adapter_linear", "b", z(2, 16, 8), "b must"),
            ("tb_adapter_linear", "out", z(4, 32), "out must"), ("tb_logits_adjust", "out", z(4, 99), "out must")]:
        with pytest.raises(ValueError, match=f"^{refused}"):
            getattr(tb, fn)(**dict(args[fn], **{name: value}))
