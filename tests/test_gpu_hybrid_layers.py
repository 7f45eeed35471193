"""The example's phases against one another: decoding and verifying after a prompt give what one prompt
of the same tokens gives.  The two ways round at different places (a chunk's products and a step's, a
tile's weights and a page's, fp16 hidden states between the layers, each through linears that differ by
the token count's kernel): ten roundings of 2^-11 that add up give 5e-3."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layers.py")
    spec = importlib.util.spec_from_file_location("hybrid_layers", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("lens,steps,parents", [
    ([70, 1, 33], 3, [[-1, 0, 0, 2], [-1], [-1, -1, 1]]),
    ([200], 20, [[-1, 0, 1, 2, 2, 1, -1]]),
])
def test_phases_agree(lens, steps, parents):
    worst, draft = example().run(lens, steps, parents, hidden=1024, key_heads=2, value_heads=8, heads=8, kv_heads=2, dim=128, page=16, pages=64,
                                 max_pages=40)
    assert worst < 5e-3 and draft < 5e-3
