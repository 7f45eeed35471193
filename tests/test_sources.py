"""What the kernels' sources hold no instance of, whatever they compute."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ternary_hadamard_rotated_gb300", "csrc")


def test_no_load_is_multicast():
    """Replicas on several GPUs run the same kernels, and none of them may load one tile into several CTAs at once."""
    sources = glob.glob(os.path.join(CSRC, "*.cu*"))
    assert len(sources) > 20
    for path in sources:
        with open(path, encoding="utf-8") as f:
            text = f.read().replace('"\n', "").replace('"', "")
        found = re.findall(r"cp\.async\.bulk[\w.:]*\s*[\w.:]*multicast[\w.:]*", re.sub(r"\s+", " ", text))
        assert not found, (os.path.basename(path), found)
