"""examples/tree_decoding.py: the cache's operators and the block norm in one program."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv, width, depth", [("s8", 2, 3), ("u4", 3, 2), ("s8", 2, 5)])
def test_tree_example(kv, width, depth):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decoding.py")
    spec = importlib.util.spec_from_file_location("tree_decoding", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(vocabulary=300, C=256, heads=2, heads_q=4, lengths=(70, 9, 2), steps=6, kv=kv, width=width,
                         depth=depth, chunk=32)
    # bf16 outputs of some deviations: half a step of 2^-8 on values of up to five or six, and the weights' as f16
    for name in ("trees", "single tokens"):
        assert found["error " + name] < 0.05, found
    assert 1.0 <= found["tokens a step"] <= depth + 1, found
