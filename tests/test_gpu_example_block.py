"""examples/w4_mlp_block.py: the 4-bit linears, the block norm and its gradients in one program."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_block_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "w4_mlp_block.py")
    spec = importlib.util.spec_from_file_location("w4_mlp_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(C=512, hidden=1024, layers=3, rows=(1, 3, 12), tokens=200)
    # bf16 between the operators: two roundings of 2^-9 a block and one of the linears' operands,
    # on values of a few deviations, over three blocks; a wrong term would show as some tenths
    for k in ("decode 1", "decode 3", "decode 12"):
        assert found[k] < 0.06, found
    # int8 rows: half a step of max|h| / 127 (about 3.5 deviations) on each of 512 products is
    # 0.008 of the result's deviation at the root mean square; 100,000 of them reach five times that
    assert found["prompt"] < 0.06, found
    assert found["last"] < found["first"] / 4, found
