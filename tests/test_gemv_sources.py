"""What the kernels of qgemv_w4 must do on ways that no run takes on purpose, read from their
source (no GPU needed): they start before the grid ahead of them has ended, and their waits are
bounded."""
import os
import re

import pytest

from integer_quantized_nn_gb300 import build as _build

pytestmark = pytest.mark.cpu


def source(name):
    with open(os.path.join(_build.CSRC, name)) as f:
        return f.read()


def roles():
    """The branches of the columns kernel: codes, sums, x, MMA."""
    s = source("qnn_gemv_columns.cu")
    body = s[s.index("    if (warp < kCodeWarps) {"):s.index("    if (warp == kMmaWarp0) tmem_dealloc")]
    parts = re.split(r"\n    \} else (?:if \(warp < \w+\) )?\{\n", body)
    assert len(parts) == 4
    return parts


def test_every_role_waits_for_the_grid_before():
    """Ahead of its first bounded wait, whose limit would else count the time of that grid."""
    for part in roles():
        first = re.search(r"\b(?:mbar_)?wait\((?:done|full)", part)
        assert "grid_dependency_wait();" in part[:first.start()], part[:200]


def test_x_copies_have_landed_when_their_role_ends():
    """Also after a wait that gave up: nothing writes to shared memory that was given back."""
    part = roles()[2]
    loop = part.index("for (int t = first; t < n; t += kStages)")
    end = part.index("\n        }\n", loop)  # of the loop
    assert "break;" in part[loop:end]
    assert "cp.async.wait_group 0;" in part[end:]


@pytest.mark.parametrize("name", ["qnn_gemv.cuh", "qnn_gemv.cu", "qnn_gemv_columns.cu"])
def test_nothing_is_loaded_as_a_constant(name):
    """The grid before may still be writing x, the bias or the image when this one has begun, and
    __ldg is for what no one writes meanwhile (and may be moved ahead of the wait)."""
    code = re.sub(r"//.*", "", source(name))
    assert not re.findall(r"__ldg\(.*|\.nc\b.*", code)
