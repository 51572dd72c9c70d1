"""The host arithmetic of the block norm's rings (no GPU needed): which leading rows may be
copied in whole 16-byte windows, against the windows themselves."""
import os
import subprocess

import pytest

from integer_quantized_nn_gb300 import build as _build

pytestmark = pytest.mark.cpu

SOURCE = """
#include <cstdio>
#include <cmath>
#include "qnn_blocknorm.cuh"
int main()
{
    long long rows, ld;
    int elem, C;
    while (scanf("%lld %lld %d %d", &rows, &ld, &elem, &C) == 4)
        printf("%lld %d\\n", (long long)qnn::ring_rows(rows, ld, elem), qnn::window_room<1>(C, elem));
    return 0;
}
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cu").write_text(SOURCE)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-w", "-I", _build.INCLUDE, "-I", _build.CSRC,
                    str(d / "ring.cu"), "-o", str(d / "ring")], check=True)

    def run(cases):
        out = subprocess.run([str(d / "ring")], input="\n".join("%d %d %d %d" % c for c in cases), check=True,
                             capture_output=True, text=True).stdout.split()
        return list(zip(map(int, out[::2]), map(int, out[1::2])))
    return run


def test_windows_stay_in_the_tensor(ring):
    cases = [(rows, C + pad, elem, C) for rows in (1, 2, 9, 20, 33) for C in (1, 2, 3, 5, 7, 8, 15, 16, 101)
             for pad in (0, 1, 6) for elem in (2, 4)]
    for (rows, ld, elem, C), (n, room) in zip(cases, ring(cases)):
        assert 0 <= n < rows, (rows, ld, elem, C)
        end = ((rows - 1) * ld + C) * elem
        windows = [(at & ~15, (at + C * elem + 15) & ~15) for at in (r * ld * elem for r in range(rows))]
        assert all(hi <= end and hi - lo <= room for lo, hi in windows[:n]), (rows, ld, elem, C)
        assert n >= rows - 8, "more rows left out than their windows ask for"


def test_pitches_beyond_any_tensor(ring):
    """A single row's pitch is not used: any value of it leaves that row out, and none divides by zero."""
    cases = [(1, ld, elem, 101) for ld in (1 << 61, 1 << 62, (1 << 63) - 1, 3 << 61) for elem in (2, 4)]
    assert [n for n, _ in ring(cases)] == [0] * len(cases)
