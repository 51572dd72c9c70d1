"""Host-side checks of the 4-bit weight product (no GPU needed): sizes of the image, the
struct's layout, refusals before any launch, and the reference the GPU tests use."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from integer_quantized_nn_gb300 import qnn
import _w4

pytestmark = pytest.mark.cpu
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qnn.h")


@pytest.fixture(scope="module")
def lib():
    return qnn.load()


def test_image_sizes(lib):
    size = qnn.qnn_gemv_w4_packed_bytes
    assert size(qnn.w4_geom(4096, 4096, 128)) == 256 * 32 * 1024 + 256 * 32 * 16 * 4
    assert size(qnn.w4_geom(4096, 4096, 128, scale_dt="bf16")) == 256 * 32 * 1024 + 256 * 32 * 16 * 2
    # ragged: 17 channels = 2 tiles, 130 inputs = 2 steps, 5 groups of 32; zero points behind the scales
    assert size(qnn.w4_geom(17, 130, 32, w_dt="u4", scale_dt="f16")) == 2 * 2 * 1024 + 2 * 5 * 16 * 2 + 2 * 5 * 16
    # one group over all inputs
    assert size(qnn.w4_geom(16, 64, 1 << 20)) == 1024 + 64
    for bad in (dict(N=0), dict(K=0), dict(K=63), dict(K=(1 << 30) + 2), dict(group=0), dict(group=48),
                dict(group=-32), dict(w_dt="s8"), dict(scale_dt="s32")):
        assert size(qnn.w4_geom(**{**dict(N=16, K=64, group=32), **bad})) == 0, bad


def test_prepack_refusals(lib):
    def call(W=16, scale=16, zero=None, out=128, **geom):
        g = qnn.w4_geom(**{**dict(N=16, K=64, group=32), **geom})
        return lib.qgemv_prepack_w4(W, scale, zero, ctypes.byref(g), out, None)
    for bad in (dict(W=None), dict(scale=None), dict(out=None), dict(zero=16), dict(w_dt="u4"), dict(K=63),
                dict(group=16), dict(w_dt="u8")):
        assert call(**bad) == qnn.QNN_ERR_INVALID_ARG, bad
    for bad in (dict(W=20), dict(scale=20), dict(out=64), dict(w_dt="u4", zero=20)):
        assert call(**bad) == qnn.QNN_ERR_ALIGNMENT, bad
    assert lib.qgemv_prepack_w4(16, 16, None, None, 16, None) == qnn.QNN_ERR_INVALID_ARG


def test_product_refusals(lib):
    def call(x=16, x_dt="bf16", ldx=0, W=128, M=1, bias=None, y=16, y_dt="bf16", ldy=0, **geom):
        g = qnn.w4_geom(**{**dict(N=16, K=64, group=32), **geom})
        return lib.qgemv_w4(x, qnn.DTYPES[x_dt], ldx, W, ctypes.byref(g), M, bias, y, qnn.DTYPES[y_dt], ldy, None)
    for bad in (dict(x=None), dict(W=None), dict(y=None), dict(M=-1), dict(ldx=63), dict(ldy=15), dict(ldx=-1),
                dict(group=33), dict(N=-16)):
        assert call(**bad) == qnn.QNN_ERR_INVALID_ARG, bad
    for bad in (dict(x_dt="s8"), dict(y_dt="s8"), dict(y_dt="f16"), dict(x_dt="f32"), dict(M=1 << 40)):
        assert call(**bad) == qnn.QNN_ERR_UNSUPPORTED, bad
    for bad in (dict(x=20), dict(W=64), dict(y=18), dict(bias=20)):
        assert call(**bad) == qnn.QNN_ERR_ALIGNMENT, bad
    assert call(M=0, x=None, y=None) == qnn.QNN_OK
    assert lib.qgemv_w4(16, 6, 0, 16, None, 1, None, 16, 6, 0, None) == qnn.QNN_ERR_INVALID_ARG


@pytest.mark.parametrize("x_dt, rows", [("bf16", 32), ("f16", 32), ("f32", 10)])
def test_more_rows_than_a_grid_has_passes(lib, x_dt, rows):
    """Refused before the rows are multiplied by anything: 3 M of fp32 rows passes 64 bits."""
    g = qnn.w4_geom(N=16, K=64, group=32)
    for M in (65535 * rows + 1, 1 << 40, (1 << 62) + 1, (1 << 63) - 1):
        assert lib.qgemv_w4(16, qnn.DTYPES[x_dt], 0, 128, ctypes.byref(g), M, None, 16, qnn.DTYPES["f32"], 0,
                            None) == qnn.QNN_ERR_UNSUPPORTED, M


def test_integer_calls_refuse_the_float_types(lib):
    shape = (ctypes.c_int64 * 2)(4, 8)
    p = qnn.qparams("sym")
    p.scale = 16
    for dt in (6, 7):
        assert lib.q_quantize(16, 16, dt, 2, shape, ctypes.byref(p), None) != qnn.QNN_OK
        assert lib.q_dequantize(16, dt, 16, 2, shape, ctypes.byref(p), None) != qnn.QNN_OK


def test_geometry_struct_matches_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "qnn.h"', "int main(void) {",
             '    printf("%zu", sizeof(qnn_w4_geom));']
    lines += [f'    printf(" %zu", offsetof(qnn_w4_geom, {f}));' for f, _ in qnn.W4Geom._fields_]
    (tmp_path / "g.c").write_text("\n".join(lines + ["    return 0;", "}"]))
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(tmp_path / "g.c"), "-o", str(tmp_path / "g")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "g")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(qnn.W4Geom)] + [getattr(qnn.W4Geom, f).offset for f, _ in qnn.W4Geom._fields_]


@pytest.mark.parametrize("w_dt", ["s4", "u4"])
def test_reference_against_single_terms(w_dt):
    """The reference itself, summed term by term from the packed bytes."""
    p = _w4.make(np.random.default_rng(3), 2, 5, 70, 32, "f32", w_dt, "f16", True)
    y, _ = _w4.reference(p)
    W, s = p["W"].numpy(), p["scale"].double().numpy()
    for m in range(2):
        for n in range(5):
            t = float(p["bias"][n])
            for k in range(70):
                c = int(W[n, k // 2]) >> (4 * (k % 2)) & 15
                c = c - int(p["zero"][n, k // 32]) if w_dt == "u4" else c - 16 * (c > 7)
                t += float(p["x"][m, k]) * c * s[n, k // 32]
            assert abs(t - y[m, n]) < 1e-12
