"""Host-side checks of the block norm (no GPU needed): refusals before any launch, the struct's
layout, and the reference of the GPU tests against autograd and differences."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from integer_quantized_nn_gb300 import qnn
import _blocknorm as bn

pytestmark = pytest.mark.cpu
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qnn.h")
OK, INVALID, UNSUPPORTED, ALIGNMENT = (qnn.QNN_OK, qnn.QNN_ERR_INVALID_ARG, qnn.QNN_ERR_UNSUPPORTED,
                                       qnn.QNN_ERR_ALIGNMENT)


@pytest.fixture(scope="module")
def lib():
    return qnn.load()


def params(**k):
    p = qnn.block_norm(**{n: v for n, v in k.items() if n in ("post", "pre", "gate_rows", "ld_r", "ld_y", "ld_h",
                                                              "res_scale", "block_scale", "eps_post", "eps_pre")})
    for n in ("gamma_post", "beta_post", "gamma_pre", "beta_pre", "gate"):
        if n in k:
            setattr(p, n, k[n])
    return p


COMMON = [
    (INVALID, dict(rows=-1)), (INVALID, dict(C=0)), (INVALID, dict(gate_rows=-1)), (INVALID, dict(ld_r=63)),
    (INVALID, dict(ld_y=63)), (INVALID, dict(ld_h=63)), (INVALID, dict(ld_h=-64)), (INVALID, dict(eps_post=-1.0)),
    (INVALID, dict(eps_pre=float("nan"))), (INVALID, dict(res_scale=float("inf"))),
    (INVALID, dict(block_scale=float("nan"))), (INVALID, dict(gamma_post=16)), (INVALID, dict(pre="none", beta_pre=16)),
    (INVALID, dict(y=None, post="rms")), (INVALID, dict(y=None, gate=16)), (UNSUPPORTED, dict(C=32769)),
    (UNSUPPORTED, dict(r_dt="f16", y_dt="bf16")), (UNSUPPORTED, dict(r_dt="f16", y_dt="f32")),
    (UNSUPPORTED, dict(y_dt="s8")), (ALIGNMENT, dict(gamma_pre=20)), (ALIGNMENT, dict(gate=24)),
    (ALIGNMENT, dict(y=20)),
]


def test_forward_refusals(lib):
    def call(r=16, r_dt="bf16", y=16, y_dt="bf16", rows=4, C=64, r_out=16, h=16, h_dt="bf16", h_scale=None, **k):
        return lib.q_block_norm(r, qnn.DTYPES[r_dt], y, qnn.DTYPES[y_dt], rows, C, ctypes.byref(params(**k)), r_out,
                                h, qnn.DTYPES[h_dt], h_scale, None)
    for want, bad in COMMON + [
            (INVALID, dict(r=None)), (INVALID, dict(r_out=None, h=None)), (INVALID, dict(h_dt="s8")),
            (INVALID, dict(h_scale=16)), (UNSUPPORTED, dict(h_dt="f32")), (UNSUPPORTED, dict(h_dt="u8")),
            (ALIGNMENT, dict(r=20)), (ALIGNMENT, dict(r_out=20)), (ALIGNMENT, dict(h=20)),
            (ALIGNMENT, dict(h_dt="s8", h_scale=20))]:
        assert call(**bad) == want, bad
    assert call(rows=0, r=None, y=None, r_out=None, h=None) == OK
    p = params()
    p.pre = 3
    assert lib.q_block_norm(16, 7, 16, 7, 4, 64, ctypes.byref(p), 16, 16, 7, None, None) == INVALID
    assert lib.q_block_norm(16, 7, 16, 7, 4, 64, None, 16, 16, 7, None, None) == INVALID


def test_backward_refusals(lib):
    def call(r_out=16, r_dt="bf16", y=16, y_dt="bf16", rows=4, C=64, dh=16, dr_out=16, dr=16, dy=None, dgate=None,
             sums=(None,) * 4, ws=16, ws_bytes=1 << 30, **k):
        return lib.q_block_norm_backward(r_out, qnn.DTYPES[r_dt], y, qnn.DTYPES[y_dt], rows, C,
                                         ctypes.byref(params(**k)), dh, dr_out, dr, dy, dgate, *sums, ws, ws_bytes,
                                         None)
    first, third = (16, None, None, None), (None, None, 16, None)
    for want, bad in COMMON + [
            (INVALID, dict(dh=None, dr_out=None)), (INVALID, dict(r_out=None)), (INVALID, dict(y=None, dy=16)),
            (INVALID, dict(dr=None)), (INVALID, dict(dgate=16)), (INVALID, dict(sums=first)),
            (INVALID, dict(sums=third)), (INVALID, dict(sums=first, gamma_pre=16, dh=None)),
            (INVALID, dict(sums=first, gamma_pre=16, ws=None)),
            (INVALID, dict(sums=first, gamma_pre=16, ws_bytes=qnn.qnn_block_norm_backward_workspace_bytes(
                4, 64, params()) - 1)),
            (ALIGNMENT, dict(dr=20)), (ALIGNMENT, dict(dy=20)), (ALIGNMENT, dict(dh=20)), (ALIGNMENT, dict(ws=20)),
            (ALIGNMENT, dict(dr_out=20)), (ALIGNMENT, dict(sums=(20, None, None, None), gamma_pre=16))]:
        assert call(**bad) == want, bad
    assert call(rows=0, r_out=None, y=None, dh=None, dr_out=None) == OK


def test_workspace_sizes(lib):
    size = qnn.qnn_block_norm_backward_workspace_bytes
    assert size(0, 64, params()) == 0 and size(-1, 64, params()) == 0 and size(4, 0, params()) == 0
    assert 0 < size(1, 64, params()) <= size(1000, 64, params()) <= size(100000, 64, params())


def test_struct_matches_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [f for f, _ in qnn.BlockNorm._fields_]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "qnn.h"', "int main(void) {",
             '    printf("%zu", sizeof(qnn_block_norm));']
    lines += [f'    printf(" %zu", offsetof(qnn_block_norm, {f}));' for f in fields] + ["    return 0;", "}"]
    (tmp_path / "g.c").write_text("\n".join(lines))
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(tmp_path / "g.c"), "-o", str(tmp_path / "g")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "g")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(qnn.BlockNorm)] + [getattr(qnn.BlockNorm, f).offset for f in fields]


GRAD_CASES = [dict(post="rms", pre="layer", gate="rows", gate_rows=3, a=0.7, b=0.4),
              dict(post="layer", pre="rms", gate="all", beta=False), dict(post="none", pre="layer", gate="rows",
                                                                          gate_rows=1, b=2.0),
              dict(post="layer", pre="none", gate="none"), dict(post="none", pre="none", gate="all"),
              dict(post="rms", pre="rms", gamma=False, beta=False), dict(post="none", pre="rms", with_y=False)]


@pytest.mark.parametrize("case", GRAD_CASES, ids=lambda c: "-".join(f"{k}={v}" for k, v in c.items()))
def test_reference_gradients(case):
    """The explicit formulas against autograd, and autograd's r and y gradients against differences."""
    p = bn.make(3, 7, 12, **case)
    names = [n for n in ("r", "y", "gate", "gamma_post", "beta_post", "gamma_pre", "beta_pre") if p[n] is not None]
    leaf = {n: p[n].double().requires_grad_() for n in names}
    f = lambda v: bn.value(p, v["r"], v.get("y"), v.get("gate"), {k: v.get(k) for k in (
        "gamma_post", "beta_post", "gamma_pre", "beta_pre")})
    r_out, h = f(leaf)
    loss = (r_out * p["dr_out"].double() + h * p["dh"].double()).sum()
    loss.backward()
    want = bn.forward(p)
    assert torch.allclose(r_out, want["r_out"][0], rtol=0, atol=1e-12)
    assert torch.allclose(h, want["h"][0], rtol=0, atol=1e-12)
    got = bn.backward(p, r_out.detach())
    for n in names:
        assert torch.allclose(got["d" + n][0], leaf[n].grad, rtol=0, atol=1e-11), n
    d = 1e-6
    for n in names:
        v = {k: t.detach().clone() for k, t in leaf.items()}
        i = (0,) * (v[n].dim() - 1) + (1,)
        both = []
        for sign in (1, -1):
            v[n][i] = leaf[n].detach()[i] + sign * d
            r2, h2 = f(v)
            both.append(float((r2 * p["dr_out"].double() + h2 * p["dh"].double()).sum()))
        # the difference's own error: cancellation of 1e-16 |loss| / 1e-6, and d^2 of the third derivative
        assert abs((both[0] - both[1]) / (2 * d) - float(leaf[n].grad[i])) < 1e-6 * (1 + abs(float(leaf[n].grad[i]))), n
