"""q_block_norm and q_block_norm_backward at the edges of their ranges of values and sizes."""
import numpy as np
import pytest
import torch

from integer_quantized_nn_gb300 import qnn
import _blocknorm as bn
from test_gpu_blocknorm import block_norm, check_backward, check_codes, check_forward, run_backward, run_forward, stored

pytestmark = pytest.mark.gpu


# a warp and a block a row, by direct loads and through rings, whole vectors and single elements
@pytest.mark.parametrize("rows,C", [(60, 96), (60, 101), (60, 2048), (60, 5001), (60, 8200), (20000, 136),
                                    (1500, 2040)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_codes_of_tiny_rows(dt, rows, C):
    """max|h| from 2^-90 down to the smallest values, where 127 / max|h| passes the fp32 range."""
    p = bn.make(31, rows, C, dt, dt, post="none", pre="none", with_y=False)
    r = p["r"].double() * torch.exp2(-90.0 - torch.arange(rows, dtype=torch.float64) % 60)[:, None]
    r[:, ::5] = 0
    p["r"] = r.to(bn.TORCH[dt])
    codes, scale = run_forward(p, s8=True)[1:]
    v = p["r"].double()
    top = v.abs().max(1).values
    assert bool((scale.cpu().numpy() == top.float().numpy() / np.float32(127)).all())
    codes, some = codes.double().cpu(), top > 0
    assert 0 < int(some.sum()) and bool((codes[~some] == 0).all())
    # two roundings of at most 127, then the nearest integer
    off = (codes[some] - v[some] * (127 / top[some])[:, None]).abs()
    assert float(off.max()) <= 0.5 + 127 * 2 * bn.U * 1.01
    assert bool((codes[some].abs().max(1).values == 127).all())


@pytest.mark.parametrize("rows", [1, 2, 3, 2000])
@pytest.mark.parametrize("gate_rows", [1 << 31, 1 << 62, (1 << 63) - 1])
def test_a_gate_group_longer_than_any_tensor(gate_rows, rows):
    """One group, of all rows, whatever its length is beyond them."""
    p = bn.make(32, rows, 64, "f32", "bf16", post="layer", gate="rows", gate_rows=gate_rows)
    check_forward(p, *run_forward(p)[:2])
    check_backward(p, stored(p), run_backward(p, stored(p)))


def equal_values(rows, C, dt, **k):
    """Rows of 1000 (1000 C is an integer below 2^24: its fp32 sum is exact in any order)."""
    assert 1000 * C < 1 << 24
    p = bn.make(33, rows, C, dt, dt, **k)
    for name in ("r", "y"):
        if p[name] is not None:
            p[name][:] = 1000
    return p


def check_equal_values(rows, C, dt):
    """A LAYER row of equal values is exactly zero once its mean is taken off."""
    p = equal_values(rows, C, dt, post="layer", pre="none", gate="all", beta=False)
    assert bool((run_forward(p)[0] == 1000).all())
    got = run_backward(p, p["r"])
    assert bool((got["dgamma_post"] == 0).all()) and bool((got["dgate"] == 0).all())
    p = equal_values(rows, C, dt, post="none", pre="layer", with_y=False)
    h = run_forward(p)[1]
    assert bool((h.cpu() == p["beta_pre"].to(h.dtype)).all())
    assert bool((run_backward(p, p["r"])["dgamma_pre"] == 0).all())


SPANS = [(5, 64), (5, 101), (5, 768), (5, 2048), (5, 5001), (5, 8192), (5, 9001), (5, 16384), (20000, 136),
         (5000, 768), (9000, 333), (400, 8192)]


@pytest.mark.parametrize("rows,C", SPANS)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_layer_rows_of_equal_values(dt, rows, C):
    check_equal_values(rows, C, dt)


# 1000 C (1 / C) in fp32 is not 1000 at these widths
@pytest.mark.parametrize("rows,C", [(5, 41), (5, 1000), (5, 2040), (5, 5017), (5, 8560), (4000, 1000), (1500, 2040)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_the_mean_of_equal_values_is_their_value(dt, rows, C):
    check_equal_values(rows, C, dt)


# more rows than blocks, at widths that a block holds without a ring
@pytest.mark.parametrize("rows,C,r_dt,y_dt,post,pre,gate", [
    (400, 8200, "bf16", "bf16", "rms", "rms", dict(gate="all")),
    (330, 9001, "f32", "f16", "layer", "rms", dict(gate="rows", gate_rows=7)),
    (320, 16384, "f16", "f16", "layer", "layer", dict(gate="rows", gate_rows=1)),
    (310, 16385, "f32", "f32", "none", "layer", dict(gate="rows", gate_rows=200)),
    (310, 32768, "f32", "bf16", "layer", "layer", {}),
])
def test_many_rows_beyond_the_rings(rows, C, r_dt, y_dt, post, pre, gate):
    p = bn.make(35, rows, C, r_dt, y_dt, post, pre, beta=pre == "layer", a=0.9, b=0.6, **gate)
    check_forward(p, *run_forward(p)[:2])
    codes, scale = run_forward(p, s8=True, want_r=False)[1:]
    check_codes(p, codes, scale)
    check_backward(p, stored(p), run_backward(p, stored(p)))


@pytest.mark.parametrize("C", [64, 101])
def test_the_pitch_of_one_row_is_not_used(C):
    p = bn.make(34, 1, C, post="layer", gate="all")
    r, y, dh, dr_out = (p[k].cuda() for k in ("r", "y", "dh", "dr_out"))

    def run(ld):
        q = block_norm(p)
        q.ld_r = q.ld_y = q.ld_h = ld
        out = [torch.zeros_like(r) for _ in range(4)] + [torch.zeros(C, device="cuda") for _ in range(4)]
        qnn.q_block_norm(r, "f32", y, "f32", 1, C, q, r_out=out[0], h=out[1])
        ws = torch.empty(qnn.qnn_block_norm_backward_workspace_bytes(1, C, q), dtype=torch.uint8, device="cuda")
        qnn.q_block_norm_backward(out[0], "f32", y, "f32", 1, C, q, dh, dr_out, out[2], out[3], ws,
                                  dgamma_pre=out[4], dbeta_pre=out[5], dgamma_post=out[6], dbeta_post=out[7])
        assert qnn.qnn_check_device_error() == qnn.QNN_OK
        return out
    assert all(torch.equal(a, b) for a, b in zip(run(0), run(1 << 62)))
