"""qgemv_w4 on the GPU against the 64-bit reference."""
import numpy as np
import pytest

from integer_quantized_nn_gb300 import qnn
from _util import torch
import _w4

pytestmark = pytest.mark.gpu


def packed(p, scale_dt):
    t = torch()
    N, K = p["q"].shape
    g = qnn.w4_geom(N, K, p["group"], w_dt=p["w_dt"], scale_dt=scale_dt)
    out = t.empty(qnn.qnn_gemv_w4_packed_bytes(g), dtype=t.uint8, device="cuda")
    qnn.qgemv_prepack_w4(p["W"].cuda(), p["scale"].cuda(), g, out,
                         zero_point=None if p["zero"] is None else p["zero"].cuda())
    return g, out


def product(p, x_dt, y_dt, scale_dt, pad_x=0, pad_y=0, stream=None):
    """The call's y [M, N], with `pad` extra elements between rows, which stay as they were."""
    t = torch()
    g, W = packed(p, scale_dt)
    M, K = p["x"].shape
    x = t.full((M, K + pad_x), float("nan"), dtype=_w4.TORCH[x_dt], device="cuda")
    x[:, :K] = p["x"].cuda()
    y = t.full((M, g.N + pad_y), 77.0, dtype=_w4.TORCH[y_dt], device="cuda")
    bias = None if p["bias"] is None else p["bias"].cuda()
    qnn.qgemv_w4(x, x_dt, W, g, M, y, y_dt, bias=bias, ldx=K + pad_x, ldy=g.N + pad_y)
    assert qnn.qnn_check_device_error() == qnn.QNN_OK
    assert bool((y[:, g.N:] == 77.0).all())
    return y[:, :g.N].double().cpu().numpy()


def check(p, y, y_dt):
    ref, mag = _w4.reference(p)
    off = np.abs(y - ref) / _w4.tolerance(ref, mag, p["q"].shape[1], p["group"], y_dt)
    assert off.max() <= 1.0, (off.max(), np.unravel_index(off.argmax(), off.shape))


# M, N, K, group, x, codes, scales, bias
CASES = [
    (1, 1, 2, 32, "bf16", "s4", "f32", False),
    (1, 16, 64, 64, "f16", "s4", "f16", False),
    (1, 17, 66, 32, "f32", "u4", "f32", True),
    (2, 15, 30, 32, "f32", "s4", "f32", True),
    (3, 100, 96, 96, "bf16", "u4", "bf16", True),
    (4, 64, 130, 4096, "f16", "u4", "f32", False),
    (5, 203, 1000, 32, "f32", "u4", "bf16", False),
    (6, 48, 2048, 64, "f32", "s4", "f32", True),
    (7, 33, 514, 160, "bf16", "s4", "f16", True),
    (8, 256, 4096, 128, "bf16", "s4", "bf16", False),
    (9, 40, 1090, 64, "f16", "u4", "f16", True),
    (10, 31, 640, 128, "f32", "s4", "f16", False),
    (11, 1003, 320, 32, "f32", "u4", "f32", True),
    (16, 80, 4090, 256, "bf16", "u4", "f32", False),
    (17, 64, 8192, 128, "f16", "s4", "f16", True),
    (24, 96, 768, 64, "bf16", "s4", "f32", False),
    (32, 129, 1536, 128, "bf16", "u4", "bf16", True),
    (33, 16, 200, 32, "f16", "s4", "f32", False),
    (70, 50, 1030, 128, "bf16", "s4", "f32", True),
    (100, 20, 70, 32, "f32", "u4", "f32", False),
    (1, 4096, 1024, 128, "bf16", "s4", "f32", False),
    (1, 24, 32768, 128, "f16", "u4", "f32", False),
    (2, 5000, 64, 32, "bf16", "s4", "f32", True),
    # more columns than one tile of 8, or x too long for shared memory
    (8, 40, 8192, 128, "bf16", "s4", "bf16", True),
    (1, 33, 60002, 64, "f16", "u4", "f32", False),
    (3, 300, 1024, 64, "f32", "u4", "f16", True),
    (12, 2500, 512, 128, "f16", "s4", "f16", False),
    (20, 130, 4096, 32, "bf16", "u4", "bf16", True),
    (32, 5000, 384, 64, "bf16", "u4", "f32", True),
    (65, 257, 130, 32, "f16", "u4", "f32", True),
    (9, 20000, 256, 128, "bf16", "s4", "f32", False),
    (31, 1030, 3000, 96, "f32", "s4", "f32", True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_product(case):
    M, N, K, group, x_dt, w_dt, scale_dt, bias = case
    p = _w4.make(np.random.default_rng(N + K), *case)
    check(p, product(p, x_dt, x_dt, scale_dt), x_dt)


@pytest.mark.parametrize("M", [2, 5, 21])
@pytest.mark.parametrize("x_dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad_x,pad_y", [(0, 1), (1, 3), (2, 1), (4, 0), (8, 0), (24, 8)])
def test_pitches_and_fp32_results(x_dt, pad_x, pad_y, M):
    """Rows apart, on and off 16-byte boundaries, NaN between them; y in fp32."""
    p = _w4.make(np.random.default_rng(5), M, 37, 328, 64, x_dt, "u4", "f32", True)
    check(p, product(p, x_dt, "f32", "f32", pad_x, pad_y), "f32")


@pytest.mark.parametrize("x_dt", ["f32", "f16", "bf16"])
def test_every_code_and_zero_point_is_exact(x_dt):
    """Unit rows of x pick single weights: y is (q - z) s with no rounding but the result's."""
    q, z = np.meshgrid(np.arange(16), np.arange(16))
    q, z = q.reshape(-1), z.reshape(-1)
    K = 64
    p = _w4.make(np.random.default_rng(1), K, 256, K, 32, x_dt, "u4", "f32", False)
    p["q"][:] = q[:, None]
    p["W"] = _w4.torch.from_numpy(((p["q"][:, 0::2] & 15) | ((p["q"][:, 1::2] & 15) << 4)).astype(np.uint8))
    p["zero"][:] = _w4.torch.from_numpy(z)[:, None]
    p["scale"][:] = 0.25
    p["x"] = _w4.torch.eye(K).to(_w4.TORCH[x_dt])
    y = product(p, x_dt, "f32", "f32")
    assert np.array_equal(y, np.broadcast_to((q - z) * 0.25, y.shape))


def test_fp32_rows_keep_their_24_bits():
    """One product per output: x times an integer, which fp32 holds to its last bit but one."""
    t = torch()
    K = 64
    p = _w4.make(np.random.default_rng(2), K, 16, K, 32, "f32", "s4", "f32", False)
    v = np.random.default_rng(4).normal(0, 1, size=K).astype(np.float32) * np.float32(2.0) ** np.arange(-32, 32)
    v[:4] = [np.float32(3.4e38), np.float32(-1.2e-32), np.float32(1.9999999), np.float32(16777215)]
    p["x"] = t.diag(t.from_numpy(v.astype(np.float32)))
    p["q"][:] = 1
    p["W"] = t.full((16, K // 2), 0x11, dtype=t.uint8)
    p["scale"][:] = 1.0
    y = product(p, "f32", "f32", "f32")
    ref = np.broadcast_to(v.astype(np.float64)[:, None], y.shape)
    assert (np.abs(y - ref) <= np.abs(ref) * 2.0 ** -22).all()


@pytest.mark.parametrize("M", [4, 13])
@pytest.mark.parametrize("x_dt", ["f32", "f16", "bf16"])
def test_infinities_and_nan_stay_in_their_row(x_dt, M):
    t = torch()
    p = _w4.make(np.random.default_rng(7), M, 40, 192, 64, x_dt, "s4", "f32", True)
    p["q"][:] |= 1  # no zero weights: inf * 0 would be NaN
    p["W"] = t.from_numpy(((p["q"][:, 0::2] & 15) | ((p["q"][:, 1::2] & 15) << 4)).astype(np.uint8))
    p["x"][1, 70] = float("inf")
    p["x"][2, 5] = float("nan")
    y = product(p, x_dt, "f32", "f32")
    assert np.array_equal(y[1], np.where(p["q"][:, 70] > 0, np.inf, -np.inf))
    assert np.isnan(y[2]).all()
    fine = [m for m in range(M) if m not in (1, 2)]
    p["x"] = p["x"][fine]
    check(p, y[fine], "f32")


def test_zero_rows_and_zero_scales():
    p = _w4.make(np.random.default_rng(8), 3, 20, 128, 32, "bf16", "u4", "f32", False)
    p["x"][1] = 0
    p["scale"][4] = 0
    y = product(p, "bf16", "bf16", "f32")
    assert (y[1] == 0).all() and (y[:, 4] == 0).all()
    check(p, y, "bf16")


def test_zero_points_out_of_range_are_reported():
    p = _w4.make(np.random.default_rng(9), 1, 16, 64, 32, "bf16", "u4", "f32", False)
    p["zero"][3, 1] = 16
    packed(p, "f32")
    assert qnn.qnn_check_device_error() == qnn.QNN_ERR_INVALID_ARG
    assert qnn.qnn_check_device_error() == qnn.QNN_OK


def test_codes_from_q_quantize():
    """Weights quantized by the library itself, group by group, and the product they give."""
    t = torch()
    N, K, group = 48, 256, 64
    rng = np.random.default_rng(11)
    w = t.from_numpy(rng.normal(0, 0.1, size=(N, K)).astype(np.float32)).cuda()
    scale = w.view(N, K // group, group).abs().amax(2) / 7
    codes = t.empty((N, K // 2), dtype=t.uint8, device="cuda")
    qnn.q_quantize(w, codes, "s4", qnn.qparams("sym", scale=scale, per_channel=True, axis=0),
                   shape=(N * (K // group), group))
    c = codes.cpu().numpy().astype(np.int64)
    q = np.stack((c & 15, c >> 4), axis=2).reshape(N, K)
    p = {"q": q - 16 * (q > 7), "group": group, "w_dt": "s4", "W": codes.cpu(), "scale": scale.cpu(), "zero": None,
         "x": t.from_numpy(rng.normal(0, 1, size=(3, K))).bfloat16(), "bias": None}
    half_step = np.repeat(scale.double().cpu().numpy(), group, axis=1) / 2
    assert (np.abs(_w4.weights(p) - w.double().cpu().numpy()) <= half_step * 1.0001).all()
    check(p, product(p, "bf16", "bf16", "f32"), "bf16")


@pytest.mark.parametrize("case", [CASES[6], CASES[9], CASES[16], CASES[27]], ids=lambda c: "-".join(map(str, c)))
def test_equal_calls_give_equal_bits(case):
    M, N, K, group, x_dt, w_dt, scale_dt, bias = case
    p = _w4.make(np.random.default_rng(1), *case)
    first = product(p, x_dt, "f32", scale_dt)
    for _ in range(3):
        assert np.array_equal(product(p, x_dt, "f32", scale_dt), first)


@pytest.mark.parametrize("M", [4, 18])
def test_side_stream_and_graph(M):
    """On a stream of the caller's, then captured and replayed on new activations."""
    t = torch()
    case = (M, 512, 1024, 128, "bf16", "u4", "f32", True)
    p = _w4.make(np.random.default_rng(12), *case)
    g, W = packed(p, "f32")
    x, y = p["x"].cuda(), t.zeros(M, 512, dtype=t.bfloat16, device="cuda")
    bias = p["bias"].cuda()
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        qnn.qgemv_w4(x, "bf16", W, g, M, y, "bf16", bias=bias)
    t.cuda.current_stream().wait_stream(side)
    check(p, y.double().cpu().numpy(), "bf16")
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        for _ in range(3):
            qnn.qgemv_w4(x, "bf16", W, g, M, y, "bf16", bias=bias)
    p["x"] = t.from_numpy(np.random.default_rng(13).normal(0, 1, size=(M, 1024))).bfloat16()
    x.copy_(p["x"])
    y.zero_()
    graph.replay()
    t.cuda.synchronize()
    check(p, y.double().cpu().numpy(), "bf16")
