"""qgemv_w4's kernel for up to 8 columns of x (a row of fp32 makes three), where its blocks take
several sets of channels and where a result has one exact value; and its other kernel beside
qgemm_s8, with which it shares the tensor memory."""
import numpy as np
import pytest

from integer_quantized_nn_gb300 import qnn
from _util import aligned_empty, torch
from test_gpu_gemv_w4 import check, packed, product
import _w4

pytestmark = pytest.mark.gpu

# M, N, K, group, x, codes, scales, bias: two, three and five sets of channels a block on 152 SMs
# (32 channels a set, two blocks an SM)
SETS = [
    (1, 12000, 256, 128, "bf16", "s4", "f32", False),
    (8, 20011, 384, 64, "f16", "u4", "f16", True),
    (2, 20000, 130, 32, "f32", "u4", "f32", True),
    (3, 28001, 1160, 96, "bf16", "u4", "bf16", True),
    (5, 48016, 64, 32, "bf16", "s4", "bf16", True),
    (1, 40000, 200, 64, "f32", "s4", "f16", False),
]


@pytest.mark.parametrize("case", SETS, ids=lambda c: "-".join(map(str, c)))
def test_more_channels_than_the_blocks_take_at_once(case):
    M, N, K, group, x_dt, w_dt, scale_dt, bias = case
    p = _w4.make(np.random.default_rng(N + K), *case)
    check(p, product(p, x_dt, x_dt, scale_dt), x_dt)
    first = product(p, x_dt, "f32", scale_dt)
    check(p, first, "f32")
    for _ in range(3):
        assert np.array_equal(product(p, x_dt, "f32", scale_dt), first)


def in_parts(p, x_dt, scale_dt, rows):
    """y in fp32, `rows` rows of x to a call."""
    t = torch()
    g, W = packed(p, scale_dt)
    x, M = p["x"].cuda(), len(p["x"])
    bias = None if p["bias"] is None else p["bias"].cuda()
    y = t.full((M, g.N), 77.0, device="cuda")
    for m in range(0, M, rows):
        n = min(rows, M - m)
        qnn.qgemv_w4(x[m:], x_dt, W, g, n, y[m:], "f32", bias=bias)
    assert qnn.qnn_check_device_error() == qnn.QNN_OK
    return y.double().cpu().numpy()


def code_bytes(t, q):
    return t.from_numpy(((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).astype(np.uint8))


ROWS = [("f32", 1), ("f32", 2), ("f16", 1), ("f16", 8), ("bf16", 3), ("bf16", 8)]


@pytest.mark.parametrize("repeat", [1, 20])  # one and two tiles of 16 channels a warp
@pytest.mark.parametrize("x_dt,rows", ROWS)
def test_every_code_and_zero_point_is_exact(x_dt, rows, repeat):
    """Unit rows of x pick single weights: y is (q - z) s with no rounding."""
    t = torch()
    q, z = np.meshgrid(np.arange(16), np.arange(16))
    q, z = np.tile(q.reshape(-1), repeat), np.tile(z.reshape(-1), repeat)
    K = 64
    p = _w4.make(np.random.default_rng(1), K, 256 * repeat, K, 32, x_dt, "u4", "f32", False)
    p["q"][:] = q[:, None]
    p["W"] = code_bytes(t, p["q"])
    p["zero"][:] = t.from_numpy(z)[:, None]
    p["scale"][:] = 0.25
    p["x"] = t.eye(K).to(_w4.TORCH[x_dt])
    y = in_parts(p, x_dt, "f32", rows)
    assert np.array_equal(y, np.broadcast_to((q - z) * 0.25, y.shape))


@pytest.mark.parametrize("N", [16, 5120])
@pytest.mark.parametrize("rows", [1, 2])
def test_fp32_rows_keep_their_24_bits(rows, N):
    """One product an output: x times one, which the three parts hold to the last bit."""
    t = torch()
    K = 64
    p = _w4.make(np.random.default_rng(2), K, N, K, 32, "f32", "s4", "f32", False)
    v = np.random.default_rng(4).normal(0, 1, size=K).astype(np.float32) * np.float32(2.0) ** np.arange(-32, 32)
    v[:4] = [np.float32(3.4e38), np.float32(-1.2e-32), np.float32(1.9999999), np.float32(16777215)]
    p["x"] = t.diag(t.from_numpy(v.astype(np.float32)))
    p["q"][:] = 1
    p["W"] = t.full((N, K // 2), 0x11, dtype=t.uint8)
    p["scale"][:] = 1.0
    y = in_parts(p, "f32", "f32", rows)
    # the parts do not overlap, and each partial sum of them is a float
    assert np.array_equal(y, np.broadcast_to(v.astype(np.float64)[:, None], y.shape))


@pytest.mark.parametrize("x_dt,rows", ROWS)
def test_infinities_and_nan_stay_in_their_row(x_dt, rows):
    t = torch()
    p = _w4.make(np.random.default_rng(7), 8, 40, 192, 64, x_dt, "s4", "f32", True)
    p["q"][:] |= 1  # no zero weights: inf * 0 would be NaN
    p["W"] = code_bytes(t, p["q"])
    p["x"][1, 70], p["x"][2, 5] = float("inf"), float("nan")
    y = in_parts(p, x_dt, "f32", rows)
    assert np.array_equal(y[1], np.where(p["q"][:, 70] > 0, np.inf, -np.inf))
    assert np.isnan(y[2]).all()
    fine = [0, 3, 4, 5, 6, 7]
    p["x"] = p["x"][fine]
    check(p, y[fine], "f32")


@pytest.mark.parametrize("M,N", [(24, 512), (32, 2500)])  # K split over clusters of four, and not
def test_in_turn_with_the_integer_gemm(M, N):
    """Each starts while the kernel before it on the stream still runs, and takes tensor memory."""
    t = torch()
    K, rng = 1024, np.random.default_rng(14)
    p = _w4.make(rng, M, N, K, 128, "bf16", "s4", "f32", False)
    g, W = packed(p, "f32")
    x = p["x"].cuda()
    A = t.from_numpy(rng.integers(-128, 128, size=(300, K)).astype(np.int8)).cuda()
    B = t.from_numpy(rng.integers(-128, 128, size=(384, K)).astype(np.int8)).cuda()
    Bp, colsum = aligned_empty(qnn.qnn_gemm_packed_b_bytes(384, K)), t.empty(384, dtype=t.int32, device="cuda")
    qnn.qgemm_prepack_b(B, Bp, colsum)
    Ap = aligned_empty(qnn.qnn_gemm_workspace_bytes(300, K))
    qnn.qgemm_pack_a(A, "s8", 300, K, Ap)
    ys = [t.zeros(M, N, dtype=t.bfloat16, device="cuda") for _ in range(6)]
    cs = [t.zeros(300, 384, dtype=t.int32, device="cuda") for _ in range(6)]

    def turns():
        for y, c in zip(ys, cs):
            qnn.qgemv_w4(x, "bf16", W, g, M, y, "bf16")
            qnn.qgemm_s8_packed(Ap, "s8", Bp, 300, 384, K, qnn.epilogue("s32"), c)

    def right():
        t.cuda.synchronize()
        assert qnn.qnn_check_device_error() == qnn.QNN_OK
        want = (A.cpu().numpy().astype(np.int64) @ B.cpu().numpy().astype(np.int64).T)
        assert all(np.array_equal(c.cpu().numpy(), want) for c in cs)
        check(p, ys[0].double().cpu().numpy(), "bf16")
        assert all(t.equal(y, ys[0]) for y in ys)
        for b in ys + cs:
            b.zero_()

    turns()
    right()
    side, graph = t.cuda.Stream(), t.cuda.CUDAGraph()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.graph(graph, stream=side):
        turns()
    for _ in range(2):
        graph.replay()
        right()
