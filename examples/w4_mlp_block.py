"""An MLP block with 4-bit weights, decoded token by token, and its norms tuned.

    python examples/w4_mlp_block.py

The block is   r' = r + gate * rms(down(gelu(up(h)))),   h' = rms(r')   with `up` and `down`
held as 4-bit codes with a scale per group of input channels.  Three steps:

1. decode: qgemv_w4 for the two linears and q_block_norm for everything between them, a
   stack of such blocks captured in one CUDA graph, against fp32 torch on the same codes;
2. prompt: q_block_norm leaves h as int8 codes with a scale per row, which qgemm_s8 takes
   through its row_scale epilogue (a linear with int8 weights of its own: the 4-bit product
   is made for few rows);
3. tune: q_block_norm_backward gives the gradients of the gate and the norms' weights, and
   plain gradient steps on them lower a loss.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from integer_quantized_nn_gb300 import qnn  # noqa: E402


class Linear4:
    """W [N, K] as s4 codes with a scale per group, prepacked for qgemv_w4."""

    def __init__(self, W, group=64):
        N, K = W.shape
        self.geom = qnn.w4_geom(N, K, group, w_dt="s4", scale_dt="f32")
        scale = (W.view(N, K // group, group).abs().amax(2) / 7).contiguous()
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
        qnn.q_quantize(W, codes, "s4", qnn.qparams("sym", scale=scale, per_channel=True, axis=0),
                       shape=(N * (K // group), group))
        self.packed = torch.empty(qnn.qnn_gemv_w4_packed_bytes(self.geom), dtype=torch.uint8, device="cuda")
        qnn.qgemv_prepack_w4(codes, scale, self.geom, self.packed)
        q = torch.stack((codes & 15, codes >> 4), 2).view(N, K // group, group).float()
        self.plain = ((q - 16 * (q > 7)) * scale[:, :, None]).view(N, K)  # what the codes stand for

    def __call__(self, x, y):
        qnn.qgemv_w4(x, "bf16", self.packed, self.geom, x.shape[0], y, "bf16")


class Block:
    def __init__(self, C, hidden, gen):
        def normal(*shape, std, mean=0.0):
            return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen)
        self.up, self.down = Linear4(normal(hidden, C, std=C ** -0.5)), Linear4(normal(C, hidden, std=hidden ** -0.5))
        self.gamma_post, self.gamma_pre = normal(C, std=0.1, mean=1.0), normal(C, std=0.1, mean=1.0)
        self.gate = normal(1, C, std=0.1, mean=0.5).bfloat16()
        self.norm = qnn.block_norm(post="rms", pre="rms", gamma_post=self.gamma_post, gamma_pre=self.gamma_pre,
                                   gate=self.gate)


def rms(x, gamma, eps=1e-6):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * gamma


def decode(blocks, M, C, hidden, gen):
    """The stack on M rows in one graph; the largest error over the result's deviation."""
    r = torch.empty(M, C, device="cuda").normal_(generator=gen)
    h = torch.empty(M, C, dtype=torch.bfloat16, device="cuda")
    a, y = torch.empty(M, hidden, dtype=torch.bfloat16, device="cuda"), torch.empty_like(h)
    start = r.clone()

    def stack():
        r.copy_(start)
        qnn.q_block_norm(r, "f32", None, "bf16", M, C, blocks[0].first, h=h)
        for b in blocks:
            b.up(h, a)
            b.down(torch.nn.functional.gelu(a), y)
            qnn.q_block_norm(r, "f32", y, "bf16", M, C, b.norm, r_out=r, h=h)  # the residual stream in place

    blocks[0].first = qnn.block_norm(pre="rms", gamma_pre=blocks[0].gamma_pre)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stack()
    graph.replay()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        graph.replay()
    end.record()
    end.synchronize()

    want, p = start.double(), rms(start.double(), blocks[0].gamma_pre.double())
    for b in blocks:
        t = torch.nn.functional.gelu(p @ b.up.plain.double().t()) @ b.down.plain.double().t()
        want = want + b.gate.double() * rms(t, b.gamma_post.double())
        p = rms(want, b.gamma_pre.double())
    return float((r - want).abs().max() / want.std()), begin.elapsed_time(end) / 20 * 1e3


def prompt(M, C, N, gen):
    """h as int8 codes with row scales into qgemm_s8; the largest error over the deviation."""
    r = torch.empty(M, C, device="cuda").normal_(generator=gen)
    W = torch.randint(-127, 128, (N, C), device="cuda", generator=gen, dtype=torch.int8)
    s_w = torch.full((N,), 0.01, device="cuda")
    buf = torch.empty(qnn.qnn_gemm_packed_b_bytes(N, C) + 1024, dtype=torch.uint8, device="cuda")
    packed = buf[-buf.data_ptr() % 1024:]
    colsum = torch.empty(N, dtype=torch.int32, device="cuda")
    qnn.qgemm_prepack_b(W, packed, colsum)
    h, scale = torch.empty(M, C, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    qnn.q_block_norm(r, "f32", None, "f32", M, C, qnn.block_norm(pre="rms"), h=h, h_dt="s8", h_scale=scale)
    y = torch.empty(M, N, device="cuda")
    qnn.qgemm_s8(h, "s8", packed, M, N, C, qnn.epilogue("dequant", D=s_w, row_scale=scale), y)
    want = rms(r.double(), 1.0) @ (W.double() * 0.01).t()
    return float((y - want).abs().max() / want.std())


def tune(block, M, C, gen, steps=20, rate=0.2):
    """Gradient steps on the gate and the norms' weights towards a target; the first and last loss."""
    r = torch.empty(M, C, device="cuda").normal_(generator=gen)
    y = torch.empty(M, C, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    target = rms(r + 0.9 * rms(y.float(), 1.2), 0.8)
    r_out, h = torch.empty_like(r), torch.empty_like(y)
    dr, dy, dgate = torch.empty_like(r), torch.empty_like(y), torch.empty_like(block.gate)
    dpre, dpost = torch.empty_like(block.gamma_pre), torch.empty_like(block.gamma_post)
    ws = torch.empty(qnn.qnn_block_norm_backward_workspace_bytes(M, C, block.norm), dtype=torch.uint8, device="cuda")
    losses = []
    for _ in range(steps):
        qnn.q_block_norm(r, "f32", y, "bf16", M, C, block.norm, r_out=r_out, h=h)
        off = h.float() - target
        losses.append(float(off.square().mean()))
        dh = (2 / M * off).bfloat16()  # of the sum over the columns, the mean over the rows
        qnn.q_block_norm_backward(r_out, "f32", y, "bf16", M, C, block.norm, dh, None, dr, dy, ws, dgate=dgate,
                                  dgamma_pre=dpre, dgamma_post=dpost)
        for w, d in ((block.gate, dgate), (block.gamma_pre, dpre), (block.gamma_post, dpost)):
            w.sub_(rate * d)
    return losses[0], losses[-1]


def main(C=1024, hidden=4096, layers=4, rows=(1, 16), tokens=512):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    blocks = [Block(C, hidden, gen) for _ in range(layers)]
    found = {}
    for M in rows:
        found["decode %d" % M], us = decode(blocks, M, C, hidden, gen)
        print("decode, %2d rows: %6.1f us for %d blocks, largest error %.4f of the deviation" % (
            M, us, layers, found["decode %d" % M]))
    found["prompt"] = prompt(tokens, C, hidden, gen)
    print("prompt, %d rows: largest error %.4f of the deviation" % (tokens, found["prompt"]))
    found["first"], found["last"] = tune(blocks[0], tokens, C, gen)
    print("tune: loss %.4f -> %.4f" % (found["first"], found["last"]))
    status = qnn.qnn_check_device_error()
    if status != qnn.QNN_OK:
        raise RuntimeError(qnn.status_string(status))
    return found


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=4)
    a = ap.parse_args()
    main(a.width, a.hidden, a.layers)
