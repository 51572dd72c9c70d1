"""Decoding with trees of drafted tokens over a quantised cache of keys and values.

    python examples/tree_decoding.py

A small transformer with random weights (norms by q_block_norm, attention by q_kv_attn; its linears are
plain products) continues a batch of prompts of different lengths:

1. the prompts enter the cache in chunks: q_kv_write quantises their keys and values, q_kv_attn attends to
   what is there and to the chunk up to each token;
2. a step drafts a tree of tokens for each sequence (the same model without its attention), writes all nodes,
   attends along the tree's branches with a mask of bits, and takes the longest path on which the
   model agrees with the draft: q_kv_keep moves that path's keys and values together, and the
   sequence's length, on the device, grows by it;
3. the same, one token a step, for comparison; and the attention of a step against fp32 torch on the values
   that q_kv_read gives back.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from integer_quantized_nn_gb300 import qnn  # noqa: E402


class Tree:
    """`width` children to every node but the last level's, level after level; node 0 is the root."""

    def __init__(self, width, depth):
        self.parent, level = [-1], [0]
        for _ in range(depth):
            below = []
            for node in level:
                below += range(len(self.parent), len(self.parent) + width)
                self.parent += [node] * width
            level = below
        self.size, self.width = len(self.parent), width
        words = -(-self.size // 32)
        bits = torch.zeros(self.size, 32 * words, dtype=torch.int64)
        for node in range(self.size):
            at = node
            while at >= 0:
                bits[node, at] = 1
                at = self.parent[at]
        self.mask = (bits.view(self.size, words, 32) << torch.arange(32)).sum(2).to(torch.int64)
        self.mask = torch.where(self.mask >= 2 ** 31, self.mask - 2 ** 32, self.mask).to(torch.int32).cuda()
        self.children = [[c for c in range(self.size) if self.parent[c] == n] for n in range(self.size)]


class Layer:
    def __init__(self, C, heads, heads_q, D, kv, batch, most, gen):
        def normal(*shape, std):
            return torch.empty(shape, device="cuda").normal_(0.0, std, generator=gen).bfloat16()
        self.heads, self.heads_q, self.D = heads, heads_q, D
        self.qkv = normal(C, (heads_q + 2 * heads) * D, std=C ** -0.5)
        self.out = normal(heads_q * D, C, std=1.5 * (heads_q * D) ** -0.5)
        self.mlp = normal(C, C, std=C ** -0.5)
        self.norm = qnn.block_norm(pre="rms")
        self.geom = qnn.kv_geom(heads, D, 16, kv_dt=kv)
        pages = batch * -(-most // 16)
        self.pages = torch.empty((pages, qnn.qnn_kv_page_bytes(self.geom)), dtype=torch.uint8, device="cuda")
        self.table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(batch, -1)

    def normed(self, r):
        h = torch.empty(r.shape, dtype=torch.bfloat16, device="cuda")
        qnn.q_block_norm(r, "f32", None, "bf16", r.shape[0], r.shape[1], self.norm, h=h)
        return h

    def attend(self, h, lens, starts, tokens, mask, write=True):
        """The heads' output; q, the call's sequences and the logarithms are left for who wants them."""
        rows = h.shape[0]
        fused = h @ self.qkv  # q, k and v side by side
        pitch, at_k, at_v = fused.shape[1], self.heads_q * self.D, (self.heads_q + self.heads) * self.D
        self.seqs = qnn.kv_seqs(self.pages, self.table, lens, rows, tokens, starts=starts)
        self.q = fused[:, :at_k]
        if write:
            qnn.q_kv_write(fused[:, at_k:], fused[:, at_v:], "bf16", self.geom, self.seqs, ld_k=pitch, ld_v=pitch)
        out = torch.empty(rows, at_k, dtype=torch.bfloat16, device="cuda")
        work = torch.empty(qnn.qnn_kv_attn_workspace_bytes(self.geom, self.seqs, self.heads_q), dtype=torch.uint8,
                           device="cuda")
        qnn.q_kv_attn(self.q, "bf16", self.heads_q, self.geom, self.seqs, self.D ** -0.5, out, work, mask=mask,
                      ld_q=pitch)
        return out


class Model:
    def __init__(self, vocabulary, C, layers, heads, heads_q, D, kv, batch, most, gen):
        self.embed, self.head = (torch.empty(vocabulary, C, device="cuda").normal_(generator=gen) for _ in range(2))
        self.layers = [Layer(C, heads, heads_q, D, kv, batch, most, gen) for _ in range(layers)]
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.batch = batch

    def logits(self, r):
        return self.layers[0].normed(r).float() @ self.head.T

    def __call__(self, tokens, starts=None, most=0, mask=None):
        """Logits of the newest tokens, which are in the cache afterwards; lens counts them already."""
        r = self.embed[tokens]
        for layer in self.layers:
            r = r + (layer.attend(layer.normed(r), self.lens, starts, most, mask) @ layer.out).float()
            r = r + torch.relu(layer.normed(r) @ layer.mlp).float()
        return self.logits(r)

    def draft(self, tokens, width):
        r = self.embed[tokens]
        for layer in self.layers:
            r = r + torch.relu(layer.normed(r) @ layer.mlp).float()
        return self.logits(r).topk(width).indices

    def prompt(self, prompts, chunk):
        """The prompts' tokens but their last, a chunk of each at a time; the last ones."""
        parts = [p[:-1] for p in prompts]
        for at in range(0, max(len(p) for p in parts), chunk):
            pieces = [p[at:at + chunk] for p in parts]
            counts = torch.tensor([len(p) for p in pieces], dtype=torch.int32, device="cuda")
            self.lens += counts
            starts = torch.cat([counts.new_zeros(1), counts.cumsum(0, dtype=torch.int32)])
            self(torch.cat(pieces), starts=starts, most=max(len(p) for p in pieces))
        return torch.stack([p[-1] for p in prompts])


def decode(model, tree, roots, steps):
    """The tokens of each sequence, at least one for each step; and the last step's attention, checked."""
    found = [[] for _ in range(model.batch)]
    mask = tree.mask.repeat(model.batch, 1)
    error = 0.0
    for step in range(steps):
        nodes = torch.empty(model.batch, tree.size, dtype=torch.int64, device="cuda")
        nodes[:, 0] = roots
        for n, below in enumerate(tree.children):
            if below:
                nodes[:, below[0]:below[-1] + 1] = model.draft(nodes[:, n], tree.width)
        model.lens += tree.size
        best = model(nodes.view(-1), most=tree.size, mask=mask).argmax(1).view(model.batch, -1)
        if step == steps - 1:
            error = compare(model, tree)
        # the path on which the model agrees
        nodes_h, best_h = nodes.tolist(), best.tolist()
        keep = torch.zeros(model.batch, tree.size, dtype=torch.int32)
        counts = []
        for b in range(model.batch):
            path = [0]
            while True:
                on = [c for c in tree.children[path[-1]] if nodes_h[b][c] == best_h[b][path[-1]]]
                if not on:
                    break
                path.append(on[0])
            keep[b, :len(path)] = torch.tensor(path)
            counts.append(len(path))
            found[b] += [best_h[b][n] for n in path]
        keep, kept = keep.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")
        for layer in model.layers:
            qnn.q_kv_keep(layer.geom, layer.seqs, keep, kept)
        model.lens -= tree.size - kept
        roots = torch.tensor([f[-1] for f in found], device="cuda")
    return found, error


def compare(model, tree):
    """The last layer's attention over the whole cache against fp32 torch: the largest error over the deviation."""
    layer, B, T = model.layers[-1], model.batch, tree.size
    lens = model.lens.tolist()
    starts = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    whole = qnn.kv_seqs(layer.pages, layer.table, model.lens, sum(lens), max(lens), starts=starts)
    k, v = (torch.empty(sum(lens), layer.heads, layer.D, device="cuda") for _ in range(2))
    qnn.q_kv_read(k, v, "f32", layer.geom, whole)
    q = layer.q.reshape(B, T, layer.heads, -1, layer.D).float()
    out = torch.empty(B * T, layer.heads_q * layer.D, dtype=torch.bfloat16, device="cuda")
    work = torch.empty(qnn.qnn_kv_attn_workspace_bytes(layer.geom, layer.seqs, layer.heads_q), dtype=torch.uint8,
                       device="cuda")
    mask = tree.mask.repeat(B, 1)
    qnn.q_kv_attn(layer.q, "bf16", layer.heads_q, layer.geom, layer.seqs, layer.D ** -0.5, out, work, mask=mask,
                  ld_q=layer.q.stride(0))
    assert qnn.qnn_check_device_error() == qnn.QNN_OK
    bits = (tree.mask[:, :, None] >> torch.arange(32, device="cuda")).bitwise_and(1).view(T, -1)[:, :T].bool()
    worst, at = 0.0, 0
    for b in range(B):
        kb, vb = k[at:at + lens[b]], v[at:at + lens[b]]
        at += lens[b]
        see = torch.cat([torch.ones(T, lens[b] - T, dtype=torch.bool, device="cuda"), bits], 1)
        x = torch.einsum("thgd,nhd->thgn", q[b], kb) * layer.D ** -0.5
        p = x.masked_fill(~see[:, None, None, :], float("-inf")).softmax(-1)
        want = torch.einsum("thgn,nhd->thgd", p, vb)
        worst = max(worst, float((out.view(B, T, -1)[b] - want.reshape(T, -1)).abs().max() / want.std()))
    return worst


def main(vocabulary=2000, C=512, layers=2, heads=2, heads_q=8, D=64, kv="s8", lengths=(300, 41, 170, 2), steps=24, width=2,
         depth=3, chunk=128):
    found = {}
    prompts = [torch.randint(vocabulary, (n,), generator=torch.Generator().manual_seed(n)).cuda() for n in lengths]
    tokens = {}
    for name, tree in (("trees", Tree(width, depth)), ("single tokens", Tree(1, 0))):
        gen = torch.Generator(device="cuda").manual_seed(1)
        count = steps if name == "trees" else max(len(t) for t in tokens["trees"])
        most = max(lengths) + (steps + 1) * (depth + 1) + tree.size
        model = Model(vocabulary, C, layers, heads, heads_q, D, kv, len(lengths), most, gen)
        tokens[name], found["error " + name] = decode(model, tree, model.prompt(prompts, chunk), count)
    made = sum(len(t) for t in tokens["trees"])
    found["tokens a step"] = made / (steps * len(lengths))
    # where the two part the logits were nearly equal: the sums of different kernels are rounded differently
    same = 0
    for a, b in zip(tokens["trees"], tokens["single tokens"]):
        same += next((i for i, (x, y) in enumerate(zip(a, b)) if x != y), len(a))
    found["same"] = same / made
    return found


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--kv", default="s8", choices=["s8", "u4"])
    parser.add_argument("--steps", type=int, default=24)
    args = parser.parse_args()
    for key, value in main(kv=args.kv, steps=args.steps).items():
        print(f"{key:24s} {value:.4g}")
