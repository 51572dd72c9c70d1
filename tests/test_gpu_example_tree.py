"""examples/tree_decoding.py: the cache's operators and the block norm in one program."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv, width, depth", [("s8", 2, 3), ("u4", 3, 2), ("s8", 2, 5)])
def test_tree_example(kv, width, depth):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decoding.py")
    spec = importlib.util.spec_from_file_location("tree_decoding", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    found = example.main(vocabulary=300, C=256, heads=2, heads_q=4, lengths=(70, 9, 2), steps=6, kv=kv, width=width,
                         depth=depth, chunk=32)
    # bf16 outputs of some deviations: half a step of 2^-8 on values of up to five or six, and the weights' as f16
    for name in ("trees", "single tokens"):
        assert found["error " + name] < 0.05, found
    assert 1.0 <= found["tokens a step"] <= depth + 1, found


@pytest.mark.parametrize("kv, width, depth", [("s8", 2, 3), ("u4", 3, 2)])
def test_the_cache_holds_the_accepted_tokens(kv, width, depth, monkeypatch):
    """After decoding with trees the first layer's cache holds, place by place, the keys and values of the prompt and
    the accepted tokens, which its own input alone determines; paths that are not a tree's first nodes were moved."""
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tree_decoding.py")
    spec = importlib.util.spec_from_file_location("tree_decoding", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    qnn, heads, heads_q, D, vocabulary, C, steps = example.qnn, 2, 4, 64, 300, 256, 6
    moved = []
    keep_call = qnn.q_kv_keep
    monkeypatch.setattr(qnn, "q_kv_keep", lambda g, s, keep, n: (moved.append((keep.tolist(), n.tolist())),
                                                                keep_call(g, s, keep, n)))
    lengths = (70, 9, 2, 33)
    prompts = [torch.randint(vocabulary, (n,), generator=torch.Generator().manual_seed(n)).cuda() for n in lengths]
    tree = example.Tree(width, depth)
    model = example.Model(vocabulary, C, 2, heads, heads_q, D, kv, len(lengths),
                          max(lengths) + (steps + 1) * (depth + 1) + tree.size,
                          torch.Generator(device="cuda").manual_seed(1))
    found, _ = example.decode(model, tree, model.prompt(prompts, 32), steps)
    assert any(k[:m] != list(range(m)) for keep, n in moved for k, m in zip(keep, n)), "nothing moved"
    held = [torch.cat([p, torch.tensor(f, device="cuda")])[:-1] for p, f in zip(prompts, found)]
    lens = [len(h) for h in held]
    assert model.lens.tolist() == lens
    layer = model.layers[0]
    starts = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    whole = qnn.kv_seqs(layer.pages, layer.table, model.lens, sum(lens), max(lens), starts=starts)
    k, v = (torch.empty(sum(lens), heads * D, device="cuda") for _ in range(2))
    qnn.q_kv_read(k, v, "f32", layer.geom, whole)
    assert qnn.qnn_check_device_error() == qnn.QNN_OK
    fused = (layer.normed(model.embed[torch.cat(held)]) @ layer.qkv).float()
    for got, want in ((k, fused[:, heads_q * D:(heads_q + heads) * D]), (v, fused[:, (heads_q + heads) * D:])):
        # bf16 products of other row counts: a step of 2^-8 apart at most, each side half a code step off, and the steps
        # may differ as their maxima do; a code step is max / 127, or (max - min) / 15 rounded to bf16
        x = want.view(len(want), heads, D)
        span = x.abs().amax(2) / 127 if kv == "s8" else (x.amax(2).clamp(min=0) - x.amin(2).clamp(max=0)) / 15
        most = x.abs().amax(2) * 2.0 ** -7
        bound = span * 1.01 + most
        off = (got.view_as(x) - x).abs().amax(2)
        assert bool((off <= bound).all()), float((off / bound).max())
