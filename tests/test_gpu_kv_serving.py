"""The quantised cache as a serving program uses it: prompts in chunks, trees of drafted tokens, accepted
paths, all operators one after the other, eager and replayed from a graph; and the sizes at which the
attention goes another way."""
from __future__ import annotations

import numpy as np
import pytest

import _kv
from integer_quantized_nn_gb300 import qnn
from test_gpu_kv import OK, Dev, check, near

pytestmark = pytest.mark.gpu


def torch():
    return pytest.importorskip("torch")


class Served:
    """A cache that grows: what is in it in numpy (c) and on the device."""

    def __init__(self, rng, batch, heads, group, D, page, kv, x_dt, most):
        t = torch()
        self.rng, self.group, self.scale = rng, group, D ** -0.5
        self.c = _kv.Cache(rng, [0] * batch, [0] * batch, heads, D, page, kv, x_dt)
        c = self.c
        pages = -(-most // page)
        self.geom = qnn.kv_geom(heads, D, page, kv_dt=kv)
        self.pages = t.full((batch * pages + 3, qnn.qnn_kv_page_bytes(self.geom)), 0xFF, dtype=t.uint8, device="cuda")
        table = rng.permutation(batch * pages + 3)[:batch * pages].reshape(batch, pages).astype(np.int32)
        self.table = t.from_numpy(table).cuda()
        self.lens = t.zeros(batch, dtype=t.int32, device="cuda")
        c.k = [np.zeros((0, heads, D), np.float32) for _ in range(batch)]
        c.v = [np.zeros((0, heads, D), np.float32) for _ in range(batch)]

    def floats(self, *shape):
        return torch().from_numpy(self.rng.normal(0, 1.2, size=shape)).to(_kv.TORCH[self.c.x_dt]).float().numpy()

    def grow(self, tokens):
        """The next tokens of each sequence: rows of k, v and q; they are in c from here on."""
        c = self.c
        k, v = ([self.floats(T, c.heads, c.D) for T in tokens] for _ in range(2))
        c.k, c.v = [np.concatenate(x) for x in zip(c.k, k)], [np.concatenate(x) for x in zip(c.v, v)]
        c.lens, c.tokens = [n + T for n, T in zip(c.lens, tokens)], list(tokens)
        c.starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
        c.rows = int(c.starts[-1])
        return np.concatenate(k), np.concatenate(v), self.floats(c.rows, c.heads * self.group, c.D)

    def accept(self, paths):
        c = self.c
        for b, path in enumerate(paths):
            n = c.lens[b] - c.tokens[b]
            c.k[b], c.v[b] = (np.concatenate([x[b][:n], x[b][n:][path]]) for x in (c.k, c.v))
            c.lens[b] = n + len(path)

    def compare(self, q, out, lse, sees=None):
        c = self.c
        w_out, w_lse, t_out, t_lse = _kv.attention(c, q, self.scale, sees)
        near(out.double().cpu().numpy().reshape(w_out.shape), w_out, t_out, "out")
        near(lse.double().cpu().numpy(), w_lse, t_lse, "lse")


@pytest.mark.parametrize("replayed", [False, True])
@pytest.mark.parametrize("kv, x_dt, heads, group, D, page, T", [
    ("s8", "bf16", 2, 4, 128, 16, 12), ("u4", "f16", 1, 8, 64, 32, 33), ("u4", "bf16", 2, 2, 96, 48, 3), ("s8", "f16", 1, 3, 160, 16, 7)])
def test_prompts_then_drafted_trees(kv, x_dt, heads, group, D, page, T, replayed):
    t = torch()
    rng = np.random.default_rng(D + T)
    batch, steps = 3, 4
    s = Served(rng, batch, heads, group, D, page, kv, x_dt, 300)
    c, dt, HQ = s.c, _kv.TORCH[x_dt], heads * group
    dev = lambda x: t.from_numpy(np.ascontiguousarray(x)).to(dt).cuda()
    # prompts, two chunks of them; a sequence without tokens in each
    for tokens in ([50, 0, 131], [70, 20, 0]):
        k, v, q = s.grow(tokens)
        s.lens.copy_(t.tensor(c.lens, dtype=t.int32))
        starts = t.from_numpy(c.starts).cuda()
        seqs = qnn.kv_seqs(s.pages, s.table, s.lens, c.rows, max(tokens), starts=starts)
        ws = t.empty(qnn.qnn_kv_attn_workspace_bytes(s.geom, seqs, HQ), dtype=t.uint8, device="cuda")
        out, lse = t.empty((c.rows, HQ * D), dtype=dt, device="cuda"), t.empty((c.rows, HQ), device="cuda")
        qnn.q_kv_write(dev(k), dev(v), x_dt, s.geom, seqs)
        qnn.q_kv_attn(dev(q), x_dt, HQ, s.geom, seqs, s.scale, out, ws, lse=lse)
        s.compare(q, out, lse)
    # a step: T drafted tokens of each sequence enter, are attended to along their trees, and a path of them stays
    rows, words = batch * T, -(-T // 32)
    seqs = qnn.kv_seqs(s.pages, s.table, s.lens, rows, T)
    ws = t.empty(qnn.qnn_kv_attn_workspace_bytes(s.geom, seqs, HQ), dtype=t.uint8, device="cuda")
    k_in, v_in = (t.empty((rows, heads * D), dtype=dt, device="cuda") for _ in range(2))
    q_in, out = (t.empty((rows, HQ * D), dtype=dt, device="cuda") for _ in range(2))
    k_out, v_out = t.empty_like(k_in), t.empty_like(v_in)
    lse = t.empty((rows, HQ), device="cuda")
    mask = t.empty((rows, words), dtype=t.int32, device="cuda")
    keep, n_keep = t.zeros((batch, T), dtype=t.int32, device="cuda"), t.zeros(batch, dtype=t.int32, device="cuda")

    def step():
        s.lens.add_(T)
        qnn.q_kv_write(k_in, v_in, x_dt, s.geom, seqs)
        qnn.q_kv_attn(q_in, x_dt, HQ, s.geom, seqs, s.scale, out, ws, mask=mask, lse=lse)
        qnn.q_kv_read(k_out, v_out, x_dt, s.geom, seqs)
        qnn.q_kv_keep(s.geom, seqs, keep, n_keep)
        s.lens.sub_(T).add_(n_keep)

    graph = None
    for i in range(steps):
        k, v, q = s.grow([T] * batch)
        sees = [_kv.random_tree(rng, T) for _ in range(batch)]
        paths = [np.flatnonzero(see[rng.integers(0, T)]) for see in sees]
        if i == 2:
            paths[1] = paths[1][:0]  # nothing of it is accepted
        kept = np.zeros((batch, T), np.int32)
        for b, path in enumerate(paths):
            kept[b, :len(path)] = path
        for to, x in ((k_in, k), (v_in, v), (q_in, q)):
            to.copy_(dev(x).view(to.shape))
        mask.copy_(t.from_numpy(_kv.mask_words(sees, words)))
        keep.copy_(t.from_numpy(kept))
        n_keep.copy_(t.tensor([len(p) for p in paths], dtype=t.int32))
        t.cuda.synchronize()
        if i == 0 or not replayed:
            step()
        else:
            if graph is None:
                graph = t.cuda.CUDAGraph()
                with t.cuda.graph(graph):
                    step()
            graph.replay()
        assert qnn.qnn_check_device_error() == OK
        s.compare(q, out, lse, sees)
        for got, parts in ((k_out, c.k), (v_out, c.v)):
            assert t.equal(got, dev(_kv.values(c.rows_of(parts), kv)).view(rows, -1))
        s.accept(paths)
        assert s.lens.tolist() == c.lens
    # all that is left, read back at once
    c.tokens = list(c.lens)
    c.starts = np.concatenate([[0], np.cumsum(c.tokens)]).astype(np.int32)
    c.rows = int(c.starts[-1])
    starts = t.from_numpy(c.starts).cuda()
    whole = qnn.kv_seqs(s.pages, s.table, s.lens, c.rows, max(c.tokens), starts=starts)
    k_all, v_all = (t.empty((c.rows, heads * D), dtype=dt, device="cuda") for _ in range(2))
    qnn.q_kv_read(k_all, v_all, x_dt, s.geom, whole)
    assert qnn.qnn_check_device_error() == OK
    for got, parts in ((k_all, c.k), (v_all, c.v)):
        assert t.equal(got, dev(_kv.values(np.concatenate(parts), kv)).view(c.rows, -1))


@pytest.mark.parametrize("rows", [8, 9, 16, 17, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("D, kv", [(64, "u4"), (96, "s8"), (128, "u4"), (128, "s8"), (160, "u4"), (192, "s8"), (256, "s8"),
                                   (256, "u4")])
def test_row_counts_around_a_tile(rows, D, kv):
    """As many rows of a head as a tile has, one less and one more, causal, the last tokens of longer ones."""
    c = _kv.Cache(np.random.default_rng(rows + D), [rows + 150, rows], [rows, rows // 2], 1, D, 16, kv, "bf16")
    check(c, Dev(c), 1)


@pytest.mark.parametrize("tokens, group", [(43, 3), (19, 7), (65, 4), (3, 86)])
def test_tiles_that_end_inside_a_token(tokens, group):
    c = _kv.Cache(np.random.default_rng(tokens), [tokens + 260, 40], [tokens, 1], 2, 64, 32, "s8", "f16")
    check(c, Dev(c), 2 * group)


@pytest.mark.parametrize("D, group, kv, masked", [(128, 4, "s8", False), (64, 2, "u4", True), (160, 8, "s8", False),
                                                  (96, 8, "u4", True), (64, 32, "s8", False)])
def test_prompts_beside_sequences_that_decode(D, group, kv, masked):
    """Few and many newest tokens in a batch, none too, in any order."""
    rng = np.random.default_rng(D + group)
    tokens = [1, 0, 2, 1, 1, 90, 1, 4, 1, 1, 3, 0, 1, 40, 1, 1, 1, 5, 8, 9, 1, 1, 0]
    lens = [n + int(x) for n, x in zip(tokens, rng.integers(0, 300, len(tokens)))]
    lens[4] = 1
    c = _kv.Cache(rng, lens, tokens, 2, D, 16, kv, "bf16")
    check(c, Dev(c), 2 * group, sees=[_kv.random_tree(rng, n) for n in tokens] if masked else None)


@pytest.mark.parametrize("most", [1, 12, 140])
def test_attention_of_a_large_batch(most):
    """More sequences than fit beside two tiles of rows; most have one token, one has `most`."""
    rng = np.random.default_rng(most)
    lens = [int(x) for x in rng.integers(0, 40, 2500)]
    tokens = [min(1, n) for n in lens]
    lens[1700], tokens[1700] = 200, most
    c = _kv.Cache(rng, lens, tokens, 1, 32, 16, "u4", "bf16")
    check(c, Dev(c), 1)


@pytest.mark.parametrize("most, D, kv", [(1, 128, "s8"), (9, 128, "s8"), (40, 256, "u4")])
def test_attention_of_the_largest_batch(most, D, kv):
    """4096 sequences: their sums take shared memory from everything else."""
    rng = np.random.default_rng(D + most)
    lens = [int(x) for x in rng.integers(0, 6, 4096)]
    tokens = [min(1, n) for n in lens]
    lens[3], tokens[3] = 300, most
    c = _kv.Cache(rng, lens, tokens, 1, D, 16, kv, "f16")
    check(c, Dev(c), 1)


@pytest.mark.parametrize("tokens", [1, 20, 150])
def test_no_pages_at_all(tokens):
    """Rows without tokens in a cache without pages: zeros and -inf, and nothing is read."""
    t = torch()
    geom = qnn.kv_geom(2, 64, 16, kv_dt="s8")
    pages = t.empty((0, qnn.qnn_kv_page_bytes(geom)), dtype=t.uint8, device="cuda")
    table, lens = t.full((2, 4), -1, dtype=t.int32, device="cuda"), t.zeros(2, dtype=t.int32, device="cuda")
    seqs = qnn.kv_seqs(pages, table, lens, 2 * tokens, tokens)
    q, out = (t.full((2 * tokens, 4 * 64), 3.0, dtype=t.bfloat16, device="cuda") for _ in range(2))
    k, v = (t.full((2 * tokens, 2 * 64), 3.0, dtype=t.bfloat16, device="cuda") for _ in range(2))
    lse = t.zeros((2 * tokens, 4), device="cuda")
    ws = t.empty(qnn.qnn_kv_attn_workspace_bytes(geom, seqs, 4), dtype=t.uint8, device="cuda")
    qnn.q_kv_write(k, v, "bf16", geom, seqs)
    qnn.q_kv_attn(q, "bf16", 4, geom, seqs, 0.1, out, ws, lse=lse)
    qnn.q_kv_read(k, v, "bf16", geom, seqs)
    assert qnn.qnn_check_device_error() == OK
    assert not out.any() and bool(t.isneginf(lse).all()) and not k.any() and not v.any()


def test_two_streams_with_their_own_workspaces():
    t = torch()
    rng = np.random.default_rng(5)
    c = _kv.Cache(rng, [900, 333], [30, 2], 2, 128, 16, "s8", "bf16")
    d = Dev(c)
    HQ = 8
    qs = [d.floats(rng.normal(0, 1, size=(c.rows, HQ, 128))).view(c.rows, -1) for _ in range(2)]
    n = qnn.qnn_kv_attn_workspace_bytes(d.geom, d.seqs, HQ)
    ws = [t.empty(n, dtype=t.uint8, device="cuda") for _ in range(2)]
    alone, both = ([t.empty_like(q) for q in qs] for _ in range(2))
    for i in range(2):
        qnn.q_kv_attn(qs[i], c.x_dt, HQ, d.geom, d.seqs, 0.1, alone[i], ws[i])
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            with t.cuda.stream(streams[i]):
                qnn.q_kv_attn(qs[i], c.x_dt, HQ, d.geom, d.seqs, 0.1, both[i], ws[i])
    t.cuda.synchronize()
    assert qnn.qnn_check_device_error() == OK
    assert all(t.equal(a, b) for a, b in zip(alone, both))


@pytest.mark.parametrize("kv", ["s8", "u4"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_one_large_channel(tokens, kv):
    """Keys and values of one large channel: the others' codes are near the zero point, and q is large where they are."""
    rng = np.random.default_rng(9)
    c = _kv.Cache(rng, [400], [tokens], 1, 128, 16, kv, "bf16")
    for x in (c.k[0], c.v[0]):
        x[:, :, 5] = _kv.bf16(x[:, :, 5] * 60)
    q = rng.normal(0, 3, size=(tokens, 4, 128))
    q[:, :, 5] *= 1e-3
    check(c, Dev(c), 4, q=q)
    # a row of q over many octaves
    check(c, Dev(c), 4, q=rng.normal(0, 1, size=(tokens, 4, 128)) * 2.0 ** -rng.integers(0, 30, size=(tokens, 4, 128)))


@pytest.mark.parametrize("D, kv", [(128, "s8"), (256, "u4")])
def test_many_rows_and_kept_tokens_beyond_32_bits(D, kv):
    """The last pages of a cache of more than 4 GiB, for 60 rows of a head, and tokens that move there."""
    t = torch()
    rng = np.random.default_rng(D)
    c = _kv.Cache(rng, [200, 133], [30, 25], 2, D, 256, kv, "bf16", spare=0)
    d = Dev(c, fill=False)
    pages = (5 << 30) // d.pages.shape[1]
    d.pages = t.empty((pages, d.pages.shape[1]), dtype=t.uint8, device="cuda")
    c.table[:, 0] = [pages - 1, pages - 2]
    c.num_pages = pages
    d.table.copy_(t.from_numpy(c.table))
    d.seqs = qnn.kv_seqs(d.pages, d.table, d.lens, c.rows, 30, starts=d.starts)
    whole_starts = d.ints([0, 200, 333])
    whole = qnn.kv_seqs(d.pages, d.table, d.lens, 333, 200, starts=whole_starts)
    qnn.q_kv_write(d.floats(np.concatenate(c.k)), d.floats(np.concatenate(c.v)), "bf16", d.geom, whole)
    check(c, d, 4)
    keep = t.tensor([[3, 4, 29], [0, 7, 24]], dtype=t.int32, device="cuda")
    n_keep = t.tensor([3, 3], dtype=t.int32, device="cuda")
    qnn.q_kv_keep(d.geom, d.seqs, keep, n_keep)
    for b, path in enumerate(keep.tolist()):
        n = c.lens[b] - c.tokens[b]
        for i, j in enumerate(path):
            c.k[b][n + i], c.v[b][n + i] = c.k[b][n + j].copy(), c.v[b][n + j].copy()
    check(c, d, 4)


def test_a_captured_mixed_batch():
    """A graph of prompts beside decoding sequences, replayed when others of them have the prompt."""
    t = torch()
    rng = np.random.default_rng(77)
    one, other = [1, 1, 120, 1, 1, 2, 1, 1], [1, 120, 1, 2, 1, 1, 1, 1]
    lens = [300, 250, 200, 31, 1, 64, 129, 400]
    c = _kv.Cache(rng, lens, one, 2, 64, 16, "s8", "bf16")
    d = Dev(c)
    q = t.empty((c.rows, 8 * 64), dtype=t.bfloat16, device="cuda")
    out, lse = t.empty_like(q), t.empty((c.rows, 8), device="cuda")
    ws = t.empty(qnn.qnn_kv_attn_workspace_bytes(d.geom, d.seqs, 8), dtype=t.uint8, device="cuda")
    qnn.q_kv_attn(q.zero_(), "bf16", 8, d.geom, d.seqs, 0.125, out, ws, lse=lse)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        qnn.q_kv_attn(q, "bf16", 8, d.geom, d.seqs, 0.125, out, ws, lse=lse)
    for tokens in (one, other, one):
        c.tokens = tokens
        c.starts = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
        d.starts.copy_(t.from_numpy(c.starts))
        x = d.floats(rng.normal(0, 1, size=(c.rows, 8, 64)))
        q.copy_(x.view(c.rows, -1))
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        w_out, w_lse, t_out, t_lse = _kv.attention(c, x.double().cpu().numpy(), 0.125)
        near(out.double().cpu().numpy().reshape(w_out.shape), w_out, t_out, "out")
        near(lse.double().cpu().numpy(), w_lse, t_lse, "lse")
    assert qnn.qnn_check_device_error() == OK


def test_both_kinds_of_wait_give_up_when_they_should():
    """One by the clock, one by counting probes, 40 ms each: neither much before nor long after."""
    t = torch()
    qnn.qnn_selftest_wait_timeout(1000)
    assert qnn.qnn_check_device_error() == qnn.QNN_ERR_TIMEOUT
    start, end = (t.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    qnn.qnn_selftest_wait_timeout(40_000_000)
    end.record()
    assert qnn.qnn_check_device_error() == qnn.QNN_ERR_TIMEOUT
    assert 60 < start.elapsed_time(end) < 160
    assert qnn.qnn_check_device_error() == OK


@pytest.mark.parametrize("tokens, D, kv", [(1, 32, "s8"), (20, 32, "s8"), (130, 64, "u4"), (40, 160, "s8")])
def test_first_pages_that_are_not_there(tokens, D, kv):
    """The first 128 tokens have no pages, and V is zero for a while behind them: that is reported, and the rest
    is attended to, tokens of zero V too.  Of so many heads that a block has several chunks of most of them."""
    t = torch()
    rng = np.random.default_rng(D + tokens)
    c = _kv.Cache(rng, [900], [tokens], 160, D, 16, kv, "bf16")
    there = _kv.Cache(rng, [772], [tokens], 160, D, 16, kv, "bf16")
    q = rng.normal(0, 1.5, size=(tokens, 160, D))
    for zero in (640, 900):
        c.v[0][128:zero] = 0
        d = Dev(c)
        q = d.floats(q).double().cpu().numpy()
        d.table[0, :8] = t.tensor([-1, c.num_pages, -5, 2 ** 31 - 1] * 2, dtype=t.int32)
        out, lse = d.attend(q, D ** -0.5)
        assert qnn.qnn_check_device_error() == qnn.QNN_ERR_INVALID_ARG
        there.k, there.v = [c.k[0][128:]], [c.v[0][128:]]
        w_out, w_lse, t_out, t_lse = _kv.attention(there, q, D ** -0.5)
        near(out, w_out, t_out, "out")
        near(lse, w_lse, t_lse, "lse")


@pytest.mark.parametrize("size_q, size_k", [(1e-36, 1e36), (1e36, 1e-36), (1e-38, 1e37), (1e-30, 1e30)])
@pytest.mark.parametrize("tokens, D", [(3, 64), (3, 128), (20, 64), (40, 128), (20, 256)])
def test_keys_and_queries_at_the_ends_of_the_range(tokens, D, size_q, size_k):
    """Scores of ordinary size from keys and queries whose products with anything else would not fit fp32."""
    rng = np.random.default_rng(D + tokens)
    c = _kv.Cache(rng, [300, 45], [tokens, 2], 1, D, 16, "s8", "bf16")
    c.k = [_kv.bf16(k * size_k) for k in c.k]
    q = rng.normal(0, 1, size=(c.rows, 4, D)) * size_q
    for scale in (D ** -0.5, -0.02, 3.0):
        check(c, Dev(c), 4, q=q, scale=scale)


@pytest.mark.parametrize("power", [24, 40, 110])
@pytest.mark.parametrize("tokens, heads, group, D, kv", [
    (7, 2, 1, 64, "s8"), (4, 2, 4, 64, "u4"), (7, 1, 1, 128, "s8"), (2, 3, 4, 128, "u4"), (9, 1, 3, 256, "s8"),
    (20, 2, 4, 64, "s8"), (40, 1, 4, 128, "u4"), (70, 2, 4, 128, "s8"), (20, 2, 4, 160, "s8"), (150, 1, 2, 256, "u4"),
    (120, 2, 1, 128, "s8"), (300, 1, 1, 64, "u4")])
def test_hidden_tokens_have_no_part_in_a_row(tokens, heads, group, D, kv, power):
    """Values of later tokens, and of other branches, 2^power times those that a row sees: its result is as exact
    as without them.  A row that sees one of them is as exact as its largest value lets it be."""
    rng = np.random.default_rng(tokens + D)
    c = _kv.Cache(rng, [tokens + 2600, tokens + 100, tokens], [tokens] * 3, heads, D, 16, kv, "bf16")
    sees = [_kv.random_tree(rng, tokens) for _ in range(3)]
    sees[1][::3] = False
    for b in range(3):
        first = c.lens[b] - tokens
        large = np.arange(1 + b, tokens, 3)
        c.v[b][first + large] = _kv.bf16(c.v[b][first + large] * 2.0 ** power)
    d = Dev(c)
    check(c, d, heads * group)
    check(c, d, heads * group, sees)
    # the last token alone
    for b in range(3):
        first = c.lens[b] - tokens
        c.v[b][first:-1] = _kv.bf16(rng.normal(0, 1, size=(tokens - 1, heads, D)))
    check(c, Dev(c), heads * group)


@pytest.mark.parametrize("D", [32, 96, 160, 192, 224])
@pytest.mark.parametrize("tokens, kv", [(24, "s8"), (70, "u4")])
def test_channels_that_do_not_fill_the_operands(D, tokens, kv):
    """Many rows of any number of channels, several chunks a block."""
    c = _kv.Cache(np.random.default_rng(D + tokens), [1500, tokens + 1, tokens], [tokens] * 3, 20, D, 16, kv, "f16")
    check(c, Dev(c), 40)


@pytest.mark.parametrize("masked", [False, True])
def test_hidden_tokens_in_a_batch_for_few_rows(masked):
    """Wide heads in more sequences than the kernel for many rows takes: tiles of 16 rows over newest tokens that
    fill several of a warp's tiles, large values among them."""
    rng = np.random.default_rng(17)
    tokens = [0] * 2100
    tokens[40], tokens[900], tokens[2099] = 280, 3, 130
    lens = list(tokens)
    lens[40], lens[900], lens[2099] = 900, 30, 130
    c = _kv.Cache(rng, lens, tokens, 1, 160, 16, "s8", "bf16")
    for b in (40, 900, 2099):
        large = lens[b] - tokens[b] + np.arange(1, tokens[b], 5)
        c.v[b][large] = _kv.bf16(c.v[b][large] * 2.0 ** rng.integers(20, 90, size=(len(large), 1, 1)))
    sees = [_kv.random_tree(rng, n) for n in tokens] if masked else None
    check(c, Dev(c), 2, sees)
