"""The cache of keys and values on the GPU: written, read back and kept against the definitions,
bit for bit, and the attention over it against the 64-bit reference."""
import numpy as np
import pytest

from integer_quantized_nn_gb300 import qnn
from _util import torch
import _kv

pytestmark = pytest.mark.gpu
OK, INVALID = qnn.QNN_OK, qnn.QNN_ERR_INVALID_ARG


class Dev:
    """A Cache's sequences on the device; `fill` writes all their tokens."""

    def __init__(self, c, fill=True, byte=0xFF, even=False):
        t = torch()
        self.c = c
        self.geom = qnn.kv_geom(c.heads, c.D, c.page, kv_dt=c.kv)
        # pages full of NaN words until they are written
        self.pages = t.full((c.num_pages, qnn.qnn_kv_page_bytes(self.geom)), byte, dtype=t.uint8, device="cuda")
        self.table, self.lens = t.from_numpy(c.table).cuda(), self.ints(c.lens)
        self.starts = None if even else t.from_numpy(c.starts).cuda()
        self.seqs = qnn.kv_seqs(self.pages, self.table, self.lens, c.rows, max(c.tokens + [0]), starts=self.starts)
        if fill and sum(c.lens):
            self.all = self.ints(np.concatenate([[0], np.cumsum(c.lens)]))
            whole = qnn.kv_seqs(self.pages, self.table, self.lens, sum(c.lens), max(c.lens), starts=self.all)
            k, v = (self.floats(np.concatenate(x)) for x in (c.k, c.v))
            qnn.q_kv_write(k, v, c.x_dt, self.geom, whole)
            assert qnn.qnn_check_device_error() == OK

    def ints(self, v):
        return torch().tensor(np.asarray(v, np.int32).tolist(), dtype=torch().int32, device="cuda")

    def floats(self, v, dt=None):
        return torch().from_numpy(np.ascontiguousarray(v)).to(_kv.TORCH[dt or self.c.x_dt]).cuda()

    def attend(self, q, scale, mask=None, pad_q=0, pad_out=0, extra=2, lse=True, ws=None):
        """out and lse as numpy; what must stay as it was is checked."""
        t, c = torch(), self.c
        rows, HQ, D = q.shape
        dt = _kv.TORCH[c.x_dt]
        qd = t.full((rows, HQ * D + pad_q), float("nan"), dtype=dt, device="cuda")
        qd[:, :HQ * D] = self.floats(q).view(rows, -1)
        out = t.full((rows + extra, HQ * D + pad_out), 77.0, dtype=dt, device="cuda")
        ls = t.full((rows + extra, HQ), 77.0, device="cuda")
        n = qnn.qnn_kv_attn_workspace_bytes(self.geom, self.seqs, HQ)
        ws = t.full((n,), 0xFF, dtype=t.uint8, device="cuda") if ws is None else ws
        m = None if mask is None else t.from_numpy(mask).cuda()
        qnn.q_kv_attn(qd, c.x_dt, HQ, self.geom, self.seqs, scale, out, ws, mask=m, lse=ls if lse else None,
                      ld_q=HQ * D + pad_q, ld_out=HQ * D + pad_out)
        assert bool((out[rows:] == 77.0).all()) and bool((out[:, HQ * D:] == 77.0).all())
        assert bool((ls[rows:] == 77.0).all())
        return out[:rows, :HQ * D].reshape(rows, HQ, D).double().cpu().numpy(), ls[:rows].double().cpu().numpy()


def near(got, want, tol, what):
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine]), what
    off = np.abs(got[fine] - want[fine]) / tol[fine]
    assert off.size == 0 or off.max() <= 1.0, (what, off.max(), int((off > 1).sum()), off.size)


def check(c, dev, HQ, sees=None, words=0, scale=None, q=None, rng=None, **how):
    """One attention call against the reference."""
    rng = rng or np.random.default_rng(c.D + HQ + sum(c.lens))
    scale = scale or c.D ** -0.5
    if q is None:
        q = rng.normal(0, 1.5, size=(c.rows, HQ, c.D))
    q = dev.floats(q).double().cpu().numpy()
    mask = None if sees is None else _kv.mask_words(sees, words or max(1, -(-max(c.tokens) // 32)))
    out, lse = dev.attend(q, scale, mask, **how)
    assert qnn.qnn_check_device_error() == OK
    w_out, w_lse, t_out, t_lse = _kv.attention(c, q, scale, sees)
    near(out, w_out, t_out, "out")
    if how.get("lse", True):
        near(lse, w_lse, t_lse, "lse")
    return out, lse


# ---- written and read back -------------------------------------------------------------

SHAPES = [(1, 32, 16), (8, 128, 16), (3, 96, 48), (5, 64, 64), (2, 160, 32), (1, 256, 256), (7, 192, 16), (4, 224, 80)]


@pytest.mark.parametrize("kv", ["s8", "u4"])
@pytest.mark.parametrize("x_dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads, D, page", SHAPES)
def test_written_values_come_back(heads, D, page, x_dt, kv):
    """All tokens written at once, then the newest of each sequence read: the definition's values,
    and what belongs to no row as it was."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(D + page), [37, 1, 0, 16, 65], [5, 1, 0, 16, 64], heads, D, page, kv, x_dt)
    d = Dev(c)
    k, v = (t.full((c.rows + 2, heads * D + 8), 77.0, dtype=_kv.TORCH[x_dt], device="cuda") for _ in range(2))
    qnn.q_kv_read(k, v, x_dt, d.geom, d.seqs, ld_k=heads * D + 8, ld_v=heads * D + 8)
    assert qnn.qnn_check_device_error() == OK
    for got, parts in ((k, c.k), (v, c.v)):
        want = d.floats(_kv.values(c.rows_of(parts), kv)).view(c.rows, -1)
        assert t.equal(got[:c.rows, :heads * D], want)
        assert bool((got[c.rows:] == 77.0).all()) and bool((got[:, heads * D:] == 77.0).all())


@pytest.mark.parametrize("x_dt, pad", [("bf16", 1), ("bf16", 4), ("bf16", 8), ("f32", 2), ("f16", 3), ("f32", 4)])
def test_rows_of_any_pitch(x_dt, pad):
    """k and v as columns of wider rows, on and off 16-byte boundaries, two pitches, NaN between."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(3), [20, 33], [20, 33], 3, 96, 16, "s8", x_dt)
    d = Dev(c, fill=False)
    n = 3 * 96
    k, v = (t.full((53, n + p), float("nan"), dtype=_kv.TORCH[x_dt], device="cuda") for p in (pad, 2 * pad))
    k[:, :n], v[:, :n] = (d.floats(np.concatenate(x)).view(53, n) for x in (c.k, c.v))
    qnn.q_kv_write(k, v, x_dt, d.geom, d.seqs, ld_k=n + pad, ld_v=n + 2 * pad)
    a, b = t.full_like(k, 5.0), t.full_like(v, 5.0)
    qnn.q_kv_read(a, b, x_dt, d.geom, d.seqs, ld_k=n + pad, ld_v=n + 2 * pad)
    assert qnn.qnn_check_device_error() == OK
    for got, parts in ((a, c.k), (b, c.v)):
        assert t.equal(got[:, :n], d.floats(_kv.values(np.concatenate(parts), "s8")).view(53, n))
        assert bool((got[:, n:] == 5.0).all())


@pytest.mark.parametrize("kv", ["s8", "u4"])
def test_codes_at_ties_and_extremes(kv):
    """Quotients on and next to ties, subnormal and huge numbers, NaN and infinities in a head."""
    c = _kv.Cache(np.random.default_rng(11), [64], [64], 2, 64, 32, kv, "f32")
    x, rng = c.k[0], np.random.default_rng(12)
    top = np.float32(127 if kv == "s8" else 15)
    for r in range(64):
        s = np.float32(2.0) ** rng.integers(-140, 110)
        ties = (rng.integers(-20, 20, size=(2, 64)) + 0.5).astype(np.float32)
        with np.errstate(all="ignore"):
            x[r] = ties * s
            x[r, :, 0] = top * s
            x[r, :, 1::3] = np.nextafter(x[r, :, 1::3], np.float32(0))
    x[5, 0, 7], x[6, 1, 9], x[7, 0, 3] = np.nan, np.inf, -np.inf
    x[8, :, :] = 0
    x[9, 0, :] = np.nan
    x[10, 1, :] = np.inf
    x[11, 0, :], x[11, 0, 5] = -3e38, 3.4e38
    x[12, 0, :] = 1e-45
    x[13, 0, :] = -7.25
    c.v[0][:] = x[::-1]
    d = Dev(c)
    t = torch()
    k, v = (t.empty((64, 2, 64), device="cuda") for _ in range(2))
    qnn.q_kv_read(k, v, "f32", d.geom, d.seqs)
    want = _kv.values(x, kv)
    # -3e38 .. 3.4e38 in u4: s = 4.27e37, z = 7, and 3.4e38 is code 15: 8 s = 3.42e38 passes fp32's 3.403e38
    beyond = ~np.isfinite(want)
    assert beyond.sum() == (kv == "u4") and (kv == "s8" or want[11, 0, 5] == np.inf)
    assert np.array_equal(k.cpu().numpy(), want) and np.array_equal(v.cpu().numpy(), want[::-1])


def test_only_the_newest_places_are_written():
    """Every byte of the pages that belongs to no newest token stays; k or v alone can be read."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(1), [40, 3, 17], [3, 3, 1], 2, 64, 16, "s8", "bf16")
    d = Dev(c)
    before = d.pages.clone()
    old = {}
    for b, p in c.row_places():
        old.setdefault(int(c.table[b, p // 16]), []).append(p % 16)
    k, v = (d.floats(np.random.default_rng(2).normal(0, 1, size=(c.rows, 2, 64))) for _ in range(2))
    qnn.q_kv_write(k, v, "bf16", d.geom, d.seqs)
    changed = (d.pages != before).view(c.num_pages, 2, 16 * (2 * 64 + 8)).cpu().numpy()
    for page in range(c.num_pages):
        slots = np.zeros(16, bool)
        for head in changed[page]:
            slots |= head[:2048].reshape(2, 16, 64).any((0, 2)) | head[2048:].reshape(2, 16, 4).any((0, 2))
        assert set(np.flatnonzero(slots)) == set(old.get(page, [])), page
    a, b = (t.full((c.rows, 2, 64), 9.0, dtype=t.bfloat16, device="cuda") for _ in range(2))
    qnn.q_kv_read(a, None, "bf16", d.geom, d.seqs)
    qnn.q_kv_read(None, b, "bf16", d.geom, d.seqs)
    assert t.equal(a, d.floats(_kv.values(k.float().cpu().numpy(), "s8")))
    assert t.equal(b, d.floats(_kv.values(v.float().cpu().numpy(), "s8")))


def test_padded_batch():
    """Sequences shorter than their newest tokens: rows without a token write nothing, read and attend as zero."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(4), [0, 2, 9, 0], [4] * 4, 2, 32, 16)
    d = Dev(c, even=True)
    k = d.floats(np.random.default_rng(5).normal(0, 1, size=(16, 2, 32)))
    kept = [x.copy() for x in c.k]
    for r, (b, p) in enumerate(c.row_places()):
        if p >= 0:
            c.k[b][p], c.v[b][p] = k[r].float().cpu().numpy(), -k[r].float().cpu().numpy()
    assert any((a != b).any() for a, b in zip(kept, c.k) if len(a))
    qnn.q_kv_write(k, -k, "bf16", d.geom, d.seqs)
    a, b = t.full_like(k, 3.0), t.full_like(k, 3.0)
    qnn.q_kv_read(a, b, "bf16", d.geom, d.seqs)
    assert t.equal(a, d.floats(_kv.values(c.rows_of(c.k), "s8"))) and t.equal(b, d.floats(_kv.values(c.rows_of(c.v), "s8")))
    out, lse = check(c, d, 4)
    assert not out[:4].any() and not out[12:].any() and np.isneginf(lse[:4]).all()


@pytest.mark.parametrize("batch", [1, 31, 32, 33, 1000, 1056, 4096])
def test_the_sequence_of_every_row(batch):
    """Starts with empty sequences among them, for every size of the search; each token in a page of its own."""
    t = torch()
    rng = np.random.default_rng(batch)
    tokens = rng.integers(0, 3, size=batch)
    tokens[-1] = 1
    starts = np.concatenate([[0], np.cumsum(tokens)])
    n = int(starts[-1])
    g = qnn.kv_geom(1, 32, 16)
    pages = t.zeros((batch, qnn.qnn_kv_page_bytes(g)), dtype=t.uint8, device="cuda")
    ints = lambda v: t.tensor(np.asarray(v).tolist(), dtype=t.int32, device="cuda")  # noqa: E731
    table, lens, st = ints(rng.permutation(batch)[:, None]), ints(tokens), ints(starts)
    s = qnn.kv_seqs(pages, table, lens, n, 2, starts=st)
    k = (1 + t.arange(n, device="cuda", dtype=t.float32))[:, None, None].expand(n, 1, 32).contiguous()
    qnn.q_kv_write(k, 2 * k, "f32", g, s)
    a, b = t.empty_like(k), t.empty_like(k)
    qnn.q_kv_read(a, b, "f32", g, s)
    assert qnn.qnn_check_device_error() == OK
    want = _kv.values(k.cpu().numpy(), "s8")
    assert np.array_equal(a.cpu().numpy(), want) and np.array_equal(b.cpu().numpy(), 2 * want)
    each = t.empty_like(k)
    for seq in rng.choice(np.flatnonzero(tokens), size=min(5, batch)):
        one = qnn.kv_seqs(pages, table[seq:seq + 1], lens[seq:seq + 1].clone(), int(tokens[seq]), int(tokens[seq]))
        one.table = table.data_ptr() + 4 * int(seq)
        qnn.q_kv_read(each, None, "f32", g, one)
        assert t.equal(each[:tokens[seq]], a[starts[seq]:starts[seq + 1]])


# ---- kept ------------------------------------------------------------------------------


@pytest.mark.parametrize("kv, D, page", [("s8", 128, 16), ("u4", 96, 16), ("u4", 128, 48), ("s8", 64, 32), ("s8", 256, 16)])
def test_accepted_tokens_move_up(kv, D, page):
    rng = np.random.default_rng(D)
    tokens = [13, 1, 40, 0, 7, 64, 5]
    c = _kv.Cache(rng, [50, 1, 40, 3, 7, 200, 5], tokens, 3, D, page, kv)
    d = Dev(c)
    n = [4, 1, 40, 0, 0, 17, 5]
    keep = np.full((7, 40), -1, np.int32)
    for b, m in enumerate(n):
        keep[b, :m] = np.sort(rng.permutation(tokens[b])[:m])
    qnn.q_kv_keep(d.geom, d.seqs, torch().from_numpy(keep).cuda(), d.ints(n))
    assert qnn.qnn_check_device_error() == OK
    for b, m in enumerate(n):
        first = c.lens[b] - tokens[b]
        for parts in (c.k, c.v):
            parts[b] = np.concatenate([parts[b][:first], parts[b][first + keep[b, :m]]])
        c.lens[b] = first + m
    c.tokens = list(c.lens)
    c.starts = np.concatenate([[0], np.cumsum(c.tokens)]).astype(np.int32)
    c.rows = int(c.starts[-1])
    t = torch()
    after = qnn.kv_seqs(d.pages, d.table, (lens := d.ints(c.lens)), c.rows, max(c.lens), starts=(st := d.ints(c.starts)))
    assert lens.numel() + 1 == st.numel()
    k, v = (t.empty((c.rows, 3, D), dtype=t.bfloat16, device="cuda") for _ in range(2))
    qnn.q_kv_read(k, v, "bf16", d.geom, after)
    assert t.equal(k, d.floats(_kv.values(np.concatenate(c.k), kv)))
    assert t.equal(v, d.floats(_kv.values(np.concatenate(c.v), kv)))


def test_kept_lists_that_are_refused_on_the_device():
    """Descending, repeated, out of range, too many: reported, that sequence's tokens stay, the others move."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(6), [20] * 7, [8] * 7, 2, 64, 16)
    d = Dev(c)
    before = d.pages.clone()
    keep = [[3, 2, 5], [1, 1, 4], [0, 2, 8], [-1, 0, 2], [1, 2, 3], [1, 2, 3], [2, 4, 7]]
    for n, moves in (([3, 3, 3, 3, 4, -1, 0], False), ([0, 0, 0, 0, 0, 0, 3], True)):
        qnn.q_kv_keep(d.geom, d.seqs, d.ints(keep), d.ints(n))
        assert qnn.qnn_check_device_error() == (OK if moves else INVALID)
        assert t.equal(d.pages, before) != moves
    for b in range(6):  # alone as well
        n = [0] * 7
        n[b] = 4 if b == 4 else -1 if b == 5 else 3
        now = d.pages.clone()
        qnn.q_kv_keep(d.geom, d.seqs, d.ints(keep), d.ints(n))
        assert qnn.qnn_check_device_error() == INVALID
        assert t.equal(d.pages, now)


# ---- attention -------------------------------------------------------------------------

# lens, newest tokens, heads, group, D, page, codes, type
CASES = [
    ([1], [1], 1, 1, 32, 16, "s8", "bf16"),
    ([17], [1], 1, 1, 64, 16, "u4", "f16"),
    ([512], [1], 8, 4, 128, 16, "s8", "bf16"),
    ([300, 1, 64, 129], [1, 1, 1, 1], 2, 8, 128, 32, "u4", "bf16"),
    ([2000, 5], [1, 1], 2, 7, 128, 64, "s8", "f16"),
    ([700], [1], 1, 16, 96, 48, "s8", "bf16"),
    ([333, 90], [1, 1], 3, 5, 160, 16, "u4", "f16"),
    ([513, 31], [1, 1], 2, 12, 256, 16, "s8", "f16"),
    ([257], [1], 1, 33, 64, 256, "s8", "bf16"),
    ([400, 3], [1, 2], 2, 40, 128, 16, "u4", "bf16"),
    ([100, 7, 40, 0], [3, 7, 1, 0], 2, 2, 64, 16, "s8", "bf16"),
    ([640, 200], [9, 30], 2, 4, 128, 64, "u4", "f16"),
    ([130, 128, 127], [130, 128, 127], 1, 2, 128, 16, "s8", "bf16"),
    ([1030], [65], 2, 4, 96, 32, "s8", "f16"),
    ([384, 77], [200, 33], 1, 6, 64, 16, "u4", "bf16"),
    ([260], [70], 1, 3, 256, 16, "u4", "bf16"),
    ([150], [150], 2, 1, 224, 16, "s8", "bf16"),
    ([90] * 40, [2] * 40, 2, 3, 32, 16, "s8", "f16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_attention(case):
    lens, tokens, heads, group, D, page, kv, x_dt = case
    c = _kv.Cache(np.random.default_rng(sum(lens)), lens, tokens, heads, D, page, kv, x_dt)
    check(c, Dev(c), heads * group)


@pytest.mark.parametrize("tokens, heads, group, D, kv, x_dt", [
    ([2, 3], 2, 2, 64, "s8", "bf16"), ([8], 1, 4, 128, "u4", "f16"), ([13, 5, 1], 3, 5, 96, "u4", "f16"),
    ([31, 32, 33], 2, 4, 128, "s8", "bf16"), ([64], 2, 8, 128, "s8", "bf16"), ([64, 20], 1, 2, 256, "u4", "bf16"),
    ([100, 64], 1, 3, 64, "s8", "f16")])
def test_trees(tokens, heads, group, D, kv, x_dt):
    """Random trees behind histories of any length, none among them; bits beyond a sequence's tokens set too."""
    rng = np.random.default_rng(D + sum(tokens))
    lens = [t + h for t, h in zip(tokens, [0, 131, 300])] + [tokens[0] + 500]
    tokens = tokens + [tokens[0]]
    lens = lens[:len(tokens) - 1] + lens[-1:]
    c = _kv.Cache(rng, lens, tokens, heads, D, 16, kv, x_dt)
    sees = [_kv.random_tree(rng, t) for t in tokens]
    words = -(-max(tokens) // 32)
    wide = [np.pad(s, ((0, 0), (0, 32 * words - len(s))), constant_values=True) for s in sees]
    d = Dev(c)
    check(c, d, heads * group, wide, words)
    # rows that see nothing but the history, or nothing at all
    for s in wide:
        s[::2] = False
    check(c, d, heads * group, wide, words)
    # one word only: tokens beyond 32 are not seen
    if words > 1:
        check(c, d, heads * group, [s[:, :32] for s in wide], 1)


def test_a_tree_sees_later_nodes_if_its_bits_say_so():
    c = _kv.Cache(np.random.default_rng(9), [140], [20], 1, 64, 16)
    check(c, Dev(c), 2, [np.ones((20, 20), bool)])


@pytest.mark.parametrize("kv", ["s8", "u4"])
@pytest.mark.parametrize("tokens, group", [(1, 4), (3, 16), (40, 4)])
def test_scales_that_differ_widely(tokens, group, kv):
    """Keys and values whose sizes differ by e^+-8 from token to token; all equal; a scale of zero."""
    rng = np.random.default_rng(21)
    c = _kv.Cache(rng, [700], [tokens], 1, 128, 16, kv, "f16", spread=np.e ** 2)
    c.k[0] = (c.k[0] / np.abs(c.k[0]).max((1, 2), keepdims=True)).astype(np.float16).astype(np.float32)
    c.v[0][5:50:3] = 0
    check(c, Dev(c), group)
    c.k[0][:] = 0
    c.v[0][:] = 1.5
    out, lse = check(c, Dev(c), group)
    # 1.5 is one code times its scale: u4 rounds that to bf16 (2^-9), weights and result are f16 (2^-11 each)
    assert np.abs(out - 1.5).max() <= 1.5 * (2.0 ** -9 + 2.0 ** -10)


@pytest.mark.parametrize("kind", ["large", "small", "rising", "falling", "zero q", "negative"])
@pytest.mark.parametrize("tokens", [1, 24])
def test_scores_of_any_size(kind, tokens):
    """Scores far apart, all alike, and a maximum that moves with every tile."""
    rng = np.random.default_rng(31)
    c = _kv.Cache(rng, [900], [tokens], 1, 64, 16, "s8", "bf16")
    q = rng.normal(0, 1, size=(tokens, 4, 64))
    scale = 0.125
    if kind == "large":
        scale = 30.0
    elif kind == "small":
        q *= 1e-30
    elif kind in ("rising", "falling"):
        ramp = np.linspace(0, 40, 900) if kind == "rising" else np.linspace(40, 0, 900)
        c.k[0] = _kv.bf16((ramp[:, None, None] * np.ones((1, 1, 64)) + rng.normal(0, 0.1, size=(900, 1, 64))) / 8)
        q = np.abs(q)
    elif kind == "zero q":
        q[:, 1:3] = 0
    else:
        scale = -0.3
    check(c, Dev(c), 4, q=q, scale=scale, rng=rng)


def test_values_beyond_the_f16_range():
    """bf16 values and queries of 1e30 and 1e-30: only their ratios matter."""
    rng = np.random.default_rng(41)
    for size_q, size_k, size_v in ((1e30, 1e-30, 1e30), (1e-20, 1e20, 1e-30), (1.0, 1.0, 1e-37)):
        c = _kv.Cache(rng, [333], [3], 1, 64, 16, "s8", "bf16")
        c.k[0], c.v[0] = _kv.bf16(c.k[0] * size_k), _kv.bf16(c.v[0] * size_v)
        check(c, Dev(c), 4, q=rng.normal(0, 1, size=(3, 4, 64)) * size_q)


def test_nan_and_infinity_stay_in_their_rows():
    t = torch()
    rng = np.random.default_rng(51)
    for tokens in (5, 50):
        c = _kv.Cache(rng, [200], [tokens], 2, 64, 16, "s8", "bf16")
        d = Dev(c)
        q = rng.normal(0, 1, size=(tokens, 8, 64))
        clean, _ = check(c, d, 8, q=q)
        q[1, 2, 3], q[3, 5, 0], q[4, 7, 9] = np.nan, np.inf, -np.inf
        out, lse = d.attend(q, 0.125)
        bad = np.zeros((tokens, 8), bool)
        bad[1, 2] = bad[3, 5] = bad[4, 7] = True
        assert np.isnan(out[bad]).all()
        assert np.array_equal(out[~bad], clean[~bad])
    # a key and a value that were not finite are written as finite codes, and poison nothing
    c = _kv.Cache(rng, [60], [1], 1, 64, 16)
    c.k[0][3, 0, 5], c.v[0][7, 0, 1], c.v[0][9, 0, :] = np.nan, np.inf, np.nan
    check(c, Dev(c), 2)
    assert t.cuda.is_available()


@pytest.mark.parametrize("tokens, pad_q, pad_out, lse", [(1, 8, 0, True), (1, 0, 16, False), (6, 128, 8, False),
                                                         (40, 24, 40, True)])
def test_pitches_and_no_lse(tokens, pad_q, pad_out, lse):
    c = _kv.Cache(np.random.default_rng(61), [150, 80], [tokens, tokens], 2, 64, 32)
    check(c, Dev(c, even=True), 6, pad_q=pad_q, pad_out=pad_out, lse=lse)


def test_shared_prefix_pages():
    """Two sequences whose first pages are the same ones."""
    c = _kv.Cache(np.random.default_rng(71), [100, 90], [2, 1], 2, 64, 16)
    c.table[1, :4] = c.table[0, :4]
    c.k[1][:64], c.v[1][:64] = c.k[0][:64], c.v[0][:64]
    check(c, Dev(c), 4)


def test_bad_pages_lengths_and_starts_are_reported():
    """Out-of-range entries: no access, the status, and the other sequences' results."""
    t = torch()
    for tokens in (1, 40):
        c = _kv.Cache(np.random.default_rng(81), [100, 90, 100], [tokens] * 3, 2, 64, 16)
        d = Dev(c)
        q = np.random.default_rng(82).normal(0, 1, size=(c.rows, 4, 64))
        good, _ = d.attend(q, 0.125)
        kv = [t.full((c.rows, 2, 64), 7.0, dtype=t.bfloat16, device="cuda") for _ in range(2)]
        first, last = slice(0, tokens), slice(2 * tokens, 3 * tokens)

        def all_calls():
            out, _ = d.attend(q, 0.125)
            assert qnn.qnn_check_device_error() == INVALID
            qnn.q_kv_read(kv[0], kv[1], "bf16", d.geom, d.seqs)
            assert qnn.qnn_check_device_error() == INVALID
            assert np.array_equal(out[first], good[first]) and np.array_equal(out[last], good[last])
            before = d.pages.clone()
            qnn.q_kv_write(kv[0], kv[1], "bf16", d.geom, d.seqs)  # the values as they are: codes may round once more
            assert qnn.qnn_check_device_error() == INVALID
            d.pages.copy_(before)
            return out[tokens:2 * tokens]

        for bad in (-1, c.num_pages, 2 ** 31 - 1, -2 ** 31):
            d.table[1, 5] = bad  # of 80 .. 89, the newest token among them
            all_calls()
            d.table[1, 5] = int(c.table[1, 5])
        for bad in (-1, 16 * c.most + 1, 2 ** 31 - 1, -2 ** 31):
            d.lens[1] = bad
            assert (all_calls() == 77.0).all()
            d.lens[1] = 90
        for at, bad in ((1, 3 * tokens + 1), (2, 0), (2, -1), (1, -2 ** 31), (3, c.rows + 1)):
            was = int(d.starts[at])
            d.starts[at] = bad
            d.attend(q, 0.125)
            assert qnn.qnn_check_device_error() == INVALID, (at, bad)
            d.starts[at] = was
        # more newest tokens than the call was told
        d.seqs.tokens = tokens - 1
        if tokens > 1:
            out, _ = d.attend(q, 0.125)
            assert qnn.qnn_check_device_error() == INVALID and (out == 77.0).all()
        d.seqs.tokens = tokens
        out, _ = d.attend(q, 0.125)
        assert qnn.qnn_check_device_error() == OK and np.array_equal(out, good)


def test_equal_calls_give_equal_bits_whatever_the_workspace_held():
    t = torch()
    for tokens in (1, 40):
        c = _kv.Cache(np.random.default_rng(91), [3000, 17, 900], [tokens, 1, tokens], 2, 128, 32)
        d = Dev(c)
        q = np.random.default_rng(92).normal(0, 1, size=(c.rows, 8, 128))
        n = qnn.qnn_kv_attn_workspace_bytes(d.geom, d.seqs, 8)
        a = d.attend(q, 0.1)
        for byte in (0, 0x7F, 0xFF):
            b = d.attend(q, 0.1, ws=t.full((n,), byte, dtype=t.uint8, device="cuda"))
            assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_another_stream_and_a_replayed_graph():
    """Lengths that grow between replays of one captured step: write, attend."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(101), [60, 30], [1, 1], 2, 64, 16)
    c.table = np.arange(16, dtype=np.int32).reshape(2, 8)
    c.num_pages = 16
    d = Dev(c, even=True)
    k, v, q = (t.zeros((2, n, 64), dtype=t.bfloat16, device="cuda") for n in (2, 2, 4))
    out = t.empty_like(q)
    ws = t.empty(qnn.qnn_kv_attn_workspace_bytes(d.geom, d.seqs, 4), dtype=t.uint8, device="cuda")

    def step():
        qnn.q_kv_write(k, v, "bf16", d.geom, d.seqs)
        qnn.q_kv_attn(q, "bf16", 4, d.geom, d.seqs, 0.125, out, ws)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    graph = t.cuda.CUDAGraph()
    lens = d.lens.clone()
    with t.cuda.stream(side):
        step()
        side.synchronize()
        with t.cuda.graph(graph, stream=side):
            step()
    d.lens.copy_(lens)
    for b in range(2):  # the step before the capture wrote its zeros in the newest tokens' places
        c.k[b][-1] = c.v[b][-1] = 0
    rng = np.random.default_rng(102)
    for i in range(20):
        new = [rng.normal(0, 1, size=(2, n, 64)) for n in (2, 2, 4)]
        for dst, x in zip((k, v, q), new):
            dst.copy_(d.floats(x))
        d.lens += 1
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for b in range(2):
            c.k[b] = np.concatenate([c.k[b], k[b:b + 1].float().cpu().numpy()])
            c.v[b] = np.concatenate([c.v[b], v[b:b + 1].float().cpu().numpy()])
            c.lens[b] += 1
        qh = q.double().cpu().numpy()
        w_out, _, t_out, _ = _kv.attention(c, qh, 0.125)
        near(out.double().cpu().numpy(), w_out, t_out, i)
    assert qnn.qnn_check_device_error() == OK


def test_places_beyond_32_bits():
    """A cache of more than 4 GiB whose last pages are in use."""
    t = torch()
    c = _kv.Cache(np.random.default_rng(111), [200, 33], [2, 1], 4, 128, 256, "s8", "bf16", spare=0)
    per = 4 * 256 * 264
    pages = (5 << 30) // per
    d = Dev(c, fill=False)
    d.pages = t.empty((pages, per), dtype=t.uint8, device="cuda")
    c.table[:, 0] = [pages - 1, pages - 2]
    c.num_pages = pages
    d.table.copy_(t.from_numpy(c.table))
    d.seqs = qnn.kv_seqs(d.pages, d.table, d.lens, c.rows, 2, starts=d.starts)
    whole_starts = d.ints([0, 200, 233])
    whole = qnn.kv_seqs(d.pages, d.table, d.lens, 233, 200, starts=whole_starts)
    qnn.q_kv_write(d.floats(np.concatenate(c.k)), d.floats(np.concatenate(c.v)), "bf16", d.geom, whole)
    check(c, d, 8)
    k = t.empty((c.rows, 4, 128), dtype=t.bfloat16, device="cuda")
    qnn.q_kv_read(k, None, "bf16", d.geom, d.seqs)
    assert t.equal(k, d.floats(_kv.values(c.rows_of(c.k), "s8")))
