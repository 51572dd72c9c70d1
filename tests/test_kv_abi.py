"""Host-side checks of the cache of keys and values (no GPU needed): sizes, the structs' layouts,
refusals before any launch, and the definitions the GPU tests use."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from integer_quantized_nn_gb300 import qnn
import _kv

pytestmark = pytest.mark.cpu
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qnn.h")
INVALID, UNSUPPORTED, ALIGNMENT = qnn.QNN_ERR_INVALID_ARG, qnn.QNN_ERR_UNSUPPORTED, qnn.QNN_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    return qnn.load()


def geom(**bad):
    return qnn.kv_geom(**{**dict(heads=2, D=64, page=16, kv_dt="s8"), **bad})


def seqs(**bad):
    s = dict(pages=128, num_pages=4, table=4, ld_table=2, lens=4, starts=None, rows=6, batch=3, tokens=2)
    s.update(bad)
    return qnn.KvSeqs(*[s[n] for n, _ in qnn.KvSeqs._fields_])


def split(bad):
    """The keys of a geometry, of the sequences, and the call's own."""
    g = {k: v for k, v in bad.items() if k in ("heads", "D", "page", "kv_dt")}
    fields = [n for n, _ in qnn.KvSeqs._fields_]
    s = {k: v for k, v in bad.items() if k in fields}
    return geom(**g), seqs(**s), {k: v for k, v in bad.items() if k not in g and k not in s}


BAD_GEOM = [dict(heads=0), dict(heads=1025), dict(D=0), dict(D=48), dict(D=288), dict(page=0), dict(page=24),
            dict(page=272), dict(kv_dt="s4"), dict(kv_dt="u8"), dict(kv_dt="f16")]
BAD_SEQS = [dict(pages=None), dict(table=None), dict(lens=None), dict(batch=-1), dict(rows=-1), dict(tokens=-1),
            dict(num_pages=-1), dict(ld_table=-1), dict(num_pages=1 << 31), dict(rows=5), dict(rows=1 << 31),
            dict(ld_table=1 << 31)]
BAD_ALIGNMENT = [dict(pages=64), dict(table=2), dict(lens=6), dict(starts=2)]


def test_page_sizes(lib):
    size = qnn.qnn_kv_page_bytes
    assert size(geom()) == 2 * 16 * (2 * 64 + 8)
    assert size(geom(heads=8, D=128, page=64)) == 8 * 64 * (2 * 128 + 8)
    assert size(geom(heads=3, D=96, page=16, kv_dt="u4")) == 3 * 16 * (2 * 48 + 8)
    for D in range(32, 257, 32):
        for page in range(16, 257, 16):
            for dt in ("s8", "u4"):
                assert size(geom(heads=1, D=D, page=page, kv_dt=dt)) % 128 == 0
    for bad in BAD_GEOM:
        assert size(geom(**bad)) == 0, bad
    assert lib.qnn_kv_page_bytes(None) == 0


@pytest.mark.parametrize("name", ["q_kv_write", "q_kv_read"])
def test_write_and_read_refusals(lib, name):
    def call(**bad):
        g, s, own = split(bad)
        a = {**dict(k=16, v=16, x_dt="bf16", ld_k=0, ld_v=0), **own}
        return getattr(lib, name)(a["k"], a["v"], qnn.DTYPES[a["x_dt"]], a["ld_k"], a["ld_v"], ctypes.byref(g),
                                  ctypes.byref(s), None)
    for bad in BAD_GEOM + BAD_SEQS + [dict(ld_k=127), dict(ld_v=127), dict(ld_k=-1), dict(ld_k=1 << 61),
                                      dict(k=None, v=None)]:
        assert call(**bad) == INVALID, bad
    for bad in [dict(batch=4097, rows=8194), dict(x_dt="s8"), dict(x_dt="s32")]:
        assert call(**bad) == UNSUPPORTED, bad
    for bad in BAD_ALIGNMENT + [dict(k=8), dict(v=24)]:
        assert call(**bad) == ALIGNMENT, bad
    if name == "q_kv_write":
        assert call(k=None) == INVALID and call(v=None) == INVALID
    for nothing in (dict(batch=0, rows=0), dict(tokens=0, rows=0), dict(batch=0, rows=0, lens=None, table=None, pages=None)):
        assert call(k=None, v=None, **nothing) == qnn.QNN_OK, nothing
    f, s = getattr(lib, name), seqs()
    assert f(16, 16, 7, 0, 0, None, ctypes.byref(s), None) == INVALID
    assert f(16, 16, 7, 0, 0, ctypes.byref(geom()), None, None) == INVALID


def test_keep_refusals(lib):
    def call(**bad):
        g, s, own = split(bad)
        a = {**dict(keep=4, ld_keep=2, n_keep=4), **own}
        return lib.q_kv_keep(ctypes.byref(g), ctypes.byref(s), a["keep"], a["ld_keep"], a["n_keep"], None)
    for bad in BAD_GEOM + BAD_SEQS + [dict(keep=None), dict(n_keep=None), dict(ld_keep=-1)]:
        assert call(**bad) == INVALID, bad
    for bad in BAD_ALIGNMENT + [dict(keep=2), dict(n_keep=5)]:
        assert call(**bad) == ALIGNMENT, bad
    assert call(ld_keep=1025) == UNSUPPORTED and call(batch=4097, rows=8194) == UNSUPPORTED
    assert call(batch=0, rows=0) == call(ld_keep=0, keep=None) == call(tokens=0, rows=0) == qnn.QNN_OK


def test_attention_refusals(lib):
    def call(**bad):
        g, s, own = split(bad)
        a = {**dict(q=16, x_dt="bf16", ld_q=0, heads_q=4, scale=0.1, mask=None, mask_words=0, out=16, ld_out=0,
                    lse=None, ws=16), **own}
        if "ws_bytes" not in a:
            a["ws_bytes"] = lib.qnn_kv_attn_workspace_bytes(ctypes.byref(g), ctypes.byref(s), a["heads_q"])
        return lib.q_kv_attn(a["q"], qnn.DTYPES[a["x_dt"]], a["ld_q"], a["heads_q"], ctypes.byref(g), ctypes.byref(s),
                             a["scale"], a["mask"], a["mask_words"], a["out"], a["ld_out"], a["lse"], a["ws"],
                             a["ws_bytes"], None)
    for bad in BAD_GEOM + BAD_SEQS + [dict(q=None), dict(out=None), dict(ws=None), dict(heads_q=0), dict(heads_q=3),
                                      dict(heads_q=-4), dict(heads_q=1 << 30), dict(scale=float("nan")),
                                      dict(scale=float("inf")), dict(mask=4), dict(mask=4, mask_words=-1),
                                      dict(mask_words=-1), dict(ld_q=255), dict(ld_out=8), dict(ld_q=1 << 61),
                                      dict(ws_bytes=0)]:
        assert call(**bad) == INVALID, bad
    for bad in [dict(x_dt="f32"), dict(x_dt="s8"), dict(batch=4097, rows=8194), dict(starts=4, tokens=(1 << 31) - 1),
                dict(starts=4, tokens=1 << 30)]:
        assert call(**bad) == UNSUPPORTED, bad
    for bad in BAD_ALIGNMENT + [dict(q=8), dict(out=18), dict(ws=8), dict(mask=2, mask_words=1), dict(lse=2),
                                dict(ld_q=257), dict(ld_out=260)]:
        assert call(**bad) == ALIGNMENT, bad
    assert call(batch=0, rows=0, q=None, out=None, ws=None) == qnn.QNN_OK
    assert call(tokens=0, rows=0, q=None, out=None, ws=None) == qnn.QNN_OK


def test_scales_that_fit_fp32_but_not_in_units_of_log2(lib):
    """2.4e38 log2(e) is beyond fp32: such a scale would make NaN of a score of zero."""
    def call(scale):
        return lib.q_kv_attn(None, qnn.DTYPES["bf16"], 0, 4, ctypes.byref(geom()), ctypes.byref(seqs(batch=0, rows=0)),
                             scale, None, 0, None, 0, None, None, 0, None)
    for scale in (0.0, 0.1, -0.1, 1e-45, 2.35e38, -2.35e38):
        assert call(scale) == qnn.QNN_OK, scale
    for scale in (2.4e38, -2.4e38, 3.4e38, float("inf"), float("nan")):
        assert call(scale) == INVALID, scale


def test_workspace_sizes(lib):
    size = lambda heads_q=4, **bad: qnn.qnn_kv_attn_workspace_bytes(*split(bad)[:2], heads_q)  # noqa: E731
    assert size() > 0
    for bad in BAD_GEOM + BAD_SEQS + BAD_ALIGNMENT:
        assert size(**bad) == 0, bad
    assert size(heads_q=3) == size(heads_q=0) == size(heads_q=-2) == 0


def test_binding_refuses_tensors_that_would_be_read_as_others(lib):
    """Columns of a wider table, 64-bit integers (torch's default): their entries are not where, or what, the
    library would read, and some may be pages of other sequences."""
    t = pytest.importorskip("torch")
    pages = t.zeros((6, 64), dtype=t.uint8)
    table, lens, starts = (t.zeros(n, dtype=t.int32) for n in ((3, 4), (3,), (4,)))
    s = qnn.kv_seqs(pages, table, lens, 3, 1, starts=starts)
    assert (s.table, s.ld_table, s.batch, s.num_pages) == (table.data_ptr(), 4, 3, 6)
    assert qnn.kv_seqs(pages[2:], table[1:], lens[1:], 2, 1).table == table.data_ptr() + 16
    assert qnn.kv_seqs(pages, table[:1, :2], lens[:1], 1, 1).ld_table == 2  # one row of it is packed

    def refused(what, call, *args, **kwargs):
        with pytest.raises(qnn.QnnError, match=what) as e:
            call(*args, **kwargs)
        assert e.value.status == INVALID
    for name, bad in (("table", table[:, :2]), ("table", table.long()), ("table", t.zeros((4, 3), dtype=t.int32).T),
                      ("table", table.float()), ("table", table.to(t.int16)), ("lens", lens.long()),
                      ("lens", t.zeros(6, dtype=t.int32)[::2]), ("lens", lens[:2]), ("starts", starts.long()),
                      ("starts", t.zeros(8, dtype=t.int32)[::2]), ("starts", starts[:3]), ("pages", pages[:, :32]),
                      ("pages", pages[::2]), ("pages", pages.to(t.int32))):
        a = {**dict(pages=pages, table=table, lens=lens, starts=starts), name: bad}
        refused(name, qnn.kv_seqs, a["pages"], a["table"], a["lens"], 3, 1, starts=a["starts"])
    keep, n_keep = t.zeros((3, 4), dtype=t.int32), t.zeros(3, dtype=t.int32)
    for name, k, n in (("keep", keep[:, :2], n_keep), ("keep", keep.long(), n_keep), ("n_keep", keep, n_keep.long()),
                       ("n_keep", keep, t.zeros(6, dtype=t.int32)[::2]), ("batch", keep[:2], n_keep),
                       ("batch", keep, n_keep[:2])):
        refused(name, qnn.q_kv_keep, geom(), s, k, n, stream=0)
    x = t.zeros(4, dtype=t.bfloat16)
    for bad in (t.zeros((3, 4), dtype=t.int32)[:, :2], t.zeros((3, 4), dtype=t.int64), t.zeros((3, 4))):
        refused("mask", qnn.q_kv_attn, x, "bf16", 4, geom(), s, 0.1, x, x, mask=bad, stream=0)
    refused("lse", qnn.q_kv_attn, x, "bf16", 4, geom(), s, 0.1, x, x, lse=t.zeros((3, 8))[:, :4], stream=0)


@pytest.mark.parametrize("name, struct", [("qnn_kv_geom", qnn.KvGeom), ("qnn_kv_seqs", qnn.KvSeqs)])
def test_structs_match_header(tmp_path, name, struct):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "qnn.h"', "int main(void) {",
             f'    printf("%zu", sizeof({name}));']
    lines += [f'    printf(" %zu", offsetof({name}, {f}));' for f, _ in struct._fields_]
    (tmp_path / "g.c").write_text("\n".join(lines + ["    return 0;", "}"]))
    subprocess.run([cc, "-I", os.path.dirname(HEADER), str(tmp_path / "g.c"), "-o", str(tmp_path / "g")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "g")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f, _ in struct._fields_]


def test_codes_of_worked_numbers():
    """The definitions by hand: s = 2 for 254, ties to even; s = 3 for -15 .. 30, z = 5."""
    q, z, s = _kv.codes(np.float32([254, 1, 3, -5, 127, 0]), "s8")
    assert s[0] == 2 and list(q) == [127, 0, 2, -2, 64, 0] and z[0] == 0
    q, z, s = _kv.codes(np.float32([30, -15, 0, 4.5, 7.5, -1.5, np.nan, np.inf, -np.inf]), "u4")
    assert s[0] == 3 and z[0] == 5 and list(q) == [15, 0, 5, 7, 7, 5, 5, 15, 0]
    q, z, s = _kv.codes(np.float32([np.nan, -np.inf, 4, 127]), "s8")
    assert s[0] == 1 and list(q) == [0, -127, 4, 127]
    for kv in ("s8", "u4"):
        assert not _kv.values(np.float32([0, -0.0, np.nan, np.inf]), kv).any()


def test_attention_reference_by_terms():
    rng = np.random.default_rng(5)
    c = _kv.Cache(rng, [5, 3, 0], [2, 3, 1], 2, 32, 16, "u4")
    q = rng.normal(0, 1, size=(c.rows, 4, 32))
    see = [np.array([[1, 0], [0, 1]], bool), np.zeros((3, 3), bool), np.zeros((1, 1), bool)]
    out, lse, _, _ = _kv.attention(c, q, 0.3, see)
    assert not out[2:].any() and np.isneginf(lse[2:]).all()
    k, v = _kv.values(c.k[0], "u4"), _kv.values(c.v[0], "u4")
    for t, at in ((0, [0, 1, 2, 3]), (1, [0, 1, 2, 4])):
        for h in range(4):
            w = [np.exp(0.3 * sum(float(q[t, h, d]) * float(k[i, h // 2, d]) for d in range(32))) for i in at]
            assert abs(np.log(sum(w)) - lse[t, h]) < 1e-12
            for d in (0, 31):
                assert abs(sum(a * float(v[i, h // 2, d]) for a, i in zip(w, at)) / sum(w) - out[t, h, d]) < 1e-12
    causal = _kv.attention(c, q, 0.3)[1]
    assert np.isfinite(causal[:5]).all() and np.isneginf(causal[5]).all()
