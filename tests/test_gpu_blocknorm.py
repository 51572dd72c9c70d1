"""q_block_norm and q_block_norm_backward on the GPU against the float64 reference and its bounds."""
import pytest
import torch

from integer_quantized_nn_gb300 import qnn
import _blocknorm as bn

pytestmark = pytest.mark.gpu


def padded(t, pad):
    """On the GPU, `pad` NaN between the rows; the tensor and the view of its rows."""
    if t is None:
        return None
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf


def blank(rows, C, pad, dt):
    return torch.full((rows, C + pad), 33.0, dtype=dt, device="cuda")


def untouched(buf, C):
    assert bool((buf[:, C:] == 33).all())
    return buf[:, :C]


def block_norm(p, pads=(0, 0, 0)):
    keep = {k: p[k].cuda() if p[k] is not None else None for k in ("gamma_post", "beta_post", "gamma_pre", "beta_pre",
                                                                   "gate")}
    ld = [p["C"] + x if x else 0 for x in pads]
    q = qnn.block_norm(post=p["post"], pre=p["pre"], eps_post=p["eps_post"], eps_pre=p["eps_pre"], res_scale=p["a"],
                       block_scale=p["b"], gate_rows=p["gate_rows"], ld_r=ld[0], ld_y=ld[1], ld_h=ld[2], **keep)
    q.keep = keep
    return q


def run_forward(p, pads=(0, 0, 0), s8=False, in_place=False, want_r=True, want_h=True):
    rows, C, q = p["rows"], p["C"], block_norm(p, pads)
    r, y = padded(p["r"], pads[0]), padded(p["y"], pads[1])
    r_out = (r if in_place else blank(rows, C, pads[0], r.dtype)) if want_r else None
    h = blank(rows, C, pads[2], torch.int8 if s8 else bn.TORCH[p["y_dt"]]) if want_h else None
    scale = torch.empty(rows, device="cuda") if s8 else None
    qnn.q_block_norm(r, p["r_dt"], y, p["y_dt"], rows, C, q, r_out=r_out, h=h, h_dt="s8" if s8 else None,
                     h_scale=scale)
    assert qnn.qnn_check_device_error() == qnn.QNN_OK
    if want_r:
        r_out = r_out[:, :C] if in_place else untouched(r_out, C)
    return r_out, untouched(h, C) if want_h else None, scale


def check_forward(p, r_out, h):
    want = bn.forward(p)
    if r_out is not None:
        assert bn.worst(r_out, want["r_out"], p["r_dt"]) <= 1
    if h is not None:
        assert bn.worst(h, want["h"], p["y_dt"]) <= 1


def check_codes(p, h, scale):
    v, e = bn.forward(p)["h"]
    top, off = v.abs().max(1).values, e.max(1).values
    s = scale.double().cpu()
    assert bool(((s - top / 127).abs() <= off / 127 + 2 * bn.U * top).all())
    # half a step of the scale that was written, and what h may be off; codes reach 127
    assert bool(((h.double().cpu() * s[:, None] - v).abs() <= (0.5 + 127 * 2 * bn.U) * s[:, None] + e).all())
    assert bool((h.abs().max(1).values.cpu()[top > 0] == 127).all())


PAIRS = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "f16"), ("f32", "bf16")]

# rows, C, and what else
SHAPES = [
    (1, 1, {}), (3, 2, dict(gate="all")), (5, 7, dict(gate="rows", gate_rows=2)), (4, 8, dict(gate="rows", gate_rows=1)),
    (17, 32, dict(gate="rows", gate_rows=5)), (9, 100, dict(gate="all")), (6, 255, {}), (33, 256, dict(gate="all")),
    (2, 264, dict(gate="rows", gate_rows=1)), (10, 512, {}), (40, 768, dict(gate="rows", gate_rows=13)),
    (7, 1003, dict(gate="rows", gate_rows=1)), (12, 1024, dict(gate="all")), (3, 1032, {}),
    (5, 1500, dict(gate="rows", gate_rows=3)), (3, 2048, dict(gate="all")), (2, 4096, {}),
    (2, 5001, dict(gate="rows", gate_rows=1)), (2, 8192, dict(gate="all")), (2, 8200, {}), (2, 9001, dict(gate="all")),
    (1, 16384, {}), (1, 32768, dict(gate="all")),
]
NORMS = [("rms", "rms"), ("layer", "layer"), ("none", "rms"), ("layer", "none"), ("rms", "layer")]


def cases():
    for i, (rows, C, more) in enumerate(SHAPES):
        for j in range(2):  # two of the type pairs and norm pairs for each shape, all met over the shapes
            r_dt, y_dt = PAIRS[(i + 2 * j) % 5]
            post, pre = NORMS[(i // 2 + 3 * j) % 5]
            yield dict(rows=rows, C=C, r_dt=r_dt, y_dt=y_dt, post=post, pre=pre, beta=(i + j) % 2 == 0,
                       a=1.0 if i % 3 else 0.75, b=1.0 if i % 4 else 0.3, **more)


def name(c):
    return "-".join(str(v) for v in c.values())


@pytest.mark.parametrize("case", list(cases()), ids=name)
def test_forward(case):
    p = bn.make(5, **case)
    r_out, h, _ = run_forward(p)
    check_forward(p, r_out, h)


@pytest.mark.parametrize("case", list(cases())[::3], ids=name)
def test_codes(case):
    p = bn.make(6, **case)
    r_out, h, scale = run_forward(p, s8=True)
    check_forward(p, r_out, None)
    check_codes(p, h, scale)


# enough rows for rings of rows in shared memory: one and several rows to a ring, a ring's
# end inside the rows, widths up to its limit and beyond
MANY = [
    (20000, 136, dict(gate="rows", gate_rows=1)), (9001, 512, dict(gate="rows", gate_rows=700)),
    (4000, 768, dict(gate="all")), (3100, 1000, dict(gate="rows", gate_rows=1)), (1500, 2040, {}),
    (650, 4096, dict(gate="rows", gate_rows=1)), (500, 5128, dict(gate="all")), (400, 8192, dict(gate="rows", gate_rows=1)),
    (9000, 333, dict(gate="rows", gate_rows=40)), (1700, 1601, {}), (700, 5001, dict(gate="all")),
]


@pytest.mark.parametrize("i", range(len(MANY)))
def test_many_rows(i):
    rows, C, more = MANY[i]
    for j in range(2):
        r_dt, y_dt = PAIRS[(2 * i + j) % 5]
        post, pre = NORMS[(i + 2 * j) % 5]
        p = bn.make(21, rows, C, r_dt, y_dt, post, pre, beta=j == 0, a=0.9, b=0.6, **more)
        r_out, h, _ = run_forward(p)
        check_forward(p, r_out, h)
        check_codes(p, *run_forward(p, s8=True)[1:])
        check_backward(p, stored(p), run_backward(p, stored(p)))


@pytest.mark.parametrize("rows,C", [(20000, 136), (5000, 768), (1500, 2048), (400, 8192)])
def test_many_rows_with_parts_left_out(rows, C):
    """No h, no r', in place, no block, no norm before: each leaves out a barrier or an array."""
    p = bn.make(22, rows, C, "f32", "bf16", gate="all", beta=False)
    check_forward(p, *run_forward(p, want_h=False)[:2])
    check_forward(p, *run_forward(p, want_r=False)[:2])
    check_forward(p, *run_forward(p, in_place=True)[:2])
    for post, pre, with_y in (("layer", "none", True), ("none", "none", True), ("none", "rms", False)):
        p = bn.make(23, rows, C, "bf16", "bf16", post, pre, gate="all" if with_y else "none", with_y=with_y)
        r_out, h, _ = run_forward(p)
        check_forward(p, r_out, h)
        check_forward(p, *run_forward(p, want_h=False)[:2])
        check_backward(p, stored(p), run_backward(p, stored(p)))
        check_backward(p, stored(p), run_backward(p, stored(p), in_place=True))
    check_backward(p, stored(p), run_backward(p, stored(p), use_dr_out=False), use_dr_out=False)


@pytest.mark.parametrize("pads", [(1, 0, 0), (0, 3, 0), (8, 16, 24), (0, 0, 5), (4, 4, 4)])
@pytest.mark.parametrize("types", PAIRS)
def test_pitches(types, pads):
    p = bn.make(7, 11, 320, *types, gate="rows", gate_rows=4)
    check_forward(p, *run_forward(p, pads)[:2])
    _, h, scale = run_forward(p, pads, s8=True)
    check_codes(p, h, scale)


@pytest.mark.parametrize("C", [96, 101, 2048])
def test_outputs_left_out_and_in_place(C):
    p = bn.make(8, 9, C, "f32", "bf16", gate="all")
    r_out, h, _ = run_forward(p, in_place=True)
    check_forward(p, r_out, h)
    check_forward(p, *run_forward(p, want_h=False)[:2])
    check_forward(p, *run_forward(p, want_r=False)[:2])
    first = bn.make(9, 9, C, "f32", "bf16", post="none", pre="rms", with_y=False, a=0.5)
    check_forward(first, *run_forward(first)[:2])


@pytest.mark.parametrize("types", PAIRS)
def test_a_large_mean_keeps_its_variance(types):
    """Centred sums: mean 60, deviation 0.5 (the bound scales with the mean, not with its square)."""
    p = bn.make(10, 6, 1200, *types, post="layer", pre="layer", mean=60.0, std=0.5, b=0.0)
    check_forward(p, *run_forward(p)[:2])


def test_zero_rows_and_rows_of_nan():
    p = bn.make(11, 8, 300, post="layer", pre="rms", gate="all", beta=False)
    p["r"][2], p["y"][2] = 0, 0
    p["y"][5, 17] = float("nan")
    p["r"][6, 3] = float("inf")
    r_out, h, _ = run_forward(p)
    assert bool((r_out[2] == 0).all()) and bool((h[2] == 0).all())
    assert bool(r_out[5].isnan().all()) and bool(h[5].isnan().all())
    assert bool(r_out[6, 3] == float("inf")) and bool(h[6, 3].isnan()) and bool((h[6, 4:] == 0).all())
    fine = [0, 1, 3, 4, 7]
    want = bn.forward(p)
    for got, k in ((r_out, "r_out"), (h, "h")):
        assert bn.worst(got[fine], tuple(t[fine] for t in want[k]), "f32") <= 1
    codes, scale = run_forward(p, s8=True)[1:]
    assert bool((codes[2] == 0).all()) and float(scale[2]) == 0


def test_no_rows():
    p = bn.make(12, 0, 64, gate="all")
    assert run_forward(p)[1].shape == (0, 64)
    got = run_backward(p, p["r"])
    for k in ("dgate", "dgamma_pre", "dbeta_pre", "dgamma_post", "dbeta_post"):
        assert bool((got[k] == 0).all()) and got[k].numel() == 64, k


# ---- backward ------------------------------------------------------------------------

GRADS = ("gate", "gamma_pre", "beta_pre", "gamma_post", "beta_post")


def run_backward(p, r_out, pads=(0, 0, 0), use_dh=True, use_dr_out=True, in_place=False, leave=()):
    rows, C, q = p["rows"], p["C"], block_norm(p, pads)
    tr, ty = bn.TORCH[p["r_dt"]], bn.TORCH[p["y_dt"]]
    r, y, dh = padded(r_out.to(tr), pads[0]), padded(p["y"], pads[1]), padded(p["dh"], pads[2])
    dr_out = padded(p["dr_out"], pads[0])
    dr = dr_out if in_place else blank(rows, C, pads[0], tr)
    dy = blank(rows, C, pads[1], ty) if y is not None else None
    grads = {"d" + k: torch.full_like(q.keep[k], 55.0) for k in GRADS if q.keep[k] is not None and k not in leave
             and (use_dh or not k.endswith("_pre"))}
    bytes_ = qnn.qnn_block_norm_backward_workspace_bytes(rows, C, q)
    ws = torch.full((bytes_ + 64,), 0xa5, dtype=torch.uint8, device="cuda")
    qnn.q_block_norm_backward(r, p["r_dt"], y, p["y_dt"], rows, C, q, dh if use_dh else None,
                              dr_out if use_dr_out else None, dr, dy, ws[:bytes_], **grads)
    assert qnn.qnn_check_device_error() == qnn.QNN_OK
    assert bool((ws[bytes_:] == 0xa5).all())
    out = {"dr": dr[:, :C] if in_place else untouched(dr, C), **grads}
    if dy is not None:
        out["dy"] = untouched(dy, C)
    return out


def check_backward(p, r_out, got, **k):
    want = bn.backward(p, r_out, **k)
    for n, t in got.items():
        dt = p["r_dt"] if n == "dr" else p["y_dt"] if n in ("dy", "dgate") else "f32"
        assert bn.worst(t, want[n], dt) <= 1, n


def stored(p):
    return bn.forward(p)["r_out"][0].to(bn.TORCH[p["r_dt"]])


@pytest.mark.parametrize("case", list(cases()), ids=name)
def test_backward(case):
    p = bn.make(13, **case)
    r_out = stored(p)
    check_backward(p, r_out, run_backward(p, r_out))


@pytest.mark.parametrize("gate,gate_rows", [("none", 0), ("all", 0), ("rows", 1), ("rows", 2), ("rows", 7),
                                            ("rows", 50), ("rows", 197), ("rows", 1300), ("rows", 5000)])
@pytest.mark.parametrize("C", [64, 75])
def test_sums_over_many_rows(C, gate, gate_rows):
    """Groups inside a block's rows, across two of them, and across many."""
    p = bn.make(14, 3001, C, "f32", "f32", post="layer", gate=gate, gate_rows=gate_rows)
    r_out = stored(p)
    check_backward(p, r_out, run_backward(p, r_out))


@pytest.mark.parametrize("pads", [(1, 0, 0), (0, 3, 0), (8, 16, 24), (0, 0, 5)])
@pytest.mark.parametrize("types", PAIRS)
def test_backward_pitches(types, pads):
    p = bn.make(15, 21, 320, *types, gate="rows", gate_rows=4)
    r_out = stored(p)
    check_backward(p, r_out, run_backward(p, r_out, pads))


@pytest.mark.parametrize("C", [96, 101, 2048])
def test_gradients_absent_left_out_and_in_place(C):
    p = bn.make(16, 30, C, "f32", "bf16", gate="all")
    r_out = stored(p)
    check_backward(p, r_out, run_backward(p, r_out, use_dh=False), use_dh=False)
    check_backward(p, r_out, run_backward(p, r_out, use_dr_out=False), use_dr_out=False)
    check_backward(p, r_out, run_backward(p, r_out, in_place=True))
    check_backward(p, r_out, run_backward(p, r_out, leave=("gate", "gamma_pre", "beta_post")))
    first = bn.make(17, 30, C, "f32", "bf16", post="none", pre="rms", with_y=False, a=0.5)
    check_backward(first, stored(first), run_backward(first, stored(first)))


def test_equal_calls_give_equal_bits():
    p = bn.make(18, 2000, 520, "bf16", "bf16", gate="rows", gate_rows=333)
    r_out = stored(p)
    first = run_backward(p, r_out)
    for _ in range(3):
        again = run_backward(p, r_out)
        assert all(torch.equal(first[k], again[k]) for k in first)


def test_side_stream_and_graph():
    p = bn.make(19, 50, 768, "bf16", "bf16", gate="all")
    rows, C, q = 50, 768, block_norm(p)
    r, y, dh, dr_out = (p[k].cuda() for k in ("r", "y", "dh", "dr_out"))
    out = {k: torch.zeros_like(r) for k in ("r_out", "h", "dr", "dy")}
    grads = {"d" + k: torch.zeros_like(q.keep[k]) for k in GRADS}
    ws = torch.empty(qnn.qnn_block_norm_backward_workspace_bytes(rows, C, q), dtype=torch.uint8, device="cuda")

    def both():
        qnn.q_block_norm(r, "bf16", y, "bf16", rows, C, q, r_out=out["r_out"], h=out["h"])
        qnn.q_block_norm_backward(out["r_out"], "bf16", y, "bf16", rows, C, q, dh, dr_out, out["dr"], out["dy"], ws,
                                  **grads)

    def check():
        torch.cuda.synchronize()
        check_forward(p, out["r_out"], out["h"])
        check_backward(p, out["r_out"].cpu(), {"dr": out["dr"], "dy": out["dy"], **grads})

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    other = bn.make(20, 50, 768, "bf16", "bf16", gate="all")
    for k, t in (("r", r), ("y", y), ("dh", dh), ("dr_out", dr_out)):
        p[k] = other[k]
        t.copy_(other[k])
    graph.replay()
    check()
