"""The single-token and block operators, as cases that can be timed and compared.

Three operators: ``qgemv_w4`` (rows of activations times 4-bit weights with group
scales), ``q_block_norm`` (the norms after and before a block with its gate and
residual scale) and ``q_block_norm_backward``.  ``own`` selects the library's calls;
otherwise ``run`` computes the same in elementary torch operations in fp32.

A case of "gemv": M rows, N outputs, K inputs, group size, x/y type, weight codes
("s4", or "u4" with zero points), scale type, bias.  A case of "norm" or
"norm_backward": rows, C, the residual stream's type r, the block's type y, the two
norms, whether they have betas, the gate ("none", "channel": one for all rows,
"sample": one for every `gate_rows` rows, "row": one a row), the residual and block
scales; "norm" also says whether h leaves as s8 codes with a scale per row.
"""
import math

import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def _gemv(name, M, N, K, group, dt, w, scale_dt, bias):
    return {"name": name, "op": "gemv", "M": M, "N": N, "K": K, "group": group, "dt": dt, "w": w,
            "scale_dt": scale_dt, "bias": bias}


def _norm(name, op, rows, C, r, y, post, pre, beta, gate, gate_rows, a, b, s8=False):
    return {"name": name, "op": op, "rows": rows, "C": C, "r": r, "y": y, "post": post, "pre": pre, "beta": beta,
            "gate": gate, "gate_rows": gate_rows, "a": a, "b": b, "s8": s8}


def listed():
    return [
        # the smallest call: the attention output projection of a 1024-wide block, one token; latency counts
        _gemv("gemv 1x1024x1024", 1, 1024, 1024, 64, "bf16", "s4", "bf16", False),
        # one token through a square projection, asymmetric codes
        _gemv("gemv 1x4096x4096 u4", 1, 4096, 4096, 128, "f16", "u4", "f16", True),
        # one token through a large projection: the weight stream alone
        _gemv("gemv 1x8192x8192", 1, 8192, 8192, 128, "bf16", "s4", "f32", False),
        # five rows in fp32, small groups, sizes that fill no tile: ragged K, odd N, rows off 16-byte boundaries
        _gemv("gemv 5x2003x4090 f32", 5, 2003, 4090, 32, "f32", "u4", "f32", True),
        # a batch of sequences decoding together, the wide MLP projection
        _gemv("gemv 32x16384x4096", 32, 16384, 4096, 128, "bf16", "s4", "bf16", True),
        # one decoded token between two linears
        _norm("norm 1x4096", "norm", 1, 4096, "bf16", "bf16", "rms", "rms", False, "channel", 0, 1.0, 1.0),
        # 64 images of 197 tokens, fp32 residual stream, LayerNorms, a gate per image
        _norm("norm 12608x768 gated", "norm", 12608, 768, "f32", "bf16", "layer", "layer", True, "sample", 197,
              1.0, 0.5),
        # a prompt's tokens on their way into an int8 linear: h as codes with a scale per row
        _norm("norm 8192x4096 s8", "norm", 8192, 4096, "bf16", "bf16", "none", "rms", False, "none", 0, 1.0, 1.0,
              True),
        # a width that is no multiple of a vector, a gate per row
        _norm("norm 777x1003 odd", "norm", 777, 1003, "f16", "f16", "layer", "rms", True, "row", 1, 0.7, 0.3),
        # training on 64 images of 197 tokens in fp32, a gate per image
        _norm("backward 12608x1024", "norm_backward", 12608, 1024, "f32", "f32", "layer", "layer", True, "sample",
              197, 1.0, 0.5),
        # training on a long sequence in bf16, gate per channel
        _norm("backward 4096x4096", "norm_backward", 4096, 4096, "bf16", "bf16", "rms", "rms", False, "channel", 0,
              1.0, 1.0),
        # a few odd rows, a gate per row
        _norm("backward 65x1003 odd", "norm_backward", 65, 1003, "f16", "f16", "rms", "layer", True, "row", 1, 0.9,
              0.4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _avoid(n):
    return n + 2 if n == 3072 else n


def draw(rng):
    if rng.random() < 0.4:
        dt = rng.choice(["f16", "bf16", "bf16", "f32"])
        while True:
            N, K = _log_int(rng, 256, 16384), 2 * _log_int(rng, 128, 8192)
            if rng.random() < 0.6:  # mostly whole tiles, as models have them
                N, K = max(64, N // 64 * 64), max(128, K // 128 * 128)
            if N * K <= 8192 * 8192:
                break
        return {"op": "gemv", "M": _log_int(rng, 1, 32), "N": _avoid(N), "K": _avoid(K),
                "group": rng.choice([32, 64, 128, 128, 256]), "dt": dt, "w": rng.choice(["s4", "u4"]),
                "scale_dt": "f32" if dt == "f32" else rng.choice([dt, "f32"]), "bias": rng.random() < 0.5}
    op = rng.choice(["norm", "norm_backward"])
    C = _log_int(rng, 128, 8192)
    if rng.random() < 0.7:
        C = max(128, C // 64 * 64)
    rows = _log_int(rng, 1, 16384)
    y = rng.choice(["bf16", "f16", "f32"])
    r = "f32" if rng.random() < 0.3 else y
    gate = rng.choice(["none", "channel", "sample", "row"])
    c = {"op": op, "rows": rows, "C": _avoid(C), "r": r, "y": y, "post": rng.choice(["none", "rms", "layer"]),
         "pre": rng.choice(["rms", "layer"]), "beta": rng.random() < 0.5, "gate": gate,
         "gate_rows": max(2, _log_int(rng, 2, max(2, rows))) if gate == "sample" else 1 if gate == "row" else 0,
         "a": rng.choice([1.0, 0.8]), "b": rng.choice([1.0, 0.5]),
         "s8": op == "norm" and rng.random() < 0.25}
    most = 12 * 4096 * 4096
    while work(c)["bytes"] > most:
        c["rows"] = c["rows"] * 2 // 3
    if c["gate"] == "sample":
        c["gate_rows"] = max(2, min(c["gate_rows"], c["rows"]))
    return c


def _groups(c):
    return 1 if c["gate"] == "channel" else -(-c["rows"] // c["gate_rows"])


def work(c):
    if c["op"] == "gemv":
        G = -(-c["K"] // c["group"])
        e = _BYTES[c["dt"]]
        return {"bytes": c["N"] * c["K"] / 2 + c["N"] * G * (_BYTES[c["scale_dt"]] + (0.5 if c["w"] == "u4" else 0))
                + c["M"] * (c["K"] + c["N"]) * e + (4 * c["N"] if c["bias"] else 0),
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    n, er, ey = c["rows"] * c["C"], _BYTES[c["r"]], _BYTES[c["y"]]
    gate = 0 if c["gate"] == "none" else _groups(c) * c["C"] * ey
    params = ((c["post"] != "none") + (c["pre"] != "none")) * (1 + c["beta"]) * c["C"] * 4
    if c["op"] == "norm":
        return {"bytes": n * (2 * er + ey + (1 if c["s8"] else ey)) + gate + params + (4 * c["rows"] if c["s8"] else 0),
                "flops": 20 * n}
    # backward: reads r', y, dh, dr'; writes dr, dy
    return {"bytes": n * (3 * er + 3 * ey) + 2 * gate + 2 * params, "flops": 40 * n}


# ---- inputs -------------------------------------------------------------------------


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=g)

    if c["op"] == "gemv":
        N, K, G = c["N"], c["K"], -(-c["K"] // c["group"])
        lo, hi = (-8, 7) if c["w"] == "s4" else (0, 15)
        # rounded normal weights; the packed byte holds element 2i in its low nibble
        q = normal(N, K, std=2.7, mean=0.0 if c["w"] == "s4" else 7.5).round_().clamp_(lo, hi).to(torch.int16) & 15
        s = {"x": normal(c["M"], K).to(_TORCH[c["dt"]]), "W": (q[:, 0::2] | (q[:, 1::2] << 4)).to(torch.uint8),
             "scale": (normal(N, G).abs_() * 0.01 + 0.005).to(_TORCH[c["scale_dt"]]),
             "zero": None, "bias": normal(N) if c["bias"] else None}
        if c["w"] == "u4":
            s["zero"] = torch.randint(5, 11, (N, G), device="cuda", generator=g, dtype=torch.int32)
        return s
    rows, C, tr, ty = c["rows"], c["C"], _TORCH[c["r"]], _TORCH[c["y"]]
    s = {"r": normal(rows, C, std=2.0, mean=0.1).to(tr), "y": normal(rows, C, mean=0.05).to(ty), "gate": None}
    for k in ("post", "pre"):
        has = c[k] != "none"
        s["gamma_" + k] = normal(C, std=0.2, mean=1.0) if has else None
        s["beta_" + k] = normal(C, std=0.2) if has and c["beta"] else None
    if c["gate"] != "none":
        s["gate"] = normal(_groups(c), C, std=0.5, mean=0.5).to(ty)
    if c["op"] == "norm_backward":
        s["dh"], s["dr_out"] = normal(rows, C).to(ty), normal(rows, C).to(tr)
    return s


def prepare(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    s["case"] = c
    if not own:
        return s
    from integer_quantized_nn_gb300 import qnn
    dev = {"device": "cuda"}
    if c["op"] == "gemv":
        geom = qnn.w4_geom(c["N"], c["K"], c["group"], w_dt=c["w"], scale_dt=c["scale_dt"])
        s["geom"] = geom
        s["packed"] = torch.empty(qnn.qnn_gemv_w4_packed_bytes(geom), dtype=torch.uint8, **dev)
        qnn.qgemv_prepack_w4(s["W"], s["scale"], geom, s["packed"], zero_point=s["zero"])
        s["out"] = torch.empty(c["M"], c["N"], dtype=_TORCH[c["dt"]], **dev)
        return s
    s["params"] = qnn.block_norm(
        post=c["post"], pre=c["pre"], eps_post=1e-5, eps_pre=1e-5, gamma_post=s["gamma_post"],
        beta_post=s["beta_post"], gamma_pre=s["gamma_pre"], beta_pre=s["beta_pre"], gate=s["gate"],
        gate_rows=0 if c["gate"] in ("none", "channel") else c["gate_rows"], res_scale=c["a"], block_scale=c["b"])
    if c["op"] == "norm":
        s["r_out"] = torch.empty_like(s["r"])
        s["h"] = torch.empty(s["y"].shape, dtype=torch.int8 if c["s8"] else s["y"].dtype, **dev)
        s["h_scale"] = torch.empty(c["rows"], **dev) if c["s8"] else None
        return s
    s["dr"], s["dy"] = torch.empty_like(s["r"]), torch.empty_like(s["y"])
    s["grads"] = {"d" + k: torch.empty_like(s[k]) for k in
                  ("gate", "gamma_pre", "beta_pre", "gamma_post", "beta_post") if s[k] is not None}
    s["ws"] = torch.empty(qnn.qnn_block_norm_backward_workspace_bytes(c["rows"], c["C"], s["params"]),
                          dtype=torch.uint8, **dev)
    return s


# ---- the plain forms ----------------------------------------------------------------


def _plain_gemv(s):
    c = s["case"]
    N, K, group = c["N"], c["K"], c["group"]
    q = torch.stack((s["W"] & 15, s["W"] >> 4), dim=2).reshape(N, K).to(torch.float32)
    if s["zero"] is None:
        q = torch.where(q > 7, q - 16, q)
    else:
        q = q - s["zero"].to(torch.float32).repeat_interleave(group, dim=1)[:, :K]
    w = q * s["scale"].to(torch.float32).repeat_interleave(group, dim=1)[:, :K]
    y = s["x"].to(torch.float32) @ w.t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _plain_xhat(x, kind, eps=1e-5):
    if kind == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + eps)
    return x * rstd, rstd


def _plain_affine(x, s, which):
    if s["gamma_" + which] is not None:
        x = x * s["gamma_" + which]
    if s["beta_" + which] is not None:
        x = x + s["beta_" + which]
    return x


def _plain_gate(s):
    c = s["case"]
    if s["gate"] is None:
        return torch.ones((), device="cuda")
    gate = s["gate"].to(torch.float32)
    return gate if c["gate"] == "channel" else gate.repeat_interleave(c["gate_rows"], dim=0)[:c["rows"]]


def _plain_norm(s):
    c = s["case"]
    p = s["y"].to(torch.float32)
    if c["post"] != "none":
        p = _plain_affine(_plain_xhat(p, c["post"])[0], s, "post")
    r = c["a"] * s["r"].to(torch.float32) + c["b"] * _plain_gate(s) * p
    h = _plain_affine(_plain_xhat(r, c["pre"])[0], s, "pre")
    r = r.to(s["r"].dtype)
    if not c["s8"]:
        return r, h.to(s["y"].dtype)
    scale = h.abs().amax(dim=1) / 127
    q = (h / scale[:, None]).round().clamp(-128, 127).to(torch.int8)
    return r, _values(q, scale)


def _values(q, scale):
    """What the codes stand for, in fp16."""
    return q * scale.to(torch.float16)[:, None]


def _plain_dnorm(g, xhat, rstd, kind):
    d = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(dim=1, keepdim=True)
    return rstd * d


def _plain_backward(s):
    c, out = s["case"], {}
    dh, y = s["dh"].to(torch.float32), s["y"].to(torch.float32)
    xhat, rstd = _plain_xhat(s["r"].to(torch.float32), c["pre"])
    out["dgamma_pre"] = (dh * xhat).sum(dim=0)
    if c["beta"]:
        out["dbeta_pre"] = dh.sum(dim=0)
    G = s["dr_out"].to(torch.float32) + _plain_dnorm(dh * s["gamma_pre"], xhat, rstd, c["pre"])
    out["dr"] = (c["a"] * G).to(s["r"].dtype)
    t = c["b"] * _plain_gate(s) * G
    p = y
    if c["post"] != "none":
        yhat, ystd = _plain_xhat(y, c["post"])
        p = _plain_affine(yhat, s, "post")
        out["dgamma_post"] = (t * yhat).sum(dim=0)
        if c["beta"]:
            out["dbeta_post"] = t.sum(dim=0)
        out["dy"] = _plain_dnorm(t * s["gamma_post"], yhat, ystd, c["post"]).to(s["y"].dtype)
    else:
        out["dy"] = t.expand_as(y).to(s["y"].dtype)
    if s["gate"] is not None:
        d = c["b"] * G * p
        if c["gate"] == "channel":
            d = d.sum(dim=0, keepdim=True)
        elif c["gate"] == "sample":
            at = torch.arange(c["rows"], device="cuda") // c["gate_rows"]
            d = torch.zeros(_groups(c), c["C"], device="cuda").index_add_(0, at, d)
        out["dgate"] = d.to(s["gate"].dtype)
    return out


def run(s):
    c = s["case"]
    if not own:
        return {"gemv": _plain_gemv, "norm": _plain_norm, "norm_backward": _plain_backward}[c["op"]](s)
    from integer_quantized_nn_gb300 import qnn
    if c["op"] == "gemv":
        qnn.qgemv_w4(s["x"], c["dt"], s["packed"], s["geom"], c["M"], s["out"], c["dt"], bias=s["bias"])
        return s["out"]
    if c["op"] == "norm":
        qnn.q_block_norm(s["r"], c["r"], s["y"], c["y"], c["rows"], c["C"], s["params"], r_out=s["r_out"], h=s["h"],
                         h_dt="s8" if c["s8"] else c["y"], h_scale=s["h_scale"])
        return s["r_out"], _values(s["h"], s["h_scale"]) if c["s8"] else s["h"]
    qnn.q_block_norm_backward(s["r"], c["r"], s["y"], c["y"], c["rows"], c["C"], s["params"], s["dh"], s["dr_out"],
                              s["dr"], s["dy"], s["ws"], **s["grads"])
    return {"dr": s["dr"], "dy": s["dy"], **s["grads"]}


# ---- from the definitions, in 64 bits -----------------------------------------------


def _exact_norm(x, kind, gamma, beta):
    if kind == "none":
        return x
    if kind == "layer":
        y = torch.nn.functional.layer_norm(x, x.shape[-1:], eps=1e-5)
    else:
        y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-5).sqrt()
    y = y if gamma is None else y * gamma
    return y if beta is None else y + beta


def exact(case, seed):
    c = dict(case)
    s = {k: v.double() if v is not None and v.is_floating_point() else v for k, v in _inputs(c, seed).items()}
    if c["op"] == "gemv":
        # one group of columns at a time: sum of x (q - z), then its scale
        codes = torch.empty(c["N"], c["K"], dtype=torch.float64, device="cuda")
        codes[:, 0::2], codes[:, 1::2] = (s["W"] % 16).double(), (s["W"] // 16).double()
        y = torch.zeros(c["M"], c["N"], dtype=torch.float64, device="cuda")
        for i, k in enumerate(range(0, c["K"], c["group"])):
            part = codes[:, k:k + c["group"]]
            part = (part + 8) % 16 - 8 if s["zero"] is None else part - s["zero"][:, i:i + 1]
            y += (s["x"][:, k:k + c["group"]] @ part.t()) * s["scale"][:, i]
        return y if s["bias"] is None else y + s["bias"]
    names = ["r", "y", "gate", "gamma_post", "beta_post", "gamma_pre", "beta_pre"]
    r, y, gate, gq, bq, gp, bp = (s[k] for k in names)
    rows = torch.arange(c["rows"], device="cuda")
    group = rows * 0 if c["gate"] in ("none", "channel") else rows // c["gate_rows"]

    def branch(y, gate, gq, bq):
        p = c["b"] * _exact_norm(y, c["post"], gq, bq)
        return p if gate is None else gate[group] * p

    if c["op"] == "norm":
        r = c["a"] * r + branch(y, gate, gq, bq)
        h = _exact_norm(r, c["pre"], gp, bp)
        if c["s8"]:
            step = h.abs().max(dim=1, keepdim=True).values / 127
            h = torch.clamp(torch.round(h / step), -128, 127) * step
        return r, h
    # the gradients by differentiating the definitions: at r' as given, then through the branch
    with torch.enable_grad():
        leaf = {k: v.requires_grad_() for k, v in zip(names, (r, y, gate, gq, bq, gp, bp)) if v is not None}
        _exact_norm(r, c["pre"], gp, bp).backward(s["dh"])
        G = r.grad + s["dr_out"]
        branch(y, gate, gq, bq).backward(G)
    out = {"d" + k: leaf[k].grad for k in names[2:] if k in leaf}
    return {"dr": c["a"] * G, "dy": y.grad, **out}
