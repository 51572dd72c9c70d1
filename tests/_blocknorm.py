"""The block norm and its gradients in float64, each with a bound on what an fp32 computation
may be off by, for the CPU and GPU tests.

The bounds follow the formulas term by term.  u = 2^-24 is one fp32 rounding; a sum over a
row's C columns passes each term through at most D = 48 of them (32 columns a thread, two
trees of 5, the factors), a sum over rows through rows / 128 + 128 (a block's rows in turn,
then the blocks)."""
from __future__ import annotations

import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U, D = 2.0 ** -24, 48


def make(seed, rows, C, r_dt="f32", y_dt="f32", post="rms", pre="layer", beta=True, gate="none", gate_rows=0, a=1.0,
         b=1.0, mean=0.1, std=1.0, with_y=True, gamma=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, m=0.0, s=1.0):
        return torch.randn(shape, generator=g, dtype=torch.float64) * s + m

    p = dict(rows=rows, C=C, r_dt=r_dt, y_dt=y_dt, post=post, pre=pre, a=a, b=b, eps_post=1e-5, eps_pre=1e-6,
             gate_rows=gate_rows if gate == "rows" else 0)
    p["r"] = normal(rows, C, m=mean, s=2 * std).to(TORCH[r_dt])
    p["y"] = normal(rows, C, m=mean, s=std).to(TORCH[y_dt]) if with_y else None
    for k in ("post", "pre"):
        on = p[k] != "none" and (with_y or k == "pre")
        p["gamma_" + k] = normal(C, m=1.0, s=0.3).float() if on and gamma else None
        p["beta_" + k] = normal(C, s=0.3).float() if on and beta else None
    groups = 1 if gate == "all" else -(-rows // gate_rows) if gate == "rows" else 0
    p["gate"] = normal(groups, C, m=0.5, s=0.5).to(TORCH[y_dt]) if gate != "none" else None
    p["dh"], p["dr_out"] = normal(rows, C).to(TORCH[y_dt]), normal(rows, C).to(TORCH[r_dt])
    return p


def d64(t):
    return None if t is None else t.double()


def gate_of(p):
    """The gate's row for each row, or one."""
    if p["gate"] is None:
        return torch.ones(1, p["C"], dtype=torch.float64)
    gate = p["gate"].double()
    return gate[torch.arange(p["rows"]) // p["gate_rows"]] if p["gate_rows"] else gate


def xhat(x, ex, kind, eps):
    """x^, its bound, rstd and rstd's relative bound, for x known to ex."""
    m = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(len(x), 1, dtype=torch.float64)
    rstd = 1 / ((x - m).square().mean(1, keepdim=True) + eps).sqrt()
    h = (x - m) * rstd
    em = (D * U * x.abs().mean(1, keepdim=True) + ex.mean(1, keepdim=True)) if kind == "layer" else 0.0
    ec = ex + em + U * (x - m).abs()  # of x - m
    # the variance moves by 2 mean((x - m) ec) at first order and its ec^2 at second
    er = (D / 2 + 4) * U + (h.abs() * ec).mean(1, keepdim=True) * rstd + (ec * rstd).square().mean(1, keepdim=True)
    return h, rstd * ec * (1 + er) + (er + 2 * U) * h.abs(), rstd, er


def affine(h, eh, gamma, beta):
    if gamma is not None:
        h, eh = h * gamma.double(), eh * gamma.double().abs()
    if beta is not None:
        h = h + beta.double()
        eh = eh + U * beta.double().abs()
    return h, eh + 2 * U * h.abs()


def forward(p):
    """{name: (value, bound)} of r_out and h, before their rounding to a type."""
    r = p["a"] * p["r"].double()
    er = U * r.abs()
    if p["y"] is not None:
        y, ey = p["y"].double(), torch.zeros(p["rows"], p["C"], dtype=torch.float64)
        if p["post"] != "none":
            h, eh, _, _ = xhat(y, ey, p["post"], p["eps_post"])
            y, ey = affine(h, eh, p["gamma_post"], p["beta_post"])
        k = p["b"] * gate_of(p)
        r, er = r + k * y, er + k.abs() * ey + 2 * U * (k * y).abs()
        er = er + U * r.abs()
    if p["pre"] == "none":
        return {"r_out": (r, er), "h": (r, er)}
    h, eh, _, _ = xhat(r, er, p["pre"], p["eps_pre"])
    return {"r_out": (r, er), "h": affine(h, eh, p["gamma_pre"], p["beta_pre"])}


def dnorm(g, eg, h, eh, rstd, er, kind):
    """rstd (g - mean(g) - x^ mean(g x^)) and its bound."""
    m1, em1 = (g.mean(1, keepdim=True), (D * U * g.abs() + eg).mean(1, keepdim=True)) if kind == "layer" else (0, 0)
    m2 = (g * h).mean(1, keepdim=True)
    em2 = (D * U * (g * h).abs() + eg * h.abs() + g.abs() * eh).mean(1, keepdim=True)
    v = g - m1 - h * m2
    size = g.abs() + abs(m1) + (h * m2).abs()
    e = eg + em1 + eh * m2.abs() + h.abs() * em2 + 3 * U * size
    return rstd * v, rstd * (e + (er + 2 * U) * size)


def backward(p, r_out, use_dh=True, use_dr_out=True):
    """{name: (value, bound)} of the gradients, for r' = r_out as stored."""
    rows, out = p["rows"], {}
    zero = torch.zeros(rows, p["C"], dtype=torch.float64)
    depth = rows / 128 + 128

    def over_rows(v, e):
        return v.sum(0), e.sum(0) + depth * U * v.abs().sum(0)

    G, eG = (p["dr_out"].double(), zero) if use_dr_out else (zero, zero)
    if use_dh:
        dh = p["dh"].double()
        if p["pre"] == "none":
            G, eG = G + dh, eG + U * (G + dh).abs()
        else:
            h, eh, rstd, er = xhat(r_out.double(), zero, p["pre"], p["eps_pre"])
            out["dgamma_pre"] = over_rows(dh * h, dh.abs() * eh + U * (dh * h).abs())
            out["dbeta_pre"] = over_rows(dh, zero)
            g = dh if p["gamma_pre"] is None else dh * p["gamma_pre"].double()
            v, e = dnorm(g, U * g.abs(), h, eh, rstd, er, p["pre"])
            G, eG = G + v, eG + e + U * (G + v).abs()
    out["dr"] = p["a"] * G, abs(p["a"]) * eG + U * (p["a"] * G).abs()
    if p["y"] is None:
        return out
    y, ey, h, eh = p["y"].double(), zero, p["y"].double(), zero
    if p["post"] != "none":
        h, eh, rstd, er = xhat(y, zero, p["post"], p["eps_post"])
        y, ey = affine(h, eh, p["gamma_post"], p["beta_post"])
    v = p["b"] * G * y
    e = abs(p["b"]) * (eG * y.abs() + G.abs() * ey) + 3 * U * v.abs()
    if p["gate"] is not None:
        if p["gate_rows"]:
            at = torch.arange(rows) // p["gate_rows"]
            sums = [torch.zeros(len(p["gate"]), p["C"], dtype=torch.float64).index_add_(0, at, t)
                    for t in (v, e + depth * U * v.abs())]
            out["dgate"] = sums[0], sums[1]
        else:
            out["dgate"] = tuple(t[None] for t in over_rows(v, e))
    k = p["b"] * gate_of(p)
    t = k * G
    et = k.abs() * eG + 2 * U * t.abs()
    out["dgamma_post"] = over_rows(t * h, et * h.abs() + t.abs() * eh + U * (t * h).abs())
    out["dbeta_post"] = over_rows(t, et)
    if p["post"] == "none":
        out["dy"] = t, et
        return out
    g, eg = (t, et) if p["gamma_post"] is None else (t * p["gamma_post"].double(),
                                                     et * p["gamma_post"].double().abs() + 2 * U * t.abs())
    out["dy"] = dnorm(g, eg, h, eh, rstd, er, p["post"])
    return out


def worst(got, want, dt):
    """How much of its bound (and its own rounding to dt) the farthest value uses: <= 1 is right."""
    v, e = want
    eps, tiny = torch.finfo(TORCH[dt]).eps, torch.finfo(TORCH[dt]).smallest_normal * torch.finfo(TORCH[dt]).eps
    room = e + (v.abs() + e) * eps / 2 + tiny
    return float(((got.double().cpu() - v).abs() / room).nan_to_num(nan=float("inf")).max()) if v.numel() else 0.0


def value(p, r, y, gate, params):
    """(r', h) by plain composition, for autograd and differences."""
    def norm(x, kind, eps, gamma, beta):
        if kind == "none":
            return x
        x = x - x.mean(1, keepdim=True) if kind == "layer" else x
        x = x / (x.square().mean(1, keepdim=True) + eps).sqrt()
        x = x if gamma is None else x * gamma
        return x if beta is None else x + beta
    out = p["a"] * r
    if y is not None:
        q = norm(y, p["post"], p["eps_post"], params["gamma_post"], params["beta_post"])
        if gate is not None:
            q = q * (gate[torch.arange(p["rows"]) // p["gate_rows"]] if p["gate_rows"] else gate)
        out = out + p["b"] * q
    return out, norm(out, p["pre"], p["eps_pre"], params["gamma_pre"], params["beta_pre"])
