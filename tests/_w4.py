"""Inputs and the 64-bit reference of the 4-bit weight products, for the CPU and GPU tests."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(rng, M, N, K, group, x_dt, w_dt, scale_dt, bias):
    """Seeded codes, scales, zero points and activations, on the host (torch tensors)."""
    G = -(-K // group)
    lo, hi = (-8, 8) if w_dt == "s4" else (0, 16)
    q = rng.integers(lo, hi, size=(N, K))
    p = {"q": q, "group": group, "w_dt": w_dt,
         "W": torch.from_numpy(((q[:, 0::2] & 15) | ((q[:, 1::2] & 15) << 4)).astype(np.uint8)),
         "scale": torch.from_numpy(rng.uniform(0.5, 2.0, size=(N, G)) * 0.02).to(TORCH[scale_dt]),
         "zero": torch.from_numpy(rng.integers(0, 16, size=(N, G)).astype(np.int32)) if w_dt == "u4" else None,
         "x": torch.from_numpy(rng.normal(0, 1, size=(M, K))).to(TORCH[x_dt]),
         "bias": torch.from_numpy(rng.normal(0, 1, size=N).astype(np.float32)) if bias else None}
    return p


def weights(p):
    """(q - z) * s in float64, [N, K]."""
    K = p["q"].shape[1]
    s = np.repeat(p["scale"].double().numpy(), p["group"], axis=1)[:, :K]
    z = 0 if p["zero"] is None else np.repeat(p["zero"].numpy(), p["group"], axis=1)[:, :K]
    return (p["q"] - z) * s


def reference(p):
    """y and the sum of the terms' magnitudes, in float64."""
    x, w = p["x"].double().numpy(), weights(p)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if p["bias"] is not None:
        y, mag = y + p["bias"].double().numpy(), mag + np.abs(p["bias"].double().numpy())
    return y, mag


def tolerance(y, mag, K, group, y_dt):
    """A product passes, in the worst order, through one rounding for each step of 16 of K,
    one for each group, and 32 more (the sum inside a step, the split of K, the three parts of
    an fp32 row, the bias); a tensor-core sum may cut instead of round, so each is up to 2^-23
    of a partial sum, which the sum of magnitudes bounds.  Then the result's own rounding."""
    err = (K / 16 + K / group + 32) * 2.0 ** -23 * mag
    dt = TORCH[y_dt]
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    return err + (np.abs(y) + err) * torch.finfo(dt).eps / 2 + tiny
