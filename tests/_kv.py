"""Inputs, the definitions in numpy, and derived bounds of the cache of keys and values, for the
CPU and GPU tests."""
from __future__ import annotations

import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def bf16(x):
    """fp32 numbers rounded to bf16, half to even."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().float().numpy()


def codes(x, kv):
    """Codes, zero points and scales of x [..., D] (fp32): the definition, operation by operation."""
    f = np.float32
    x = np.asarray(x, np.float32)
    fin = np.where(np.isfinite(x), x, f(0))
    with np.errstate(all="ignore"):
        if kv == "s8":
            s = np.abs(fin).max(-1, keepdims=True) / f(127)
            q = np.where(s > 0, np.rint(x / np.where(s > 0, s, f(1))), f(0))
            q = np.where(np.isnan(x), f(0), np.clip(q, f(-127), f(127)))
            return q.astype(np.int32), np.zeros(s.shape, np.int32), s
        lo, hi = np.minimum(fin.min(-1, keepdims=True), f(0)), np.maximum(fin.max(-1, keepdims=True), f(0))
        s = bf16(hi / f(15) - lo / f(15))
        d = np.where(s > 0, s, f(1))
        z = np.where(s > 0, np.clip(np.rint(-lo / d), f(0), f(15)), f(0))
        q = np.where((s > 0) & ~np.isnan(x), np.rint(x / d), f(0))
        return np.clip(q + z, f(0), f(15)).astype(np.int32), z.astype(np.int32), s


def values(x, kv):
    """What the cache makes of x: fp32."""
    q, z, s = codes(x, kv)
    return (q - z).astype(np.float32) * s


class Cache:
    """Sequences with their tokens' keys and values in numpy (fp32 numbers of the type x_dt) and
    their pages in any order: entries that no token needs are -1."""

    def __init__(self, rng, lens, tokens, heads, D, page, kv="s8", x_dt="bf16", spare=2, spread=1.0):
        self.lens, self.tokens, self.heads, self.D, self.page, self.kv, self.x_dt = \
            list(lens), list(tokens), heads, D, page, kv, x_dt
        def values_of(n):
            v = rng.normal(0, 1, size=(n, heads, D)) * rng.uniform(0.3, 2.0, size=(1, heads, D))
            v *= np.exp(rng.normal(0, 1, size=(n, heads, 1)) * np.log(spread))
            return torch.from_numpy(v).to(TORCH[x_dt]).float().numpy()
        self.k, self.v = [values_of(n) for n in self.lens], [values_of(n) for n in self.lens]
        need = [-(-n // page) for n in self.lens]
        self.most = max(need + [1])
        free = list(rng.permutation(sum(need) + spare))
        self.num_pages = len(free)
        self.table = np.full((len(self.lens), self.most), -1, np.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = [free.pop() for _ in range(n)]
        self.starts = np.concatenate([[0], np.cumsum(self.tokens)]).astype(np.int32)
        self.rows = int(self.starts[-1])

    def row_places(self):
        """(sequence, position) of each row; positions below 0 have no token."""
        return [(b, n - t + i) for b, (n, t) in enumerate(zip(self.lens, self.tokens)) for i in range(t)]

    def rows_of(self, parts):
        """The newest tokens' rows of k or v, zeros where there is no token."""
        none = np.zeros((self.heads, self.D), np.float32)
        return np.stack([parts[b][p] if p >= 0 else none for b, p in self.row_places()]) if self.rows else \
            np.zeros((0, self.heads, self.D), np.float32)


def random_tree(rng, T):
    """[T, T] booleans: node i sees itself and its ancestors."""
    see = np.zeros((T, T), bool)
    for i in range(T):
        if i:
            see[i] = see[rng.integers(max(0, i - 5), i)]
        see[i, i] = True
    return see


def mask_words(sees, words):
    """The bits of a list of [T, T'] booleans as int32 [rows, words]."""
    out = np.zeros((sum(len(s) for s in sees), words), np.uint32)
    r = 0
    for s in sees:
        for row in s:
            for j in np.flatnonzero(row):
                if j < 32 * words:
                    out[r, j // 32] |= np.uint32(1) << np.uint32(j % 32)
            r += 1
    return out.view(np.int32)


def attention(cache, q, scale, sees=None):
    """out, lse and their bounds in float64; q [rows, heads_q, D], sees: a [T, T'] for each sequence.

    A score's relative or absolute errors reach its weight e^x: each fp32 sum of D products passes
    D / 16 + 16 roundings (a tensor core may cut: 2^-23 of the sum of magnitudes), the factors and
    the subtraction of the maximum four more of the score and maximum (2^-23 each), q as f16
    after its row's scaling 2^-37 of the row's largest; 2^-21 for the exponential and what is
    near it.  A weight, with V's scale in it, is rounded to f16: 2^-11, or 2^-31 of the largest
    where it is small, codes up to 127.  Sums over n tokens pass n / 16 + 64 roundings at most
    (one in 16 tokens' products, the parts' joining), the denominator's as many."""
    rows, HQ, D = q.shape
    G = HQ // cache.heads
    out, lse = np.zeros(q.shape), np.full((rows, HQ), -np.inf)
    tol_out, tol_lse = np.zeros(q.shape), np.zeros((rows, HQ))
    kq = [values(k, cache.kv).astype(np.float64) for k in cache.k]
    vq = [values(v, cache.kv).astype(np.float64) for v in cache.v]
    sv = [codes(v, cache.kv)[2].astype(np.float64) for v in cache.v]
    for r, (b, pos) in enumerate(cache.row_places()):
        n, T = cache.lens[b], cache.tokens[b]
        t = pos - (n - T)
        see = np.arange(n) < n - T
        new = np.arange(max(0, n - T), n)
        if sees is None:
            see[new] = new <= pos
        else:
            j = new - (n - T)
            see[new] = [bool(x < sees[b].shape[1] and sees[b][t, x]) for x in j]
        at = np.flatnonzero(see)
        if len(at) == 0:
            continue
        for h in range(HQ):
            qh, k, v = q[r, h].astype(np.float64), kq[b][at, h // G], vq[b][at, h // G]
            x = scale * (k @ qh)
            mag = abs(scale) * (np.abs(k) @ np.abs(qh))
            m = x.max()
            p = np.exp(x - m)
            total = p.sum()
            delta = (D / 16 + 16) * 2.0 ** -23 * mag + 4 * 2.0 ** -23 * (np.abs(x) + abs(m)) + 2.0 ** -21 + \
                abs(scale) * 2.0 ** -37 * np.abs(qh).max() * np.abs(k).sum(1)
            sums = (len(at) / 16 + 64) * 2.0 ** -23
            wide = (p * delta).sum() / total  # of the denominator, relative
            out[r, h] = p @ v / total
            terms = np.abs(v)
            tol_out[r, h] = (p * (delta + 2.0 ** -11 + sums)) @ terms / total \
                + (wide + sums) * (p @ terms) / total \
                + len(at) * 2.0 ** -31 * 127 * sv[b][at, h // G].max() / total
            lse[r, h] = m + np.log(total)
            tol_lse[r, h] = wide + sums + 2.0 ** -22 * (1 + abs(m) + abs(np.log(total)))
    dt = torch.finfo(TORCH[cache.x_dt])
    tol_out = tol_out + (np.abs(out) + tol_out) * dt.eps / 2 + dt.smallest_normal * dt.eps
    return out, lse, tol_out, tol_lse
