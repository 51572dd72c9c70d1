"""The operators of a quantised cache of keys and values, as cases that can be timed and compared.

Four operators: ``q_kv_write`` (quantises the newest tokens' keys and values into the pages of a
cache), ``q_kv_read`` (the values back), ``q_kv_attn`` (attention over the cache for the newest
tokens of every sequence: one token, a tree of drafted ones, a chunk of a prompt) and ``q_kv_keep``
(the accepted tokens of a tree move up in the cache).  ``own`` selects the library's calls;
otherwise ``run`` computes the same in elementary torch operations in fp32.

A case: batch sequences of up to `len` tokens, the newest `T` of which the call is about
("ragged": both differ from sequence to sequence), heads of keys and values and D channels each,
`page` tokens a page, codes `kv` ("s8", "u4"), the type `dt` of what is not in the cache.  "attn"
also has the heads of q and the mask: "tree" (each drafted token sees its ancestors) or "causal".
"fused": q, k and v are columns of one tensor, as a fused projection leaves them.  What "write" and
"keep" leave in the cache is read back as part of the pass.
"""
import math
import random

import torch

own = False

_TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def _case(name, op, batch, length, T, heads, D, page, kv, dt, ragged=False, fused=False, heads_q=0, mask="causal"):
    return {"name": name, "op": op, "batch": batch, "len": length, "T": T, "heads": heads, "D": D, "page": page,
            "kv": kv, "dt": dt, "ragged": ragged, "fused": fused, "heads_q": heads_q, "mask": mask}


def listed():
    return [
        # the smallest call: one decoded token of one sequence goes into the cache; latency counts
        _case("write 1 token s8", "write", 1, 300, 1, 8, 128, 16, "s8", "bf16", fused=True),
        # four prompts of different lengths enter the cache in 4 bits, from a fused projection
        _case("write prompts u4", "write", 4, 4000, 4000, 8, 128, 64, "u4", "bf16", ragged=True, fused=True),
        # the cached prefixes of eight sequences come back for a layer that recomputes them
        _case("read 8x4096 s8", "read", 8, 4096, 4096, 8, 128, 64, "s8", "bf16"),
        # odd lengths, an odd number of narrower heads, fp32 out
        _case("read odd u4 f32", "read", 3, 1357, 1357, 5, 96, 16, "u4", "f32", ragged=True),
        # one token of one short sequence; latency counts
        _case("attn 1x512 s8", "attn", 1, 512, 1, 8, 128, 16, "s8", "bf16", heads_q=32),
        # a batch of sequences of different lengths decoding together: the stream of the cache
        _case("attn 64x8192 s8 ragged", "attn", 64, 8192, 1, 8, 128, 64, "s8", "bf16", ragged=True, heads_q=64),
        # one token over one long document in 4 bits: few rows, a long axis
        _case("attn 1x131072 u4", "attn", 1, 131072, 1, 8, 128, 32, "u4", "f16", heads_q=32),
        # trees of 64 drafted tokens being verified
        _case("attn tree 8x64 8192 s8", "attn", 8, 8192, 64, 8, 128, 64, "s8", "bf16", heads_q=32, mask="tree"),
        # small trees of different sizes, odd lengths, five query heads to one of the cache, fused q
        _case("attn tree odd u4", "attn", 5, 1777, 13, 3, 96, 16, "u4", "f16", ragged=True, fused=True, heads_q=15,
              mask="tree"),
        # a chunk of a long prompt attends to what is cached of it and to itself
        _case("attn prompt 2048 of 8192", "attn", 1, 8192, 2048, 8, 128, 64, "s8", "bf16", heads_q=32),
        # the drafted trees of a batch enter the cache, and the accepted paths are kept
        _case("keep 32x64 s8", "keep", 32, 4096, 64, 8, 128, 64, "s8", "bf16"),
        # the same for odd trees in 4 bits
        _case("keep odd u4", "keep", 5, 777, 13, 3, 96, 16, "u4", "f16", ragged=True, fused=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "write", "read", "keep"])
    c = {"op": op, "batch": _log_int(rng, 1, 64), "len": _log_int(rng, 1, 131072), "T": 1,
         "heads": rng.choice([1, 2, 3, 4, 8, 8]), "D": rng.choice([64, 96, 128, 128, 128, 256]),
         "page": rng.choice([16, 32, 64, 128]), "kv": rng.choice(["s8", "s8", "u4"]),
         "dt": rng.choice(["bf16", "bf16", "f16"]), "ragged": rng.random() < 0.5, "fused": rng.random() < 0.3,
         "heads_q": 0, "mask": "causal"}
    if op == "attn":
        c["heads_q"] = c["heads"] * rng.choice([1, 2, 4, 4, 5, 7, 8])
        kind = rng.choice(["token", "token", "tree", "tree", "prompt"])
        if kind != "token":
            c["T"] = _log_int(rng, 2, 64 if kind == "tree" else 2048)
            c["mask"] = "tree" if kind == "tree" else "causal"
    elif op == "keep":
        c["T"] = _log_int(rng, 2, 64)
    elif op == "read" or rng.random() < 0.5:
        c["T"] = c["len"]
        if rng.random() < 0.3:
            c["dt"] = "f32"
    c["len"] = max(c["len"], c["T"])
    most = {"attn": _size(listed()[5]), "write": 1 << 24, "keep": 1 << 24, "read": 1 << 25}[op]
    while _size(c) > most or work(c)["flops"] > 2.4e11:
        c["batch"] = max(1, c["batch"] // 2)
        if c["batch"] == 1:
            c["len"] = max(1, c["len"] * 3 // 5)
            c["T"] = min(c["T"], c["len"])
    return c


def _size(c):
    """Elements that a pass goes over: of the padded cache and the scores, or of the tokens."""
    if c["op"] == "attn":
        return max(c["batch"] * c["len"] * c["heads"] * c["D"], c["batch"] * c["heads_q"] * c["T"] * c["len"] // 2)
    return c["batch"] * c["T"] * c["heads"] * c["D"]


def _tokens(c):
    """The newest tokens of each sequence."""
    if not c["ragged"]:
        return [c["T"]] * c["batch"]
    return [1 + (c["T"] - 1) * ((3 * b + 3) % 4 + 1) // 4 for b in range(c["batch"])]


def _lens(c):
    """The tokens of each sequence, the newest among them."""
    if not c["ragged"]:
        return [c["len"]] * c["batch"]
    return [max(t, c["len"] * ((5 * b + 7) % 8 + 1) // 8) for b, t in enumerate(_tokens(c))]


def _kept(c):
    """How many of them are accepted."""
    return [min(t, 1 + (5 * b + 3) % 7) for b, t in enumerate(_tokens(c))]


def work(c):
    new, lens, e = _tokens(c), _lens(c), _BYTES[c["dt"]]
    rows, token = sum(new), 2 * c["heads"] * (c["D"] * (1 if c["kv"] == "s8" else 0.5) + 4)
    values = 2 * c["heads"] * c["D"] * e
    if c["op"] == "write":  # k and v in, codes out and in again, values out
        return {"bytes": rows * 2 * (values + token), "flops": rows * 2 * c["heads"] * c["D"] * 6}
    if c["op"] == "read":
        return {"bytes": rows * (values + token), "flops": rows * 2 * c["heads"] * c["D"] * 2}
    if c["op"] == "keep":
        n = sum(_kept(c))
        return {"bytes": rows * (values + token) + n * (3 * token + values), "flops": rows * 2 * c["heads"] * c["D"] * 5}
    seen = sum(t * (n - t) + (t if c["mask"] == "tree" else t * (t + 1) // 2) for t, n in zip(new, lens))
    return {"bytes": sum(lens) * token + rows * c["heads_q"] * (2 * c["D"] * e + 4)
            + (rows * -(-c["T"] // 32) * 4 if c["mask"] == "tree" else 0),
            "flops": 4 * seen * c["heads_q"] * c["D"]}


# ---- inputs -------------------------------------------------------------------------


def _tree_words(r, T, words):
    """A random tree's rows of bits: node i sees itself and its ancestors."""
    seen = [1]
    for i in range(1, T):
        seen.append(seen[r.randrange(max(0, i - 9), i)] | 1 << i)
    signed = lambda w: w - (1 << 32) if w >> 31 else w  # noqa: E731
    return [[signed(s >> 32 * k & 0xffffffff) for k in range(words)] for s in seen]


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)
    new, lens, H, D, HQ, dt = _tokens(c), _lens(c), c["heads"], c["D"], c["heads_q"], _TORCH[c["dt"]]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rows, starts = sum(new), [sum(new[:b]) for b in range(c["batch"] + 1)]
    held = lens if c["op"] in ("attn", "read") else new  # the tokens whose keys and values are made
    total = sum(held)
    # channels differ in size, as those of keys do
    spread = torch.empty(2, H, D, device="cuda").uniform_(0.3, 2.0, generator=g)
    wide = HQ if c["op"] != "attn" else 0
    fused = torch.empty(total, wide + 2 * H, D, device="cuda").normal_(0.0, 1.0, generator=g)
    fused[:, wide:wide + H] *= spread[0]
    fused[:, wide + H:] *= spread[1]
    fused = fused.to(dt)
    s = {"k": fused[:, wide:wide + H], "v": fused[:, wide + H:], "lens": ints(lens), "starts": ints(starts),
         "held": ints([sum(held[:b]) for b in range(c["batch"] + 1)]), "mask": None}
    if not c["fused"] or c["op"] in ("attn", "read"):
        s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
    if c["op"] == "attn":
        s["q"] = torch.empty(rows, HQ + 2 * H if c["fused"] else HQ, D, device="cuda")
        s["q"] = s["q"].normal_(0.0, 1.5, generator=g).to(dt)[:, :HQ]
        if c["mask"] == "tree":
            words = -(-c["T"] // 32)
            s["mask"] = ints([w for t in new for w in _tree_words(r, t, words)])
    if c["op"] == "keep":
        most, n = max(_kept(c)), _kept(c)
        s["keep"] = ints([sorted(r.sample(range(t), m)) + [-1] * (most - m) for t, m in zip(new, n)])
        s["n_keep"] = ints(n)
        s["lens_after"] = ints([a - t + m for a, t, m in zip(lens, new, n)])
        s["starts_after"] = ints([sum(n[:b]) for b in range(c["batch"] + 1)])
    # pages handed out in any order; entries that no token needs say so
    need = [-(-n // c["page"]) for n in lens]
    free = list(range(sum(need) + 3))
    r.shuffle(free)
    s["table"] = ints([[free.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need])
    s["num_pages"] = sum(need) + 3
    return s


def prepare(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    s["case"] = c
    if not own:
        if c["op"] in ("attn", "read"):
            s["cache"] = tuple(_padded(s, _plain_codes(s[k], c["kv"])) for k in ("k", "v"))
            del s["k"], s["v"]
        return s
    from integer_quantized_nn_gb300 import qnn
    new, n, dt, dev = _tokens(c), sum(_tokens(c)), _TORCH[c["dt"]], {"device": "cuda"}
    s["geom"] = geom = qnn.kv_geom(c["heads"], c["D"], c["page"], kv_dt=c["kv"])
    s["pages"] = torch.empty(s["num_pages"], qnn.qnn_kv_page_bytes(geom), dtype=torch.uint8, **dev)
    # the newest tokens of each sequence; equally many: no starts
    s["seqs"] = qnn.kv_seqs(s["pages"], s["table"], s["lens"], n, c["T"], starts=s["starts"] if c["ragged"] else None)
    if c["op"] in ("attn", "read"):
        whole = qnn.kv_seqs(s["pages"], s["table"], s["lens"], sum(_lens(c)), max(_lens(c)), starts=s["held"])
        qnn.q_kv_write(s["k"], s["v"], c["dt"], geom, whole)
        del s["k"], s["v"]
    if c["op"] == "attn":
        s["out"] = torch.empty(n, c["heads_q"], c["D"], dtype=dt, **dev)
        s["lse"] = torch.empty(n, c["heads_q"], **dev)
        s["ws"] = torch.empty(qnn.qnn_kv_attn_workspace_bytes(geom, s["seqs"], c["heads_q"]), dtype=torch.uint8, **dev)
        return s
    if c["op"] == "keep":
        n = sum(_kept(c))
        s["after"] = qnn.kv_seqs(s["pages"], s["table"], s["lens_after"], n, max(_kept(c)), starts=s["starts_after"])
    s["values"] = [torch.empty(n, c["heads"], c["D"], dtype=dt, **dev) for _ in range(2)]
    return s


# ---- the plain forms ----------------------------------------------------------------


def _plain_codes(x, kv):
    """Codes less their zero points, and scales, of each token and head: [tokens, heads, D], [tokens, heads, 1]."""
    x = x.to(torch.float32)
    if kv == "s8":
        s = x.abs().amax(dim=2, keepdim=True) / torch.tensor(127.0, device="cuda")
        q = torch.round(x / torch.where(s > 0, s, 1.0)).clamp(-127, 127)
        return q.to(torch.int8), s
    lo, hi = x.amin(dim=2, keepdim=True).clamp(max=0.0), x.amax(dim=2, keepdim=True).clamp(min=0.0)
    n = torch.tensor(15.0, device="cuda")
    s = (hi / n - lo / n).to(torch.bfloat16).to(torch.float32)
    d = torch.where(s > 0, s, 1.0)
    z = torch.round(-lo / d).clamp(0, 15)
    return ((torch.round(x / d) + z).clamp(0, 15) - z).to(torch.int8), s


def _padded(s, parts):
    """[tokens, ...] as [batch, longest, ...]."""
    at = torch.arange(max(_lens(s["case"])), device="cuda")
    i = (s["held"][:-1, None] + at).clamp(max=parts[0].shape[0] - 1).long()
    return tuple(p[i] for p in parts)


def _plain_values(codes, scale):
    return codes.to(torch.float32) * scale


def _row_places(starts, rows):
    """The sequence of each row, and the row's place in it."""
    row = torch.arange(rows, device="cuda")
    b = (row[:, None] >= starts[None, 1:]).sum(dim=1)
    return b, row - starts[b]


def _plain_read(s):
    c = s["case"]
    b, t = _row_places(s["starts"], sum(_tokens(c)))
    at = s["lens"][b] - (s["starts"][b + 1] - s["starts"][b]) + t
    return tuple(_plain_values(q[b, at], scale[b, at]).to(_TORCH[c["dt"]]) for q, scale in s["cache"])


def _plain_write(s):
    c = s["case"]
    kv = tuple(_plain_codes(s[x], c["kv"]) for x in ("k", "v"))
    if c["op"] == "keep":
        b, t = _row_places(s["starts_after"], sum(_kept(c)))
        kept = s["starts"][b] + s["keep"][b, t]
        kv = tuple((q[kept], scale[kept]) for q, scale in kv)
    return tuple(_plain_values(q, scale).to(_TORCH[c["dt"]]) for q, scale in kv)


def _plain_visible(s, T, L):
    """[batch, T, L]: which positions each newest token sees."""
    new = (s["starts"][1:] - s["starts"][:-1])[:, None, None]
    t, j = torch.arange(T, device="cuda")[None, :, None], torch.arange(L, device="cuda")[None, None, :]
    drafted = j - (s["lens"][:, None, None] - new)  # the place among the newest; negative: before them
    if s["mask"] is None:
        return (drafted < new) & (drafted <= t)
    row = (s["starts"][:-1, None] + t[:, :, 0]).clamp(max=s["mask"].shape[0] - 1).long()
    bits = (s["mask"][row][:, :, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    bits = bits.reshape(row.shape[0], T, -1).to(torch.bool)
    i = drafted.clamp(0, bits.shape[2] - 1).expand(-1, T, -1)
    return (drafted < new) & ((drafted < 0) | bits.gather(2, i.long()))


def _plain_attn(s):
    c = s["case"]
    B, T, H, D, HQ = c["batch"], max(_tokens(c)), c["heads"], c["D"], c["heads_q"]
    k, v = (_plain_values(q, scale).transpose(1, 2) for q, scale in s["cache"])  # [B, H, L, D]
    row = (s["starts"][:-1, None] + torch.arange(T, device="cuda")).clamp(max=s["q"].shape[0] - 1).long()
    q = s["q"][row].to(torch.float32).reshape(B, T, H, HQ // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    x = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).reshape(B, H, T, HQ // H, -1)
    x = torch.where(_plain_visible(s, T, k.shape[2])[:, None, :, None], x, -torch.inf)
    m = x.amax(dim=4, keepdim=True)
    p = torch.exp(x - torch.where(m > -torch.inf, m, 0.0))
    total = p.sum(dim=4, keepdim=True)
    out = (p.reshape(B, H, -1, k.shape[2]) @ v).reshape(B, H, T, -1, D) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total))[..., 0]
    b, t = _row_places(s["starts"], s["q"].shape[0])
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(B, T, HQ, D)[b, t].to(_TORCH[c["dt"]]),
            "lse": lse.permute(0, 2, 1, 3).reshape(B, T, HQ)[b, t]}


def run(s):
    c = s["case"]
    if not own:
        return {"attn": _plain_attn, "read": _plain_read}.get(c["op"], _plain_write)(s)
    from integer_quantized_nn_gb300 import qnn
    if c["op"] == "attn":
        qnn.q_kv_attn(s["q"], c["dt"], c["heads_q"], s["geom"], s["seqs"], 1 / math.sqrt(c["D"]), s["out"], s["ws"],
                      mask=s["mask"], lse=s["lse"], ld_q=s["q"].stride(0))
        return {"out": s["out"], "lse": s["lse"]}
    seqs = s["seqs"]
    if c["op"] != "read":
        qnn.q_kv_write(s["k"], s["v"], c["dt"], s["geom"], seqs, ld_k=s["k"].stride(0), ld_v=s["v"].stride(0))
    if c["op"] == "keep":
        qnn.q_kv_keep(s["geom"], seqs, s["keep"], s["n_keep"])
        seqs = s["after"]
    qnn.q_kv_read(s["values"][0], s["values"][1], c["dt"], s["geom"], seqs)
    return tuple(s["values"])


# ---- from the definitions, in 64 bits -----------------------------------------------


def _exact_values(x, kv):
    """What the codes of x [tokens, heads, D] stand for; the roundings of scale and quotients to
    fp32 (and bf16) are part of the definition, each of one operation on exact operands."""
    f32 = lambda a: a.to(torch.float32).double()  # noqa: E731
    x = x.double()
    if kv == "s8":
        s = f32(torch.linalg.vector_norm(x, float("inf"), dim=-1, keepdim=True) / 127)
        q = torch.where(s == 0, 0.0, f32(x / s)).round()
        return torch.minimum(torch.maximum(q, q.new_tensor(-127.0)), q.new_tensor(127.0)) * s
    top = torch.relu(x).max(dim=-1, keepdim=True).values
    low = torch.relu(-x).max(dim=-1, keepdim=True).values
    s = f32(f32(top / 15) + f32(low / 15)).to(torch.float32).bfloat16().double()
    z = torch.where(s == 0, 0.0, f32(low / s)).round().clamp(max=15)
    q = torch.where(s == 0, 0.0, f32(x / s)).round() + z
    return (q.clamp(0, 15) - z) * s


def exact(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    k, v = _exact_values(s["k"], c["kv"]), _exact_values(s["v"], c["kv"])
    new, lens, held = _tokens(c), _lens(c), s["held"].tolist()
    if c["op"] == "write":
        return k, v
    if c["op"] == "read":
        pick = torch.cat([torch.arange(held[b] + lens[b] - new[b], held[b] + lens[b], device="cuda")
                          for b in range(c["batch"])])
        return k[pick], v[pick]
    if c["op"] == "keep":
        pick = torch.cat([held[b] + s["keep"][b, :n] for b, n in enumerate(_kept(c))])
        return k[pick], v[pick]
    HQ, G = c["heads_q"], c["heads_q"] // c["heads"]
    out = torch.empty(sum(new), HQ, c["D"], dtype=torch.float64, device="cuda")
    lse = torch.empty(sum(new), HQ, dtype=torch.float64, device="cuda")
    first = 0
    for b in range(c["batch"]):
        T, n = new[b], lens[b]
        hide = torch.zeros(T, n, dtype=torch.bool, device="cuda")
        if c["mask"] == "causal":
            hide[:, n - T:] = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
        else:
            j = torch.arange(T, device="cuda")
            hide[:, n - T:] = (s["mask"][first:first + T].long()[:, j // 32] >> (j % 32)) % 2 == 0
        for h in range(HQ):
            kb, vb = k[held[b]:held[b] + n, h // G], v[held[b]:held[b] + n, h // G]
            x = (s["q"][first:first + T, h].double() @ kb.t()) / math.sqrt(c["D"])
            x.masked_fill_(hide, -math.inf)
            out[first:first + T, h] = torch.softmax(x, dim=1) @ vb
            lse[first:first + T, h] = torch.logsumexp(x, dim=1)
        first += T
    return {"out": out, "lse": lse}
