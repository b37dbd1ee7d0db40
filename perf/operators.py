"""What the attention side of a decode step costs: the cases, in plain torch and through the library.

Three operators that stand between the quantised projections of a decoder layer:

* ``append``    - new keys and values, rotated by their position, into a paged cache that holds 8 bits per
                  value with one scale for each block of tokens and head (and the queries rotated in the same call);
* ``attention`` - causal attention of those queries over that cache (one token, a few, or a whole prompt);
* ``norm``      - the norm after a block, its gate and residual scale, and the norm before the next block.

``run`` computes a case in plain torch (32 bits, elementary operations) or, where ``own`` is set, with the calls
that a user makes.  ``exact`` computes the same in 64 bits, sequence by sequence, from the definitions.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
QMAX = {"int8": 127.0, "e4m3": 448.0}
EPS = 1e-6


# ---------------------------------------------------------------- cases
def _append(name, batch, new, kv, hq, hkv, d, dtype, fmt, page, block, rot, style="half", ragged=False):
    return {"name": name, "op": "append", "batch": batch, "new": new, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "fmt": fmt, "page": page, "block": block, "rot": rot, "style": style, "ragged": ragged}


def _attention(name, batch, new, kv, hq, hkv, d, dtype, fmt, page, block, window=0, softcap=0.0, ragged=False):
    return {"name": name, "op": "attention", "batch": batch, "new": new, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "fmt": fmt, "page": page, "block": block, "window": window, "softcap": softcap,
            "ragged": ragged}


def _norm(name, rows, n, dtype, res, gate, scale, offset):
    return {"name": name, "op": "norm", "rows": rows, "n": n, "dtype": dtype, "res": res, "gate": gate,
            "scale": scale, "offset": offset}


def listed():
    return [
        # one decoded token of one user, fp32 as the projections give it: the smallest call there is
        _append("append_token", 1, 1, 38, 8, 4, 256, "f32", "int8", 64, 16, 256),
        # a serving batch, one token each, at every place of a block
        _append("append_batch61", 61, 1, 16, 32, 8, 128, "bf16", "e4m3", 16, 16, 64, style="interleaved", ragged=True),
        # a whole prompt of odd length behind a short prefix
        _append("append_prompt", 1, 4093, 4111, 8, 4, 256, "f32", "int8", 64, 32, 256),
        # the first tokens of a reply: nothing but latency
        _attention("attn_token_short", 1, 1, 37, 8, 4, 256, "f32", "int8", 64, 16),
        # one user, one kv head shared by eight query heads, a few thousand tokens of context
        _attention("attn_token_8k", 1, 1, 8191, 8, 1, 256, "f32", "int8", 64, 16),
        # one user with a very long document
        _attention("attn_token_128k", 1, 1, 131071, 16, 8, 128, "bf16", "e4m3", 64, 32),
        # a serving batch of unequal lengths
        _attention("attn_batch64", 64, 1, 8192, 32, 8, 128, "bf16", "int8", 64, 16, ragged=True),
        # drafted tokens verified together, a sliding window and soft-capped scores
        _attention("attn_verify5", 8, 5, 2049, 8, 4, 256, "f32", "e4m3", 32, 16, window=512, softcap=50.0, ragged=True),
        # a chunk of a long prompt over what is already in the cache
        _attention("attn_prompt", 1, 2048, 8192, 16, 8, 128, "bf16", "int8", 64, 16),
        # one decoded token's hidden state between two blocks
        _norm("norm_token", 1, 2048, "f32", "f32", "none", 1.0, 0.0),
        # a serving batch of an odd width, each row with its own gate
        _norm("norm_rows61_odd", 61, 1531, "bf16", "f32", "row", 0.5, 1.0),
        # a prompt's hidden states
        _norm("norm_prompt", 8191, 2048, "bf16", "bf16", "vector", 0.75, 1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "norm"])
    if op == "norm":
        n = _log(rng, 64, 16384)
        return {k: v for k, v in _norm("", _log(rng, 1, min(8191, max(1, 8191 * 2048 // n))), n,
                                       *rng.choice([("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")]),
                                       rng.choice(["none", "vector", "row"]), rng.choice([1.0, 0.5, 0.75]),
                                       rng.choice([0.0, 1.0])).items() if k != "name"}
    d = rng.choice([64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    block = min(page, rng.choice([16, 32, 64]))
    dtype, fmt = rng.choice(["f32", "bf16", "f16"]), rng.choice(["int8", "e4m3"])
    ragged = rng.random() < 0.5
    if op == "append":
        batch = rng.choice([1, 1, _log(rng, 1, 128)])
        most = max(1, 4093 * 16 * 256 // (batch * (2 * hkv + hq) * d))  # the listed prompt's values
        new = rng.choice([1, _log(rng, 1, min(4093, most))])
        c = _append("", batch, new, new + rng.randrange(0, 64), hq, hkv, d, dtype, fmt, page, block,
                    rng.choice([d, d // 2, d // 4]), rng.choice(["half", "interleaved"]), ragged)
    else:
        batch = rng.choice([1, _log(rng, 1, 64)])
        # within the largest listed cases: 0.6 GB of cache, 1.2e11 operations
        kv = _log(rng, 1, max(1, min(131071, 64 * 8192 * 1024 // (batch * hkv * d) // 4)))
        most = max(1, min(2048, kv, 10 ** 11 // (4 * d * hq * batch * kv)))
        new = rng.choice([1, _log(rng, 1, min(16, most)), _log(rng, 1, most)])
        c = _attention("", batch, new, kv, hq, hkv, d, dtype, fmt, page, block, rng.choice([0, 0, 0, 512, 129]),
                       rng.choice([0.0, 0.0, 50.0]), ragged)
    del c["name"]
    return c


def _lengths(c):
    """(tokens in the cache after the call, new tokens) of each sequence: fixed by the case, not by the seed."""
    kv, new = [], []
    for b in range(c["batch"]):
        f = (b * 37 % c["batch"]) / c["batch"] if c["ragged"] else 0.0
        n = max(1, c["new"] - int(c["new"] * f / 2))
        new.append(n)
        kv.append(max(n, c["kv"] - int(c["kv"] * 0.9 * f)))
    return kv, new


def _visible(c):
    """(query, token) pairs that the mask leaves, and the cache tokens that some query sees, over all sequences."""
    pairs = tokens = 0
    for kv, new in zip(*_lengths(c)):
        w = c["window"] or kv
        lo, hi = kv - new, kv - 1  # positions of the first and the last query
        short = max(0, min(hi, w - 2) - lo + 1)  # queries that see the whole past
        pairs += short * (2 * lo + short + 1) // 2 + (new - short) * w
        tokens += kv - max(0, lo - w + 1)
    return pairs, tokens


def work(c):
    if c["op"] == "norm":
        e, r = DTYPES[c["dtype"]].itemsize, DTYPES[c["res"]].itemsize
        gate = {"none": 0, "vector": c["n"], "row": c["rows"] * c["n"]}[c["gate"]]
        return {"bytes": c["rows"] * c["n"] * (2 * e + 2 * r) + (2 * c["n"] + gate) * e, "flops": 10 * c["rows"] * c["n"]}
    e = DTYPES[c["dtype"]].itemsize
    if c["op"] == "append":
        t = sum(_lengths(c)[1])
        return {"bytes": t * c["d"] * (c["hkv"] * (2 * e + 2) + c["hq"] * 2 * e) + t * c["rot"] * 4,
                "flops": t * c["d"] * (4 * c["hkv"] + 3 * (c["hkv"] + c["hq"]))}
    pairs, tokens = _visible(c)
    return {"bytes": tokens * c["hkv"] * (2 * c["d"] + 8.0 / c["block"]) + 2 * sum(_lengths(c)[1]) * c["hq"] * c["d"] * e,
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ---------------------------------------------------------------- inputs
def _normal(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _eight_bits(x, fmt):
    """Codes of values within the format's range: int8, or e4m3."""
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _cache(c, g):
    """A filled cache: keys with a few loud channels, values, tokens of unequal size; pages in random order."""
    kv, new = _lengths(c)
    pages = [-(-n // c["page"]) for n in kv]
    total, nb = sum(pages), c["page"] // c["block"]
    x = torch.randn((2, total, c["hkv"], nb, c["block"], c["d"]), generator=g, device="cuda")
    loud = 1 + 3 * (torch.rand((2, 1, c["hkv"], 1, 1, c["d"]), generator=g, device="cuda") > 0.95)
    x *= loud * torch.exp(0.4 * torch.randn((2, total, c["hkv"], nb, c["block"], 1), generator=g, device="cuda"))
    scales = x.abs().amax(dim=(4, 5)) / QMAX[c["fmt"]]
    x /= scales[..., None, None]
    codes = _eight_bits(x, c["fmt"]).view(2, total, c["hkv"], c["page"], c["d"])
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((c["batch"], max(pages)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)])
    return {"codes": codes, "scales": scales, "table": table, "block": c["block"],
            "kv_len": torch.tensor(kv, dtype=torch.int32, device="cuda"),
            "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"), "tokens": int(cu[-1])}


def _inputs(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm":
        rows, n = c["rows"], c["n"]
        gate = None if c["gate"] == "none" else _normal(g, (n,) if c["gate"] == "vector" else (rows, n), dt)
        # the residual stream has outgrown the block's output, as it does in the later layers
        return {"y": _normal(g, (rows, n), dt), "h": (8 * _normal(g, (rows, n))).to(DTYPES[c["res"]]),
                "w_post": (0.1 * _normal(g, (n,)) + 1 - c["offset"]).to(dt),
                "w_pre": (0.1 * _normal(g, (n,)) + 1 - c["offset"]).to(dt), "gate": gate}
    s = _cache(c, g)
    t = s["tokens"]
    s["q"] = _normal(g, (t, c["hq"], c["d"]), dt)
    if c["op"] == "append":
        s["k"] = _normal(g, (t, c["hkv"], c["d"]), dt)
        s["v"] = (0.7 * _normal(g, (t, c["hkv"], c["d"]))).to(dt)
        f = 10000.0 ** (-torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / c["rot"])
        a = torch.arange(c["kv"], device="cuda", dtype=torch.float64)[:, None] * f
        s["cos"], s["sin"] = a.cos().float(), a.sin().float()
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    if own:
        import quantized_weight_gemv_gb300 as qg
        if case["op"] == "norm":
            s["h_out"], s["z"] = torch.empty_like(s["h"]), torch.empty_like(s["y"])
            s["plan"] = qg.NormGateResidual(s["y"], s["h"], s["w_post"], s["w_pre"], gate=s["gate"],
                                            res_scale=case["scale"], eps=EPS, w_offset=case["offset"],
                                            h_out=s["h_out"], z=s["z"])
            return s
        s["cache"] = qg.KV8Cache(s["codes"], s["scales"], s["table"], s["block"])
        s["out"] = torch.empty_like(s["q"])
        cu = s["cu"] if case["new"] > 1 else None  # one token per sequence needs no offsets
        if case["op"] == "append":
            s["plan"] = qg.KV8Append(s["cache"], s["k"], s["v"], s["kv_len"], cu, cos=s["cos"], sin=s["sin"],
                                     rope_style=case["style"], q=s["q"], q_out=s["out"])
        else:
            s["plan"] = qg.KV8Attention(s["cache"], s["q"], s["kv_len"], cu, out=s["out"],
                                        window=case["window"], softcap=case["softcap"])
    return s


# ---------------------------------------------------------------- the plain forms
def _rms(x, w, offset):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + offset)


def _plain_norm(s):
    c = s["case"]
    u = _rms(s["y"].float(), s["w_post"], c["offset"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = (s["h"].float() + u) * c["scale"]
    return {"h": h.to(s["h"].dtype), "z": _rms(h, s["w_pre"], c["offset"]).to(s["y"].dtype)}


def _places(s):
    """The sequence and the position of each new token."""
    t = torch.arange(s["tokens"], device="cuda", dtype=torch.int32)
    b = torch.searchsorted(s["cu"][1:], t, right=True)
    first = s["kv_len"] - (s["cu"][1:] - s["cu"][:-1])
    return b, (first[b] + t - s["cu"][b]).long(), first[b].long()


def _rotate(x, cos, sin, rot, style):
    """The first `rot` values of each head rotated, in pairs (i, i + rot/2) or (2i, 2i + 1)."""
    c, s, r, rest = cos[:, None], sin[:, None], x[..., :rot], x[..., rot:]
    if style == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        return torch.cat([a * c - b * s, b * c + a * s, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), rest], -1)


def _plain_append(s):
    c = s["case"]
    pages, hkv, page, d = s["codes"].shape[1:]
    blk, nb, qmax = c["block"], c["page"] // c["block"], QMAX[c["fmt"]]
    b, pos, first = _places(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["style"]).to(s["q"].dtype)
    x = torch.stack([_rotate(s["k"].float(), cos, sin, c["rot"], c["style"]), s["v"].float()])
    where = s["table"][b, pos // page].long()
    flat = where * nb + pos % page // blk  # the block of each new token
    # a block's scale only grows while it fills; the first token in it starts it anew
    old = s["scales"].transpose(2, 3).reshape(2, pages * nb, hkv)
    old[:, flat] = old[:, flat] * (first > pos // blk * blk)[:, None]
    new = torch.zeros_like(old).scatter_reduce_(1, flat[:, None].expand(2, -1, hkv), x.abs().amax(-1), "amax")
    new = torch.maximum(old, new / qmax)
    old, new = (v.view(2, pages, nb, hkv).transpose(2, 3) for v in (old, new))
    was = s["codes"].float().view(2, pages, hkv, nb, blk, d) * old[..., None, None]
    at = new[..., None, None]
    codes = _eight_bits(torch.where(at > 0, was / at, 0.0), c["fmt"]).view(torch.uint8).reshape(s["codes"].shape)
    step = new[:, where, :, pos % page // blk].permute(1, 0, 2)[..., None]
    codes[:, where, :, pos % page] = _eight_bits(torch.where(step > 0, x / step, 0.0),
                                                 c["fmt"]).view(torch.uint8).transpose(0, 1)
    s["codes"].view(torch.uint8).copy_(codes)
    s["scales"].copy_(new)
    values = s["codes"].float().view(2, pages, hkv, nb, blk, d) * at
    return {"q": q, "kv": values.reshape(s["codes"].shape)}


def _plain_attention(s):
    c = s["case"]
    n, g = c["new"], c["hq"] // c["hkv"]
    pages, hkv, page, d = s["codes"].shape[1:]
    tab = s["table"].long()
    length = tab.shape[1] * page
    codes = s["codes"].view(torch.uint8)[:, tab].view(s["codes"].dtype).float()  # [2][batch][pages][hkv][page][d]
    step = s["scales"][:, tab].repeat_interleave(c["block"], -1)[..., None]
    k, v = (codes * step).transpose(2, 3).reshape(2, c["batch"], c["hkv"], length, d)
    b, pos, first = _places(s)
    row = pos - first
    q = torch.zeros((c["batch"], n, c["hq"], d), device="cuda")
    q[b, row] = s["q"].float()
    q = q.view(c["batch"], n, hkv, g * d).transpose(1, 2).reshape(c["batch"], hkv, n * g, d)
    p = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    if c["softcap"]:
        p = c["softcap"] * torch.tanh(p / c["softcap"])
    new = s["cu"][1:] - s["cu"][:-1]
    at = (s["kv_len"] - new)[:, None] + torch.arange(n, device="cuda")  # the position of each query
    t = torch.arange(length, device="cuda")
    seen = t <= at[..., None]
    if c["window"]:
        seen = seen & (t > at[..., None] - c["window"])
    p = p.view(c["batch"], hkv, n, g, length).masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(c["batch"], hkv, n * g, length)
    o = torch.matmul(p, v).view(c["batch"], hkv, n, g * d).transpose(1, 2).reshape(c["batch"], n, c["hq"], d)
    return o[b, row].to(s["q"].dtype)


def run(s):
    op = s["case"]["op"]
    if own:
        s["plan"].run()
        if op == "norm":
            return {"h": s["h_out"], "z": s["z"]}
        # the cache's codes come back as the values they stand for
        return {"q": s["out"], "kv": s["cache"].values()} if op == "append" else s["out"]
    return {"norm": _plain_norm, "append": _plain_append, "attention": _plain_attention}[op](s)


# ---------------------------------------------------------------- 64 bits
def _exact_norm(c, s):
    def rms(x, w):
        return x / ((x ** 2).sum(-1, keepdim=True) / c["n"] + EPS).sqrt() * (c["offset"] + w.double())
    u = rms(s["y"].double(), s["w_post"])
    h = c["scale"] * (s["h"].double() + (u if s["gate"] is None else s["gate"].double() * u))
    return {"h": h, "z": rms(h, s["w_pre"])}


def _turned(x, pos, c):
    """x [tokens][heads][d] as complex pairs, turned by position x frequency (the 32-bit tables hold its cos and sin)."""
    (cos, sin), r = c["tables"], c["rot"]
    x = x.double()
    h = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["style"] == "half" else x[..., :r].unflatten(-1, (r // 2, 2))
    z = torch.view_as_complex(h.contiguous()) * torch.complex(cos[pos].double(), sin[pos].double())[:, None]
    h = torch.view_as_real(z)
    h = h.transpose(-1, -2).flatten(-2) if c["style"] == "half" else h.flatten(-2)
    return torch.cat([h, x[..., r:]], -1)


def _exact_append(c, s):
    c = {**c, "tables": (s["cos"], s["sin"])}
    blk, page, qmax = c["block"], c["page"], QMAX[c["fmt"]]
    codes, scales = s["codes"].double().cpu(), s["scales"].double().cpu()
    table, at, out = s["table"].cpu(), 0, []
    for b, (kv, new) in enumerate(zip(*_lengths(c))):
        pos = torch.arange(kv - new, kv, device="cuda")
        out.append(_turned(s["q"][at:at + new], pos, c))
        x = torch.stack([_turned(s["k"][at:at + new], pos, c), s["v"][at:at + new].double()]).cpu()
        at += new
        for start in range((kv - new) // blk * blk, kv, blk):
            lo, hi = max(start, kv - new), min(start + blk, kv)
            i, w = int(table[b, start // page]), start % page // blk
            part = x[:, lo - (kv - new):hi - (kv - new)].transpose(1, 2)  # [2][hkv][tokens][d]
            was = scales[:, i, :, w] if lo > start else torch.zeros_like(scales[:, i, :, w])
            now = torch.maximum(was, part.abs().amax((2, 3)) / qmax)
            here = codes[:, i, :, w * blk:(w + 1) * blk]
            here = here * (was / now)[..., None, None]
            here[:, :, lo - start:hi - start] = part / now[..., None, None]
            codes[:, i, :, w * blk:(w + 1) * blk] = _eight_bits(here, c["fmt"]).double()
            scales[:, i, :, w] = now
    kv = codes.unflatten(3, (-1, blk)) * scales[..., None, None]
    return {"q": torch.cat(out), "kv": kv.flatten(3, 4)}


def _exact_attention(c, s):
    out, at, g = [], 0, c["hq"] // c["hkv"]
    for b, (kv, new) in enumerate(zip(*_lengths(c))):
        ids = s["table"][b, :-(-kv // c["page"])].long()
        x = s["codes"].view(torch.uint8)[:, ids].view(s["codes"].dtype).double().unflatten(3, (-1, c["block"]))
        x = (x * s["scales"][:, ids].double()[..., None, None]).flatten(3, 4).transpose(1, 2).flatten(2, 3)[:, :, :kv]
        q = s["q"][at:at + new].double().unflatten(1, (-1, g))
        at += new
        e = torch.einsum("nhgd,hld->hgnl", q, x[0]) / math.sqrt(c["d"])
        if c["softcap"]:
            e = c["softcap"] * torch.tanh(e / c["softcap"])
        j, i = torch.arange(kv, device="cuda"), torch.arange(kv - new, kv, device="cuda")[:, None]
        hide = (j > i) | (j <= i - (c["window"] or kv))
        e = torch.softmax(e.masked_fill(hide, -math.inf), -1)
        out.append(torch.einsum("hgnl,hld->nhgd", e, x[1]).flatten(1, 2))
    return torch.cat(out)


def exact(case, seed):
    s = _inputs(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attention": _exact_attention}[case["op"]](case, s)
