"""Plain implementations of the cache, attention and norm operators for the tests (numpy, CPU).

The append's codes are defined by correctly rounded fp32 steps, so its reference is fp32
numpy, step by step, and is compared bit for bit; attention and the norms are in 64 bits.
"""
import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def e4m3_values():
    """The value of each of the 256 codes."""
    return torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()


E4M3 = e4m3_values()


def to_codes(x, fmt):
    """Nearest code, ties to even, saturating; NaN gives 0.  fp32 in, uint8 bit patterns out."""
    x = np.where(np.isnan(x), np.float32(0), x)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    pos = E4M3[:127].astype(np.float64)  # 0 .. 448, ascending
    a = np.minimum(np.abs(x).astype(np.float64), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    near = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (near | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def code_values(codes, fmt):
    return codes.view(np.int8).astype(np.float32) if fmt == "int8" else E4M3[codes]


def rotate(x, cos, sin, style):
    """x fp32 [..., d]; cos, sin fp32 [..., rot/2]; every product and sum rounded on its own."""
    x = x.copy()
    r = 2 * cos.shape[-1]
    if style == "half":
        a, b = x[..., :r // 2].copy(), x[..., r // 2:r].copy()
        x[..., :r // 2] = a * cos - b * sin
        x[..., r // 2:r] = b * cos + a * sin
    else:
        a, b = x[..., 0:r:2].copy(), x[..., 1:r:2].copy()
        x[..., 0:r:2] = a * cos - b * sin
        x[..., 1:r:2] = b * cos + a * sin
    return x


def append(codes, scales, table, fmt, block, k, v, first, new, cos=None, sin=None, positions=None, style="half"):
    """codes uint8 [2][pages][heads][page][d] and scales fp32, changed in place; k, v fp32 [tokens][heads][d]."""
    page, t = codes.shape[3], 0
    f32 = np.float32
    for b, (f, n) in enumerate(zip(first, new)):
        for start in range(f // block * block, f + n, block):
            lo, hi = max(start, f), min(start + block, f + n)
            rows = slice(t + lo - f, t + hi - f)
            i, w = table[b][start // page], start % page
            kk = k[rows]
            if cos is not None:
                at = positions[rows] if positions is not None else np.arange(lo, hi)
                kk = rotate(kk, cos[at][:, None], sin[at][:, None], style)
            for which, x in ((0, kk), (1, v[rows])):
                for h in range(codes.shape[2]):
                    a = np.abs(x[:, h])
                    a = a[np.isfinite(a)]
                    old = f32(0) if lo == start else scales[which, i, h, w // block]
                    s = max(old, f32((a.max() if a.size else f32(0)) / f32(QMAX[fmt])))
                    here = codes[which, i, h, w:w + block]
                    if lo == start:
                        here[:] = 0
                    elif s > old:
                        here[:] = to_codes(code_values(here, fmt) * old / s, fmt)
                    with np.errstate(over="ignore", invalid="ignore"):
                        here[lo - start:hi - start] = to_codes(x[:, h] / s, fmt) if s > 0 else 0
                    scales[which, i, h, w // block] = s
        t += n


def dequantise(codes, scales, fmt, block):
    """fp64 values of codes [..., page, d] with scales [..., page // block]."""
    return code_values(codes, fmt).astype(np.float64) * np.repeat(scales.astype(np.float64), block, -1)[..., None]


def attention(kv, table, page, q, first, new, scale, window=0, softcap=0.0):
    """kv fp64 [2][pages][heads][page][d]; q fp64 [tokens][hq][d] -> (out, lse) in 64 bits."""
    hq, hkv = q.shape[1], kv.shape[2]
    out, lse, t = np.zeros_like(q), np.full(q.shape[:2], -np.inf), 0
    for b, (f, n) in enumerate(zip(first, new)):
        for i in range(n):
            p = f + i
            lo = max(0, p - window + 1) if window > 0 else 0
            at = np.arange(lo, p + 1)
            ids = np.asarray(table[b])[at // page]
            for h in range(hq):
                g = h // (hq // hkv)
                s = kv[0, ids, g, at % page] @ q[t, h] * scale
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                m = s.max()
                e = np.exp(s - m)
                out[t, h] = e @ kv[1, ids, g, at % page] / e.sum()
                lse[t, h] = m + np.log(e.sum())
            t += 1
    return out, lse


def norm(y, h, w_post, w_pre, gate, res_scale, eps, w_offset):
    """All fp64; any of y, w_post, w_pre, gate None."""
    def rms(x, w):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (w + w_offset)
    if y is not None:
        u = y if w_post is None else rms(y, w_post)
        h = h + (u if gate is None else gate * u)
    h = h * res_scale
    return h, None if w_pre is None else rms(h, w_pre)


class Scene:
    """A cache on both sides, sequences with `first` tokens already in it and `new` ones to come."""

    def __init__(self, seed, fmt, heads, d, page, block, first, new, extra_pages=3, quiet=False):
        self.rng = np.random.default_rng(seed)
        self.fmt, self.heads, self.d, self.page, self.block = fmt, heads, d, page, block
        self.first, self.new = list(first), list(new)
        need = [-(-(f + n) // page) for f, n in zip(first, new)]
        pages = sum(need) + extra_pages
        order = self.rng.permutation(pages)
        self.table = np.full((len(first), max(need + [1])), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        x = self.rng.standard_normal((2, pages, heads, page // block, block, d)).astype(np.float32)
        x *= np.exp(0.5 * self.rng.standard_normal((2, pages, heads, page // block, block, 1))).astype(np.float32)
        self.scales = (np.abs(x).max((4, 5)) / np.float32(QMAX[fmt])).astype(np.float32)
        self.codes = to_codes(x / self.scales[..., None, None], fmt).reshape(2, pages, heads, page, d)
        if quiet:
            return
        # what no sequence holds yet may be anything: the largest codes (8-bit NaN) and scales that are not finite
        held = np.zeros((pages, page), bool)
        for b, f in enumerate(first):
            for j in range(f):
                held[self.table[b, j // page], j % page] = True
        junk = np.uint8(0x7f)
        for w in range(2):
            self.codes[w].transpose(0, 2, 1, 3)[~held] = junk
            used = held.reshape(pages, page // block, block).any(2)
            self.scales[w].transpose(0, 2, 1)[~used] = np.float32(np.nan if w else np.inf)

    def rows(self, heads, dtype):
        """(torch CPU tensor of dtype, the same as fp64 numpy) [tokens][heads][d]."""
        t = torch.from_numpy(self.rng.standard_normal((sum(self.new), heads, self.d)).astype(np.float32)).to(dtype)
        return t, t.double().numpy()

    def device(self, qg, dev="cuda"):
        codes = torch.from_numpy(self.codes.copy()).to(dev).view(CODE[self.fmt])
        return qg.KV8Cache(codes, torch.from_numpy(self.scales.copy()).to(dev),
                           torch.from_numpy(self.table).to(dev), self.block)

    def kv_len(self, dev="cuda"):
        return torch.tensor([f + n for f, n in zip(self.first, self.new)], dtype=torch.int32, device=dev)

    def cu(self, dev="cuda"):
        return torch.tensor(np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32), device=dev)

    def fill(self):
        """Clean contents for the new tokens too (what an append would have left): returns self."""
        for b, (f, n) in enumerate(zip(self.first, self.new)):
            for j in range(f, f + n):
                i, s = self.table[b, j // self.page], j % self.page
                for w in range(2):
                    bad = ~np.isfinite(self.scales[w, i, :, s // self.block])
                    self.scales[w, i, :, s // self.block][bad] = 0.02
                    self.codes[w, i, :, s] = to_codes(
                        (self.rng.standard_normal((self.heads, self.d)) * QMAX[self.fmt] / 3).astype(np.float32), self.fmt)
        return self

    def values(self):
        with np.errstate(invalid="ignore"):
            return dequantise(self.codes, self.scales, self.fmt, self.block)


def tables(n_pos, rot):
    f = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    a = np.arange(n_pos)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
