"""Plain fp64 numpy forms of the cache attention and of the norms around a block (test infrastructure)."""
import numpy as np


def attention(k, v, q, first, scale, window=0, softcap=0.0):
    """k, v [length][kv heads][d]; q [tokens][heads][d], token i at position first + i -> [tokens][heads][d]."""
    out = np.zeros_like(q)
    for i in range(q.shape[0]):
        lo, hi = max(0, first + i - window + 1) if window > 0 else 0, first + i + 1
        for h in range(q.shape[1]):
            g = h // (q.shape[1] // k.shape[1])
            s = k[lo:hi, g] @ q[i, h] * scale
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            e = np.exp(s - s.max())
            out[i, h] = e @ v[lo:hi, g] / e.sum()
    return out


def norms(y, h, w_post, w_pre, res_scale, eps):
    """(h', z) of rows y, h: h' = (h + rms(y) w_post) res_scale, z = rms(h') w_pre."""
    def rms(x):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = (h + rms(y) * w_post) * res_scale
    return h, rms(h) * w_pre
