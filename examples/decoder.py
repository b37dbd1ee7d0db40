"""A small decoder put together from the library's calls: prompt in chunks, then one token at a time.

Random Q4 weights in the shapes of the decode-layer workload (hidden 2048, 8 query and 4 kv heads of 256,
FFN 16384) and a soft-capped Q4 head; per layer

    q, k, v  = Wq z, Wk z, Wv z            qgemv_grouped (one token) or qgemv_batched (a chunk)
    cache   <- rotated k, v; q rotated     kv8_rope_append
    a        = attention(q, cache)         kv8_attention (a sliding window on every other layer)
    h, z     = norms around o = Wo a       rmsnorm_gate_residual
    f        = gelu(Wg z) * (Wu z)         two GEMVs, PyTorch for the gate
    h, z     = norms around Wd f           rmsnorm_gate_residual, with the layer's residual scale

and ``vocab_softcap_argmax`` picks the next token.  A decode step has no host decision in it, so it is
captured in a CUDA graph and replayed, the sequence length being advanced on the device.

    python examples/decoder.py --layers 4 --prompt 100 --tokens 32
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import datagen  # noqa: E402
import quantized_weight_gemv_gb300 as qg  # noqa: E402

HIDDEN, FFN, Q_HEADS, KV_HEADS, HEAD_DIM, VOCAB = 2048, 16384, 8, 4, 256, 8192
CHUNK = 8  # prompt tokens per pass: qgemv_batched takes batch * k <= 131072
WINDOW = 512
PAGE, BLOCK = 64, 16
PROJECTIONS = {"q": (Q_HEADS * HEAD_DIM, HIDDEN), "k": (KV_HEADS * HEAD_DIM, HIDDEN), "v": (KV_HEADS * HEAD_DIM, HIDDEN),
               "o": (HIDDEN, Q_HEADS * HEAD_DIM), "gate": (FFN, HIDDEN), "up": (FFN, HIDDEN), "down": (HIDDEN, FFN)}


class Layer:
    def __init__(self, seed, device, max_tokens, window):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.w = {name: qg.to_device(datagen.make_quantized(4, seed + i, *shape), device)
                  for i, (name, shape) in enumerate(PROJECTIONS.items())}
        self.norms = [1 + 0.1 * torch.randn(HIDDEN, generator=g, device=device) for _ in range(3)]
        self.scale = 0.9  # the layer's residual scale
        self.window = window
        pages = -(-max_tokens // PAGE)
        self.cache = qg.KV8Cache.empty(pages, KV_HEADS, HEAD_DIM, 1, pages, PAGE, BLOCK, device=device)
        self.cache.page_table.copy_(torch.randperm(pages, generator=g, device=device).to(torch.int32)[None])


class Decoder:
    """``prefill(tokens)`` reads a prompt, ``step()`` enqueues one decode step; ``token`` holds the last pick."""

    def __init__(self, layers: int = 4, max_tokens: int = 1024, seed: int = 1, device="cuda"):
        device = torch.device(device, 0) if device == "cuda" else torch.device(device)
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.device, self.max_tokens = device, max_tokens
        self.layers = [Layer(seed + 100 * (i + 1), device, max_tokens, WINDOW if i % 2 == 0 else 0) for i in range(layers)]
        self.head = qg.to_device(datagen.make_quantized(4, seed, VOCAB, HIDDEN), device)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g, device=device)
        self.norm_in = 1 + 0.1 * torch.randn(HIDDEN, generator=g, device=device)
        self.norm_out = 1 + 0.1 * torch.randn(HIDDEN, generator=g, device=device)
        f = 10000.0 ** (-torch.arange(HEAD_DIM // 2, device=device) * 2.0 / HEAD_DIM)
        a = torch.arange(max_tokens, device=device)[:, None] * f
        self.cos, self.sin = a.cos().contiguous(), a.sin().contiguous()
        self.kv_len = torch.zeros(1, dtype=torch.int32, device=device)
        self.token = torch.zeros(1, dtype=torch.int32, device=device)
        self.logits = torch.empty(VOCAB, device=device)
        self.vocab_ws = qg.vocab_workspace(device)
        self.kv_ws = qg.kv8_workspace(HEAD_DIM, device)
        self._passes = {}

    def _plan(self, tokens):
        """The calls of a pass over `tokens` new tokens, with their buffers: made once per count."""
        if tokens in self._passes:
            return self._passes[tokens]
        new = lambda n: torch.empty(tokens, n, device=self.device)  # noqa: E731
        h, z, gate = new(HIDDEN), new(HIDDEN), new(FFN)
        cu = torch.tensor([0, tokens], dtype=torch.int32, device=self.device) if tokens > 1 else None
        calls = [qg.NormGateResidual(None, h, w_pre=self.norm_in, h_out=None, z=z).run]
        for i, layer in enumerate(self.layers):
            after = self.layers[i + 1].norms[0] if i + 1 < len(self.layers) else self.norm_out
            out = {name: new(n) for name, (n, _) in PROJECTIONS.items()}
            heads = lambda t: t.view(tokens, -1, HEAD_DIM)  # noqa: E731
            append = qg.KV8Append(layer.cache, heads(out["k"]), heads(out["v"]), self.kv_len, cu, self.cos, self.sin,
                                  q=heads(out["q"]), q_out=heads(out["q"]))
            attend = qg.KV8Attention(layer.cache, heads(out["q"]), self.kv_len, cu, window=layer.window, ws=self.kv_ws)
            a = attend.out.view(tokens, -1)
            calls += self._products(layer, [("q", z), ("k", z), ("v", z)], out, tokens)
            calls += [append.run, attend.run]
            calls += self._products(layer, [("o", a)], out, tokens)
            calls += [qg.NormGateResidual(out["o"], h, layer.norms[1], layer.norms[2], h_out=h, z=z).run]
            calls += self._products(layer, [("gate", z), ("up", z)], out, tokens)
            calls += [lambda o=out: torch.mul(torch.nn.functional.gelu(o["gate"], approximate="tanh"), o["up"], out=gate)]
            calls += self._products(layer, [("down", gate)], out, tokens)
            calls += [qg.NormGateResidual(out["down"], h, layer.norms[0], after, res_scale=layer.scale, h_out=h, z=z).run]
        self._passes[tokens] = (h, z, calls)
        return self._passes[tokens]

    def _products(self, layer, what, out, tokens):
        if tokens == 1 and len(what) > 1:
            group = qg.GroupedGemv(4, [layer.w[n] for n, _ in what], [x[0] for _, x in what], [out[n][0] for n, _ in what])
            return [group.run]
        calls = []
        for n, x in what:
            w = layer.w[n]
            ws = qg.batched_workspace(4, x.shape[1], tokens, self.device)
            calls.append(lambda w=w, n=n, x=x, ws=ws: qg.qgemv_batched(4, w["lo"], None, w["scale"], w["min"], x, out[n], ws=ws))
        return calls

    def forward(self, embeddings):
        """One pass over [tokens][HIDDEN] new embeddings; returns the normed hidden states."""
        tokens = embeddings.shape[0]
        h, z, calls = self._plan(tokens)
        self.kv_len += tokens
        h.copy_(embeddings)
        for call in calls:
            call()
        return z

    def pick(self, z):
        qg.vocab_softcap_argmax(4, self.head["lo"], None, self.head["scale"], self.head["min"], z, 30.0,
                                logits=self.logits, argmax=self.token, ws=self.vocab_ws)

    def prefill(self, tokens):
        for at in range(0, tokens.numel(), CHUNK):
            z = self.forward(self.embed[tokens[at:at + CHUNK].long()])
        self.pick(z[-1].contiguous())

    def step(self):
        z = self.forward(self.embed[self.token.long()])
        self.pick(z[0])

    def capture(self):
        """The decode step as a CUDA graph (run one step eagerly first)."""
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--tokens", type=int, default=32)
    args = ap.parse_args()
    m = Decoder(args.layers, max_tokens=args.prompt + args.tokens + 2)
    prompt = torch.randint(0, VOCAB, (args.prompt,), device=m.device)
    m.prefill(prompt)
    picked = [int(m.token)]
    m.step()
    picked.append(int(m.token))
    graph = m.capture()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(args.tokens - 2):
        graph.replay()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(1, args.tokens - 2)
    if qg.device_error():
        raise RuntimeError("device error word set")
    print(f"{args.layers} layers, {args.prompt} prompt tokens, then {args.tokens}: first picks {picked}, last {int(m.token)}, "
          f"{t * 1e6:.0f} us per decoded token")


if __name__ == "__main__":
    main()
