"""The example decoder: its cache, attention and norm calls against their definitions as they are used, the
chunked prompt against token by token, and the captured decode step against the eager one."""
import numpy as np
import pytest
import torch

import quantized_weight_gemv_gb300 as qg
from examples import decoder as E
from tests import _kv8 as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def models():
    from quantized_weight_gemv_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield [E.Decoder(layers=2, max_tokens=128, seed=7) for _ in range(2)]
    assert qg.device_error() == 0


def test_prompt_in_chunks_and_token_by_token_agree(models):
    a, b = models
    prompt = torch.randint(0, E.VOCAB, (45,), generator=torch.Generator().manual_seed(3)).to(a.device)
    a.prefill(prompt)
    for i in range(prompt.numel()):
        z = b.forward(b.embed[prompt[i:i + 1].long()])
    b.pick(z[0])
    assert int(a.kv_len) == int(b.kv_len) == 45
    # the passes sum in another order and a rounded code may flip: 8-bit activations set the scale
    la, lb = a.logits.double().cpu().numpy(), b.logits.double().cpu().numpy()
    assert np.linalg.norm(la - lb) <= 0.05 * np.linalg.norm(la)
    va, vb = (m.layers[0].cache.values().double().cpu().numpy()[:, m.layers[0].cache.page_table[0, 0].item()] for m in models)
    held = slice(0, 45)
    assert np.abs(va[:, :, held] - vb[:, :, held]).max() <= np.abs(va).max() / 60  # one code, now and then


def test_attention_and_norms_as_used(models):
    """The pieces of the last pass of layer 1, recomputed in 64 bits from the tensors that went into them."""
    m = models[0]
    h0 = m.embed[m.token.long()].clone()
    layer = m.layers[0]
    seen = {}
    _, _, calls = m._plan(1)
    for c in calls:  # the plans of layer 0, in order
        owner = getattr(c, "__self__", None)
        if isinstance(owner, qg.KV8Attention):
            seen.setdefault("attend", owner)
        if isinstance(owner, qg.NormGateResidual):
            seen.setdefault("norms", []).append(owner)
    first = calls.index(seen["attend"].run) if seen["attend"].run in calls else None
    m.kv_len += 1
    m._plan(1)[0].copy_(h0)
    for c in calls[:first + 1]:
        c()
    n = int(m.kv_len)
    kv = layer.cache.values().double().cpu().numpy()
    q = seen["attend"].keep[1].double().cpu().numpy()
    ref, _ = K.attention(kv, layer.cache.page_table.cpu().numpy(), E.PAGE, q, [n - 1], [1], E.HEAD_DIM ** -0.5, layer.window)
    out = seen["attend"].out.double().cpu().numpy()
    assert np.abs(out - ref).max() <= 2.2e-5 * np.abs(kv[1]).max()
    calls[first + 1]()  # o
    norm = seen["norms"][1]
    y, h, w_post, w_pre = (t.double().cpu().numpy() for t in norm.keep[:4])
    norm.run()
    hr, zr = K.norm(y, h, w_post, w_pre, None, 1.0, float(np.float32(1e-6)), 0.0)
    assert np.abs(norm.h_out.double().cpu().numpy() - hr).max() <= 2.0 ** -18 * np.abs(hr).max()
    assert np.abs(norm.z.double().cpu().numpy() - zr).max() <= 2.0 ** -18 * np.abs(zr).max()
    for c in calls[first + 3:]:
        c()
    m.pick(m._plan(1)[1][0])


def test_captured_step_is_the_eager_step(models):
    a, b = models
    for m in models:  # bring both to the same state
        m.kv_len.zero_()
        m.prefill(torch.arange(5, 25, device=m.device))
        m.step()
    assert torch.equal(a.logits, b.logits) and int(a.token) == int(b.token)
    graph = a.capture()
    picks = []
    for _ in range(6):
        graph.replay()
        b.step()
        picks.append((int(a.token), int(b.token)))
    assert all(x == y for x, y in picks)
    assert torch.equal(a.logits, b.logits) and int(a.kv_len) == int(b.kv_len) == 27
