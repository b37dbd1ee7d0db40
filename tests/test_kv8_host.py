"""Host-only checks of the cache, attention and norm calls: bad arguments are refused with the documented
status before anything touches the GPU, and the test reference's own steps hold."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_weight_gemv_gb300 as qg
from quantized_weight_gemv_gb300 import build as qbuild
from tests import _kv8 as K

A, MIS = 0x10000, 0x10004  # stand-in addresses, never dereferenced on these paths
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qg.lib()


def cache(**kw):
    c = dict(k=A, v=A, k_scale=A, v_scale=A, page_table=A, format=0, n_pages=4, n_kv_heads=2, head_dim=64, page_size=32,
             scale_block=16, batch=2, max_pages=2)
    c.update(kw)
    return qg.KV8CacheStruct(**c)


def append_args(**kw):
    a = dict(k=A, v=A, q=A, q_out=A, cos=A, sin=A, positions=None, kv_len=A, cu_tokens=A, k_stride=128, v_stride=128,
             q_stride=256, q_out_stride=256, tokens=3, n_q_heads=4, dtype=0, rot_dim=64, rope_style=0, n_pos=100)
    a.update(kw)
    return qg.KV8AppendArgs(**a)


def attention_args(**kw):
    a = dict(q=A, out=A, lse=None, kv_len=A, cu_tokens=A, q_stride=256, out_stride=256, tokens=3, n_q_heads=4, dtype=0,
             window=0, scale=0.125, softcap=0.0)
    a.update(kw)
    return qg.KV8AttentionArgs(**a)


def norm_args(**kw):
    a = dict(y=A, h=A, gate=None, w_post=A, w_pre=A, h_out=A, z=A, y_stride=64, h_stride=64, gate_stride=0,
             h_out_stride=64, z_stride=64, rows=2, n=64, dtype=0, res_dtype=0, eps=1e-6, w_offset=0.0, res_scale=1.0)
    a.update(kw)
    return qg.NormArgs(**a)


BAD_CACHE = [
    (dict(format=2), -3), (dict(head_dim=96), -3), (dict(head_dim=512), -3), (dict(page_size=24), -3),
    (dict(page_size=8), -3), (dict(page_size=512), -3), (dict(scale_block=8), -3), (dict(scale_block=128), -3),
    (dict(scale_block=64), -1), (dict(n_pages=0), -1), (dict(n_kv_heads=0), -1), (dict(batch=0), -1),
    (dict(max_pages=0), -1), (dict(batch=4097, max_pages=1), -3), (dict(max_pages=1 << 30), -3), (dict(k=None), -1),
    (dict(v=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(page_table=None), -1),
    (dict(k=MIS), -2), (dict(v=MIS), -2),
]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_cache_refusals(lib, kw, status):
    c = cache(**kw)
    assert lib.kv8_rope_append(ctypes.byref(c), ctypes.byref(append_args()), 0, None) == status
    ws = lib.kv8_attention_workspace_bytes(64)
    assert lib.kv8_attention(ctypes.byref(c), ctypes.byref(attention_args()), P(A), ws, 0, None) == status


def test_values_refusals(lib):
    c = ctypes.byref(cache())
    assert lib.kv8_values(None, P(A), P(A), 0, None) == -1
    assert lib.kv8_values(c, None, None, 0, None) == -1
    assert lib.kv8_values(c, P(MIS), P(A), 0, None) == -2
    assert lib.kv8_values(c, P(A), P(MIS), 0, None) == -2


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), -3), (dict(tokens=-1), -1), (dict(cu_tokens=None), -1), (dict(kv_len=None), -1), (dict(sin=None), -1),
    (dict(q_out=None), -1), (dict(q=None), -1), (dict(n_q_heads=0), -1), (dict(rope_style=2), -3), (dict(rot_dim=12), -1),
    (dict(rot_dim=72), -1), (dict(rot_dim=-8), -1), (dict(n_pos=0), -1), (dict(cos=MIS), -2), (dict(k=None), -1),
    (dict(v=None), -1), (dict(k=MIS), -2), (dict(v=MIS), -2), (dict(q=MIS), -2), (dict(q_out=MIS), -2),
    (dict(k_stride=64), -1), (dict(v_stride=127), -1), (dict(k_stride=130), -2), (dict(q_stride=258), -2),
    (dict(q_out_stride=128), -1), (dict(dtype=1, k_stride=132), -2),
])
def test_append_refusals(lib, kw, status):
    assert lib.kv8_rope_append(ctypes.byref(cache()), ctypes.byref(append_args(**kw)), 0, None) == status
    assert lib.kv8_rope_append(None, ctypes.byref(append_args()), 0, None) == -1
    assert lib.kv8_rope_append(ctypes.byref(cache()), None, 0, None) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=-1), -3), (dict(tokens=-1), -1), (dict(cu_tokens=None), -1), (dict(kv_len=None), -1),
    (dict(n_q_heads=0), -1), (dict(n_q_heads=3), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(softcap=float("nan")), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(q=MIS), -2), (dict(out=MIS), -2),
    (dict(q_stride=192), -1), (dict(out_stride=257), -2),
])
def test_attention_refusals(lib, kw, status):
    ws = lib.kv8_attention_workspace_bytes(64)
    call = lambda a, w=P(A), n=ws: lib.kv8_attention(ctypes.byref(cache()), ctypes.byref(a), w, n, 0, None)  # noqa: E731
    assert call(attention_args(**kw)) == status
    assert call(attention_args(), None) == -4
    assert call(attention_args(), P(A), ws - 1) == -4
    assert call(attention_args(), P(MIS)) == -2


def test_empty_calls_touch_nothing(lib):
    ws = lib.kv8_attention_workspace_bytes(64)
    assert ws > 0 and lib.kv8_attention_workspace_bytes(80) == 0
    none = dict(tokens=0, kv_len=None)
    assert lib.kv8_rope_append(ctypes.byref(cache()), ctypes.byref(append_args(k=None, v=None, **none)), 0, None) == 0
    assert lib.kv8_attention(ctypes.byref(cache()), ctypes.byref(attention_args(q=None, **none)), None, 0, 0, None) == 0
    assert lib.rmsnorm_gate_residual(ctypes.byref(norm_args(rows=0)), 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), -3), (dict(res_dtype=1), -3), (dict(dtype=1, res_dtype=2), -3), (dict(rows=-1), -1), (dict(n=0), -1),
    (dict(n=32769, h_stride=40000), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(w_offset=float("inf")), -1), (dict(res_scale=float("nan")), -1), (dict(h=None), -1), (dict(z=None), -1),
    (dict(w_pre=None), -1), (dict(h_out=None, z=None, w_pre=None), -1), (dict(y=None), -1), (dict(y_stride=63), -1),
    (dict(h_stride=63), -1), (dict(z_stride=0), -1), (dict(h_out_stride=1), -1), (dict(gate=A, gate_stride=63), -1),
    (dict(h=0x10002), -2), (dict(z=0x10001), -2), (dict(dtype=2, y=0x10001), -2),
])
def test_norm_refusals(lib, kw, status):
    assert lib.rmsnorm_gate_residual(ctypes.byref(norm_args(**kw)), 0, None) == status
    assert lib.rmsnorm_gate_residual(None, 0, None) == -1


def test_binding_refuses_host_tensors(lib):
    z = torch.zeros
    with pytest.raises(ValueError):
        qg.KV8Cache(z(2, 1, 1, 16, 64, dtype=torch.int8), z(2, 1, 1, 1), z(1, 1, dtype=torch.int32))
    with pytest.raises(TypeError):
        qg.rmsnorm_gate_residual(z(4), z(4))
    with pytest.raises(ValueError):
        qg.rmsnorm_gate_residual(z(1, 4), z(1, 4), z(4), z(4))


def test_reference_codes_against_torch():
    """The tests' own quantiser: torch's conversion for e4m3 in range, round-half-even for int8."""
    x = np.concatenate([np.linspace(-448, 448, 20001), K.E4M3[:127], (K.E4M3[:126] + K.E4M3[1:127]) / 2]).astype(np.float32)
    assert np.array_equal(K.to_codes(x, "e4m3"), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert K.to_codes(np.float32([np.inf, -1e9, np.nan]), "e4m3").tolist() == [0x7e, 0xfe, 0]
    assert K.to_codes(np.float32([0.5, 1.5, -2.5, 200, -np.inf, np.nan]), "int8").view(np.int8).tolist() == [0, 2, -2, 127, -127, 0]


@pytest.mark.parametrize("style", ["half", "interleaved"])
def test_reference_rotation_keeps_lengths_and_relative_positions(style):
    rng = np.random.default_rng(0)
    cos, sin = K.tables(50, 32)
    a, b = rng.standard_normal((2, 64)).astype(np.float32)
    dots = []
    for i, j in ((3, 10), (20, 27), (42, 49)):
        x, y = K.rotate(a[None], cos[i:i + 1], sin[i:i + 1], style)[0], K.rotate(b[None], cos[j:j + 1], sin[j:j + 1], style)[0]
        assert abs(np.linalg.norm(x) - np.linalg.norm(a)) < 1e-5
        dots.append(x @ y)
    assert np.ptp(dots) < 1e-4


def test_reference_attention_against_a_dense_softmax():
    s = K.Scene(1, "int8", 1, 64, 16, 16, [0], [20]).fill()
    q, q64 = s.rows(1, torch.float32)
    out, lse = K.attention(s.values(), s.table, 16, q64, [0], [20], 0.125)
    at = np.arange(20)
    k, v = (s.values()[w, s.table[0, at // 16], 0, at % 16] for w in range(2))
    sc = np.where(np.tril(np.ones((20, 20), bool)), q64[:, 0] @ k.T * 0.125, -np.inf)
    e = np.exp(sc)
    assert np.allclose(out[:, 0], e / e.sum(1, keepdims=True) @ v, rtol=1e-12, atol=1e-12)
    assert np.allclose(lse[:, 0], np.log(e.sum(1)), rtol=1e-12)
