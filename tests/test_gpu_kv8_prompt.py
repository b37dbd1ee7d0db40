"""The prompt form of the cache attention (64 or more query rows per kv head and sequence), at its edges.

64 query heads per kv head put single tokens on that path too, so every length, mask and
kind of content that the decode form meets is met here as well.
"""
import numpy as np
import pytest
import torch

import quantized_weight_gemv_gb300 as qg
from tests import _kv8 as K
from tests._gpu import DEV
from tests.test_gpu_kv8 import BF16, F16, F32, TOL, check_attention

pytestmark = pytest.mark.gpu

HQ = 64  # query heads over one kv head


@pytest.fixture(scope="module", autouse=True)
def _built():
    from quantized_weight_gemv_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert qg.device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_lengths(fmt, dtype, d):
    s = K.Scene(d, fmt, 1, d, 32, 16, [0, 1, 14, 15, 16, 62, 63, 64, 65, 126, 127, 128, 300], [1] * 13).fill()
    check_attention(s, dtype, HQ)
    check_attention(s, dtype, HQ, use_cu=False)


@pytest.mark.parametrize("d,group", [(64, 16), (128, 24), (256, 40)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ragged_row_tiles(d, group, dtype):
    """Row tiles that end inside a token's heads, sequences with none, one and many tokens."""
    s = K.Scene(d + group, "int8", 2, d, 16, 16, [0, 5, 9, 200, 31], [13, 0, 1, 7, 20]).fill()
    check_attention(s, dtype, 2 * group)


@pytest.mark.parametrize("window", [1, 15, 16, 64, 65, 1000])
def test_windows(window):
    s = K.Scene(window, "e4m3", 1, 64, 16, 16, [0, 5, 150, 400], [3, 1, 20, 1]).fill()
    check_attention(s, F32, HQ, window=window)


@pytest.mark.parametrize("d", [64, 256])
def test_softcap_and_negative_scale(d):
    s = K.Scene(41, "int8", 1, d, 32, 32, [0, 77, 300], [4, 1, 1]).fill()
    check_attention(s, F32, HQ, softcap=2.0, gain=2.0)
    check_attention(s, F32, HQ, scale=-0.05)
    check_attention(s, F32, HQ, softcap=2.0, scale=-0.05)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_few_rows_over_a_long_cache(d, dtype):
    """Token tiles shared out over the SMs and added up, the same every time; some shares find nothing to do."""
    s = K.Scene(42, "int8", 1, d, 64, 16, [5000], [2], quiet=True)
    check_attention(s, dtype, HQ, runs=4)
    s = K.Scene(43, "e4m3", 1, d, 64, 16, [70, 900], [3, 1], quiet=True)
    check_attention(s, dtype, HQ, runs=2)


def test_reference_moves_up_again_and_again():
    """Scores that grow along the sequence by far more than the slack, and fall."""
    for order in (1, -1):
        s = K.Scene(44, "int8", 1, 64, 16, 16, [639], [1]).fill()
        for j in range(40):
            s.scales[0, s.table[0, j]] = np.float32(0.002 * (1 + (j if order > 0 else 39 - j)))
        check_attention(s, F32, HQ, gain=2.0)


def test_values_of_any_scale():
    s = K.Scene(45, "int8", 1, 64, 16, 16, [120], [1]).fill()
    ids = s.table[0]
    for j, e in enumerate((-40, 10, -3, 0, 12, -60, 5, 1)):
        s.scales[1, ids[j]] *= np.float32(2.0 ** e)
    s.scales[1, ids[3]] = 0.0
    check_attention(s, F32, HQ)
    s.scales[1] *= np.float32(2.0 ** -90)
    check_attention(s, F32, HQ)


def test_freed_pages_behind_the_window():
    s = K.Scene(46, "e4m3", 1, 64, 16, 16, [200], [1]).fill()
    s.codes[:, s.table[0, :5]] = 0x7f
    kv = s.values()
    q, q64 = s.rows(HQ, F32)
    ref, _ = K.attention(kv, s.table, 16, q64, s.first, s.new, 0.125, 64)
    c = s.device(qg)
    c.page_table[0, :5] = -1
    out = qg.kv8_attention(c, q.to(DEV), s.kv_len(), None, window=64, scale=0.125)
    assert np.abs(out.cpu().double().numpy() - ref).max() <= TOL[F32] * np.nanmax(np.abs(kv[1][s.table[0, 8:]]))
    assert qg.device_error() == 0


def test_rows_with_nothing_to_see():
    s = K.Scene(47, "e4m3", 1, 64, 16, 16, [6, 10], [1, 3]).fill()
    q, q64 = s.rows(HQ, F32)
    c = s.device(qg)
    lens = s.kv_len()
    lens[1] = 2  # three tokens, two of them in the cache
    lse = torch.empty(q.shape[:2], device=DEV)
    out = qg.kv8_attention(c, q.to(DEV), lens, s.cu(), lse=lse).cpu().double().numpy()
    assert not out[1].any() and (lse[1] == -np.inf).all()
    kv = s.values()
    ref, _ = K.attention(kv, s.table, 16, q64[[0, 2, 3]], [6, 0], [1, 2], 0.125)
    top = max(np.abs(kv[1][s.table[0, 0]][:, :7]).max(), np.abs(kv[1][s.table[1, 0]][:, :2]).max())
    assert np.abs(out[[0, 2, 3]] - ref).max() <= TOL[F32] * top
    lens[1] = 0
    out = qg.kv8_attention(c, q.to(DEV), lens, s.cu())
    assert not out[1:].any() and torch.isfinite(out).all()
    assert qg.device_error() == 0


def test_skips_what_is_out_of_range():
    s = K.Scene(48, "e4m3", 1, 64, 16, 16, [40, 40, 40], [1, 1, 1]).fill()
    q, q64 = s.rows(HQ, F32)
    kv = s.values()
    c = s.device(qg)
    c.page_table[1, 1] = 1 << 29  # tokens 16..31 of sequence 1 cannot be read
    out = qg.kv8_attention(c, q.to(DEV), s.kv_len()).cpu().double().numpy()
    assert qg.device_error() == 32
    ref, _ = K.attention(kv, s.table, 16, q64, s.first, s.new, 0.125)
    top = TOL[F32] * np.nanmax(np.abs(kv[1][np.isfinite(kv[1])]))
    assert np.abs(out[[0, 2]] - ref[[0, 2]]).max() <= top
    at = np.r_[0:16, 32:41]
    ids = s.table[1][at // 16]
    sc = kv[0, ids, 0, at % 16] @ q64[1].T * 0.125
    e = np.exp(sc - sc.max(0))
    assert np.abs(out[1] - (e / e.sum(0)).T @ kv[1, ids, 0, at % 16]).max() <= top
    lens = s.kv_len()
    lens[2] = 1 << 28  # longer than the page table
    out = qg.kv8_attention(s.device(qg), q.to(DEV), lens).cpu().double().numpy()
    assert qg.device_error() == 32
    assert np.abs(out[:2] - ref[:2]).max() <= top and not out[2].any()


def test_queries_that_are_not_finite_stay_in_their_row():
    s = K.Scene(49, "int8", 1, 64, 16, 16, [40], [3]).fill()
    q, q64 = s.rows(HQ, F32)
    q[1, 2, 5] = np.nan
    q[2, 0, 5] = np.inf
    kv = s.values()
    ref, _ = K.attention(kv, s.table, 16, np.where(np.isfinite(q64), q64, 0), s.first, s.new, 0.125)
    out = qg.kv8_attention(s.device(qg), q.to(DEV), s.kv_len(), s.cu()).cpu().double().numpy()
    keep = np.ones((3, HQ), bool)
    keep[1, 2] = keep[2, 0] = False
    assert np.isnan(out[1, 2]).all()
    v = kv[1][s.table[0, :3]]
    assert np.abs((out - ref)[keep]).max() <= TOL[F32] * np.abs(v[np.isfinite(v)]).max()


def test_hidden_block_scales_do_not_matter():
    """Blocks that some rows of a tile see and others do not: a scale that is not finite stays with those who see it."""
    for hq, new in ((HQ, 40), (4, 3)):
        s = K.Scene(50, "int8", 1, 64, 16, 16, [30], [new]).fill()
        i, blk = s.table[0, 2], 0  # tokens 32.. are seen by the later rows only
        kv_ok = s.values()
        s.scales[1, i, 0, blk] = np.inf
        q, q64 = s.rows(hq, F32)
        ref, _ = K.attention(kv_ok, s.table, 16, q64, s.first, s.new, 0.125)
        out = qg.kv8_attention(s.device(qg), q.to(DEV), s.kv_len(), s.cu()).cpu().double().numpy()
        assert np.abs(out[:2] - ref[:2]).max() <= TOL[F32] * np.abs(kv_ok[1][s.table[0, :2]]).max()


def test_strided_rows():
    s = K.Scene(51, "int8", 1, 64, 16, 16, [5, 50], [4, 4]).fill()
    wide = torch.from_numpy(s.rng.standard_normal((8, HQ + 4, 64)).astype(np.float32)).to(DEV)
    q = wide[:, 2:HQ + 2]
    store = torch.full((8, HQ + 2, 64), 7.0, device=DEV)
    got = qg.kv8_attention(s.device(qg), q, s.kv_len(), s.cu(), out=store[:, 1:HQ + 1])
    plain = qg.kv8_attention(s.device(qg), q.contiguous(), s.kv_len(), s.cu())
    assert torch.equal(got, plain)
    assert (store[:, 0] == 7).all() and (store[:, HQ + 1] == 7).all()


def test_many_sequences():
    """More sequences than SMs, most of one token, on both forms."""
    rng = np.random.default_rng(5)
    first, new = rng.integers(0, 60, 300), rng.integers(0, 3, 300)
    s = K.Scene(52, "int8", 1, 64, 16, 16, first, new).fill()
    check_attention(s, BF16, 2)
    check_attention(s, BF16, HQ * 2)


def test_values_read_back():
    for fmt in ("int8", "e4m3"):
        s = K.Scene(53, fmt, 2, 128, 64, 32, [100], [1], quiet=True)
        got = s.device(qg).values().cpu().numpy()
        scale = np.repeat(s.scales, 32, -1)[..., None]
        assert np.array_equal(got, K.code_values(s.codes, fmt) * scale)
