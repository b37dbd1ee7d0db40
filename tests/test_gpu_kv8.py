"""The 8-bit cache's append and the attention over it, on the GPU, against the plain forms of tests/_kv8.py."""
import numpy as np
import pytest
import torch

import quantized_weight_gemv_gb300 as qg
from tests import _kv8 as K
from tests._gpu import DEV

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from quantized_weight_gemv_gb300 import build
    build.build()
    assert torch.cuda.is_available()
    yield
    assert qg.device_error() == 0


# ---------------------------------------------------------------- append
def check_append(s, dtype, hq=0, rot=None, style="half", positions=False, calls=1, inputs=None):
    """Appends the scene's new tokens and compares codes and scales bit for bit; returns the device cache."""
    rot = s.d if rot is None else rot
    n_pos = max(f + n for f, n in zip(s.first, s.new)) + 7
    cos, sin = K.tables(n_pos, rot) if rot else (None, None)
    k, _ = s.rows(s.heads, dtype) if inputs is None else inputs[0]
    v, _ = s.rows(s.heads, dtype) if inputs is None else inputs[1]
    q, _ = s.rows(hq, dtype) if hq else (None, None)
    at = None
    if positions:
        at = s.rng.integers(0, n_pos, sum(s.new)).astype(np.int32)
    codes, scales = s.codes.copy(), s.scales.copy()
    K.append(codes, scales, s.table, s.fmt, s.block, k.float().numpy(), v.float().numpy(), s.first, s.new, cos, sin,
             at, style)
    c = s.device(qg)
    to = lambda a: None if a is None else torch.as_tensor(a).to(DEV)  # noqa: E731
    for _ in range(calls):
        out = qg.kv8_rope_append(c, to(k), to(v), s.kv_len(), s.cu(), to(cos), to(sin), to(at), style, to(q))
    got, got_s = c.codes.view(torch.uint8).cpu().numpy(), c.scales.cpu().numpy()
    assert np.array_equal(got_s.view(np.uint32), scales.view(np.uint32)), "scales"
    assert np.array_equal(got, codes), f"{(got != codes).sum()} codes differ"
    if hq:
        pos = np.concatenate([np.arange(f, f + n) for f, n in zip(s.first, s.new)]) if at is None else at
        ref = q.float().numpy()
        if rot:
            ref = K.rotate(ref, cos[pos][:, None], sin[pos][:, None], style)
        assert torch.equal(out.cpu(), torch.from_numpy(ref).to(dtype))
    s.codes, s.scales = codes, scales
    return c


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_ragged_batch_is_bit_exact(fmt, dtype, d):
    # starts and ends at, before and after block and page edges; a sequence without tokens
    s = K.Scene(d, fmt, 3, d, 32, 16, [0, 15, 16, 17, 31, 5, 0], [1, 1, 1, 40, 2, 0, 33])
    check_append(s, dtype, hq=6)


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("rot,d", [(0, 64), (8, 64), (32, 128), (64, 256), (256, 256)])
def test_append_rotations(style, rot, d):
    s = K.Scene(rot + 1, "int8", 2, d, 16, 16, [3, 60], [21, 1])
    check_append(s, F32, hq=4, rot=rot, style=style)
    s = K.Scene(rot + 2, "e4m3", 2, d, 16, 16, [3, 60], [21, 1])
    check_append(s, BF16, hq=2, rot=rot, style=style, positions=rot > 0)


@pytest.mark.parametrize("page,block", [(16, 16), (64, 16), (64, 32), (64, 64), (256, 64)])
@pytest.mark.parametrize("d", [64, 256])
def test_append_block_and_page_sizes(page, block, d):
    s = K.Scene(page + block, "int8", 2, d, page, block, [0, 7, 200], [150, 1, 70])
    check_append(s, F32)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_token_by_token_grows_scales(fmt):
    """One token at a time over two blocks, each louder or quieter than the last: scales only grow within a block."""
    s = K.Scene(5, fmt, 2, 64, 16, 16, [0, 9], [1, 1])
    for step in range(40):
        x = [s.rows(2, F32) for _ in range(2)]
        loud = np.float32(np.exp(s.rng.standard_normal() * 2))
        x = [(t * loud, None) for t, _ in x]
        if any(f // 16 >= s.table.shape[1] or s.table[b, f // 16] < 0 for b, f in enumerate(s.first)):  # a page is full
            s = K.Scene(6 + step, fmt, 2, 64, 16, 16, s.first, [1, 1])
        check_append(s, F32, inputs=x)
        s.first = [f + 1 for f in s.first]


def test_append_again_changes_nothing():
    s = K.Scene(11, "int8", 2, 128, 32, 32, [13, 40], [5, 30])
    check_append(s, F32, calls=3)


def test_append_after_rolled_back_tokens():
    """Rejected drafts: the lengths go back, their slots are overwritten, the scale they grew stays."""
    s = K.Scene(12, "int8", 2, 64, 16, 16, [3], [9])
    check_append(s, F32)
    s.first, s.new = [5], [4]
    check_append(s, F32)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_values_that_are_not_finite_or_zero(fmt):
    s = K.Scene(13, fmt, 1, 64, 16, 16, [0, 4, 16], [6, 3, 16])
    x = []
    for _ in range(2):
        t, _ = s.rows(1, F32)
        t[0, 0, 3], t[1, 0, 7], t[2, 0, 9] = np.inf, -np.inf, np.nan
        t[6:9] = 0.0                       # zeros behind tokens already there
        t[9:] = 0.0                        # a block of zeros but for one infinity
        t[12, 0, 5] = np.inf
        t[13] = 1e-44                      # a subnormal scale that underflows
        x.append((t, None))
    check_append(s, F32, rot=0, inputs=x)


def test_append_without_offsets_and_with_strides():
    """One token per sequence (no cu_tokens); k, v and q as slices of one fused projection's rows."""
    s = K.Scene(14, "int8", 2, 64, 16, 16, [0, 15, 16, 100], [1, 1, 1, 1])
    fused = torch.from_numpy(s.rng.standard_normal((4, 8, 64)).astype(np.float32)).to(DEV)
    q, k, v = fused[:, :4], fused[:, 4:6], fused[:, 6:]
    cos, sin = K.tables(128, 64)
    codes, scales = s.codes.copy(), s.scales.copy()
    f = fused.cpu().numpy()
    K.append(codes, scales, s.table, "int8", 16, f[:, 4:6], f[:, 6:], s.first, s.new, cos, sin)
    c = s.device(qg)
    out = qg.kv8_rope_append(c, k, v, s.kv_len(), None, torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV),
                             q=q, q_out=q)  # in place
    assert np.array_equal(c.codes.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(c.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    pos = np.array(s.first)
    assert np.array_equal(out.cpu().numpy(), K.rotate(f[:, :4], cos[pos][:, None], sin[pos][:, None], "half"))
    assert np.array_equal(fused[:, 4:].cpu().numpy(), f[:, 4:])


def test_append_many_sequences():
    """More sequences than a CTA has threads, some without tokens."""
    rng = np.random.default_rng(3)
    n = 700
    first, new = rng.integers(0, 40, n), rng.integers(0, 3, n)
    check_append(K.Scene(15, "int8", 1, 64, 16, 16, first, new), BF16, hq=1)


def test_append_skips_what_is_out_of_range():
    s = K.Scene(16, "int8", 1, 64, 16, 16, [4, 4, 4], [2, 2, 2])
    k, v = s.rows(1, F32)[0].to(DEV), s.rows(1, F32)[0].to(DEV)
    for case in ("page", "negative", "long"):
        c = s.device(qg)
        lens = s.kv_len()
        if case == "page":
            c.page_table[1, 0] = c.codes.shape[1] if case == "page" else 0
        elif case == "negative":
            lens[1] = 1  # fewer tokens than the call adds
        else:
            lens[1] = 1 << 20
        before = c.codes.view(torch.uint8).clone()
        qg.kv8_rope_append(c, k, v, lens, s.cu())
        assert qg.device_error() == 32
        codes, scales = s.codes.copy(), s.scales.copy()
        keep = [0, 1, 4, 5]
        K.append(codes, scales, s.table[[0, 2]], "int8", 16, k.cpu().numpy()[keep], v.cpu().numpy()[keep], [4, 4], [2, 2])
        assert np.array_equal(c.codes.view(torch.uint8).cpu().numpy(), codes), case
        assert not torch.equal(before, c.codes.view(torch.uint8))


# ---------------------------------------------------------------- attention
# Outputs are averages of values, so errors are measured against the largest |value| of the head.
# fp32 rows: a base-2 score x carries the rounding of its products' sum, of the query's two
# binary16 pieces (2^-22) and of the factors and 2^x itself, together below (|x| + 2) 2^-21 for
# head_dim <= 256; with |x| < 64 here a weight is off by less than 64 * 2^-21 * ln 2 = 2.1e-5 of
# itself, and the average by no more.  16-bit rows: the weight's rounding to binary16 (2^-11)
# and the output's (2^-9 of a bfloat16, 2^-11 of a binary16) come on top.
TOL = {F32: 2.2e-5, F16: 2.0 ** -10, BF16: 2.0 ** -8}


def check_attention(s, dtype, hq, window=0, softcap=0.0, scale=None, use_cu=True, gain=1.0, runs=1):
    scale = s.d ** -0.5 if scale is None else scale
    q, _ = s.rows(hq, dtype)
    q = (q * gain).to(dtype)
    kv = s.values()
    ref, ref_lse = K.attention(kv, s.table, s.page, q.double().numpy(), s.first, s.new, scale, window, softcap)
    c = s.device(qg)
    lse = torch.full(q.shape[:2], np.nan, device=DEV)
    out = torch.full(q.shape, np.nan, dtype=dtype, device=DEV)
    plan = qg.KV8Attention(c, q.to(DEV), s.kv_len(), s.cu() if use_cu else None, out=out, scale=scale, window=window,
                           softcap=softcap, lse=lse)
    got = plan.run().clone()
    for _ in range(runs - 1):
        assert torch.equal(plan.run(), got), "a second run differs"
    held = np.abs(np.where(np.isfinite(kv[1]), kv[1], 0.0))
    top = max(held[np.asarray(s.table[b])[np.arange(f + n) // s.page], :, np.arange(f + n) % s.page].max()
              for b, (f, n) in enumerate(zip(s.first, s.new)) if n)
    err = np.abs(got.double().cpu().numpy() - ref).max() / top
    assert np.isfinite(got.double().cpu().numpy()).all(), "outputs that are not finite"
    assert err <= TOL[dtype], f"error {err:.3e} of the largest value"
    el = np.abs(lse.cpu().double().numpy() - ref_lse).max()
    assert el <= 64 * 2.0 ** -21 * 2, f"log-sum-exp off by {el:.3e}"
    return err


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 2, 3, 8])
def test_attention_single_tokens(fmt, dtype, d, group):
    s = K.Scene(d + group, fmt, 2, d, 32, 16, [0, 1, 14, 15, 16, 126, 127, 128, 300], [1] * 9).fill()
    check_attention(s, dtype, 2 * group, use_cu=group != 1)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,group", [(64, 4), (128, 2), (256, 1), (256, 5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_several_tokens(fmt, d, group, dtype):
    # prompts, drafts and single tokens together; a sequence without tokens
    s = K.Scene(d, fmt, 2, d, 16, 16, [0, 0, 37, 100, 9, 255], [17, 1, 5, 3, 0, 33]).fill()
    check_attention(s, dtype, 2 * group)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1000])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_attention_windows(window, dtype):
    s = K.Scene(window, "e4m3", 2, 64, 16, 16, [0, 5, 150, 400], [3, 1, 20, 1]).fill()
    check_attention(s, dtype, 6, window=window)


def test_attention_window_leaves_freed_pages_alone():
    """Pages wholly behind the window have been given back: their ids are -1 and nothing reads them."""
    s = K.Scene(21, "e4m3", 1, 64, 16, 16, [200], [1]).fill()
    s.codes[:, s.table[0, :5]] = 0x7f
    kv = s.values()
    q, q64 = s.rows(2, F32)
    ref, _ = K.attention(kv, s.table, 16, q64, s.first, s.new, 0.125, 64)
    c = s.device(qg)
    c.page_table[0, :5] = -1
    out = qg.kv8_attention(c, q.to(DEV), s.kv_len(), None, window=64, scale=0.125)
    assert np.abs(out.cpu().double().numpy() - ref).max() <= TOL[F32] * np.nanmax(np.abs(kv[1][s.table[0, 8:]]))
    assert qg.device_error() == 0


@pytest.mark.parametrize("softcap", [0.5, 30.0])
def test_attention_softcap(softcap):
    s = K.Scene(22, "int8", 2, 128, 32, 32, [0, 77, 300], [4, 1, 1]).fill()
    check_attention(s, F32, 4, softcap=softcap, gain=3.0)


@pytest.mark.parametrize("d,group,dtype", [(64, 1, F32), (128, 4, BF16), (256, 8, F32), (256, 2, F16)])
def test_attention_long_and_split(d, group, dtype):
    """One sequence over many CTAs beside short ones: partials merged, in the same order every time."""
    s = K.Scene(23, "int8", 1, d, 64, 16, [5000, 3, 700], [1, 1, 2], quiet=True)
    check_attention(s, dtype, group, runs=4)


def test_attention_values_of_any_scale():
    """Scales that differ by many powers of two between blocks, and blocks of zeros."""
    s = K.Scene(24, "int8", 1, 64, 16, 16, [120], [1]).fill()
    ids = s.table[0]
    for j, e in enumerate((-40, 10, -3, 0, 12, -60, 5, 1)):
        s.scales[1, ids[j]] *= np.float32(2.0 ** e)
    s.scales[1, ids[3]] = 0.0
    check_attention(s, F32, 2)
    s.scales[1] *= np.float32(2.0 ** -90)
    check_attention(s, F32, 2)


def test_attention_scores_far_apart():
    """One token that takes all the weight, at the start, in the middle and at the end, after small ones."""
    for hot in (0, 70, 128):
        s = K.Scene(25 + hot, "int8", 1, 64, 16, 16, [128], [1]).fill()
        i, j = s.table[0, hot // 16], hot % 16
        s.codes[0, i, 0, j] = 127
        check_attention(s, F32, 2, gain=8.0, scale=0.02)


def test_attention_rows_with_nothing_to_see():
    """Positions before the sequence's start: zeros and a log-sum-exp of -inf, the other rows as ever."""
    s = K.Scene(26, "e4m3", 2, 64, 16, 16, [6, 10], [1, 3]).fill()
    q, q64 = s.rows(4, F32)
    c = s.device(qg)
    lens = s.kv_len()
    lens[1] = 2  # three tokens, two of them in the cache: the first sits at position -1
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


def test_attention_skips_what_is_out_of_range():
    s = K.Scene(27, "int8", 1, 64, 16, 16, [40, 40, 40], [1, 1, 1]).fill()
    q, q64 = s.rows(2, F32)
    kv = s.values()
    c = s.device(qg)
    c.page_table[1, 1] = 1 << 29  # tokens 16..31 of sequence 1 cannot be read
    out = qg.kv8_attention(c, q.to(DEV), s.kv_len()).cpu().double().numpy()
    assert qg.device_error() == 32
    ref, _ = K.attention(kv, s.table, 16, q64, s.first, s.new, 0.125)
    top = TOL[F32] * np.abs(kv[1][np.isfinite(kv[1])]).max()
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


def test_attention_queries_that_are_not_finite_stay_in_their_row():
    s = K.Scene(28, "int8", 1, 64, 16, 16, [40], [3]).fill()
    q, q64 = s.rows(4, F32)
    q[1, 2, 5] = np.nan
    q[2, 0, 5] = np.inf
    kv = s.values()
    ref, _ = K.attention(kv, s.table, 16, np.where(np.isfinite(q64), q64, 0), s.first, s.new, 0.125)
    out = qg.kv8_attention(s.device(qg), q.to(DEV), s.kv_len(), s.cu()).cpu().double().numpy()
    keep = np.ones((3, 4), bool)
    keep[1, 2] = keep[2, 0] = False
    assert np.isnan(out[1, 2]).all()
    assert np.abs((out - ref)[keep]).max() <= TOL[F32] * np.abs(kv[1][s.table[0, :3]])[np.isfinite(kv[1][s.table[0, :3]])].max()


def test_attention_zero_queries_average_the_values():
    """Equal scores: the output is the mean of the visible values."""
    s = K.Scene(29, "int8", 1, 128, 16, 16, [99], [1]).fill()
    q = torch.zeros(1, 2, 128, device=DEV)
    lse = torch.empty(1, 2, device=DEV)
    out = qg.kv8_attention(s.device(qg), q, s.kv_len(), lse=lse).cpu().double().numpy()
    at = np.arange(100)
    v = s.values()[1, s.table[0, at // 16], 0, at % 16]
    assert np.abs(out[0] - v.mean(0)).max() <= TOL[F32] * np.abs(v).max()
    assert np.abs(lse.cpu().numpy() - np.log(100)).max() <= 1e-5


def test_attention_strided_rows():
    s = K.Scene(30, "int8", 2, 64, 16, 16, [5, 50], [4, 4]).fill()
    wide = torch.from_numpy(s.rng.standard_normal((8, 12, 64)).astype(np.float32)).to(DEV)
    q = wide[:, 2:6]
    store = torch.full((8, 6, 64), 7.0, device=DEV)
    got = qg.kv8_attention(s.device(qg), q, s.kv_len(), s.cu(), out=store[:, 1:5])
    plain = qg.kv8_attention(s.device(qg), q.contiguous(), s.kv_len(), s.cu())
    assert torch.equal(got, plain)
    assert (store[:, 0] == 7).all() and (store[:, 5] == 7).all()


def test_append_then_attention_on_another_stream_and_in_a_graph():
    """A decode step as it is used: append and attention chained with programmatic dependent launch on a side
    stream and captured in a graph, the lengths and rows rewritten in place between replays."""
    s = K.Scene(31, "int8", 2, 128, 16, 16, [30, 3], [1, 1])
    cos, sin = K.tables(64, 128)
    c = s.device(qg)
    side = torch.cuda.Stream()
    rows = [torch.zeros(2, h, 128, device=DEV) for h in (2, 2, 4)]
    lens = s.kv_len()
    out = torch.empty(2, 4, 128, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = qg.KV8Append(c, rows[0], rows[1], lens, None, torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV),
                         q=rows[2], flags=qg.QG_FLAG_PDL)
        b = qg.KV8Attention(c, a.q_out, lens, out=out, flags=qg.QG_FLAG_PDL)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            a.run()
            b.run()
        for step in range(3):
            new = [s.rows(h, F32)[0] for h in (2, 2, 4)]
            for dst, src in zip(rows, new):
                dst.copy_(src)
            graph.replay()
            side.synchronize()
            K.append(s.codes, s.scales, s.table, "int8", 16, new[0].numpy(), new[1].numpy(), s.first, [1, 1], cos, sin)
            assert np.array_equal(c.codes.view(torch.uint8).cpu().numpy()[:, s.table[:, 0]], s.codes[:, s.table[:, 0]])
            q = K.rotate(new[2].numpy(), cos[s.first][:, None], sin[s.first][:, None], "half").astype(np.float64)
            kv = s.values()
            ref, _ = K.attention(kv, s.table, 16, q, s.first, [1, 1], 128 ** -0.5)
            assert np.abs(out.cpu().double().numpy() - ref).max() <= TOL[F32] * 20
            s.first = [s.first[0], s.first[1] + 1] if step else [s.first[0] + 1, s.first[1] + 1]
            if s.first[0] > 31:
                s.first[0] = 31
            lens.copy_(torch.tensor([f + 1 for f in s.first], dtype=torch.int32))


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB: the last pages are appended to and read."""
    pages, page, d = 270000, 64, 256
    codes = torch.empty((2, pages, 1, page, d), dtype=torch.int8, device=DEV)
    scales = torch.empty((2, pages, 1, page // 16), device=DEV)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device=DEV)
    c = qg.KV8Cache(codes, scales, table, 16)
    s = K.Scene(32, "int8", 1, d, page, 16, [0], [150], extra_pages=0)
    k, v, q = (s.rows(h, F32)[0] for h in (1, 1, 2))
    cu = s.cu()
    qg.kv8_rope_append(c, k.to(DEV), v.to(DEV), s.kv_len(), cu)
    K.append(s.codes, s.scales, s.table, "int8", 16, k.numpy(), v.numpy(), [0], [150])
    for j, i in enumerate((pages - 1, 3, pages - 2)):
        held = min(64, 150 - 64 * j)
        assert np.array_equal(codes[:, i, :, :held].view(torch.uint8).cpu().numpy(), s.codes[:, s.table[0, j], :, :held])
    out = qg.kv8_attention(c, q.to(DEV), s.kv_len(), cu).cpu().double().numpy()
    kv = s.values()
    ref, _ = K.attention(kv, s.table, page, q.double().numpy(), [0], [150], 1 / 16)
    assert np.abs(out - ref).max() <= TOL[F32] * 5
    del codes, scales, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("d,group", [(64, 8), (128, 2), (256, 2)])
def test_attention_prompts(dtype, d, group):
    """Whole prompts and long chunks behind a prefix: many row tiles."""
    s = K.Scene(33, "int8", 1, d, 32, 16, [0, 130, 0, 63], [193, 70, 16, 1]).fill()
    check_attention(s, dtype, group)
    s = K.Scene(34, "e4m3", 2, d, 64, 64, [257], [150]).fill()
    check_attention(s, dtype, 2 * group, window=90, softcap=20.0)


def test_empty_calls():
    s = K.Scene(35, "int8", 1, 64, 16, 16, [4, 4], [0, 0])
    c = s.device(qg)
    e = torch.empty(0, 1, 64, device=DEV)
    before = c.codes.clone()
    qg.kv8_rope_append(c, e, e, s.kv_len(), s.cu(), q=e)
    assert qg.kv8_attention(c, e, s.kv_len(), s.cu()).numel() == 0
    assert torch.equal(before, c.codes)
