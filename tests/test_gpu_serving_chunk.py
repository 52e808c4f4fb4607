"""Attention of chunks over the paged 4-bit cache (fsa_attention_chunk) against its 64-bit definition.

The tolerance, with eps/2 of a type as a rounding's largest relative error:
  - a score is a sum of D exact products in fp32, each addition off by at most 2^-23 (it may cut), so by
    (D + 8) 2^-23 of scale * sum |q||k|, and moves a weight by as much relatively, in the numerator
    and in the denominator: twice that of sum p|v| / sum p;
  - a probability is rounded to f16, 2^-11 of it (where V goes as bf16, E8M0 scales outside 2^-23 .. 2^13, to bf16, 2^-8):
    that of sum p|v| / sum p.  The largest carries at least 2^7, and below 2^-14 a step is 2^-24: half of that over 2^7,
    2^-32 of the largest |v|, a key; times 2 for sums that are reached by rescaling;
  - its exponential and the sums, 16 keys an addition, a rescaling a tile: (n / 16 + n / 128) 2^-23 + 2^-18 of the same;
  - q goes as f16, exact to 2^-18 of its row's maximum and off by at most 2^-29 of that below: 2^-29 max|q| sum|k| in a score,
    times scale; E2M1 blocks of a key below 2^-36 of its largest are off by at most 2^-37 of that, D 2^-37 <= 2^-30 as much together;
  - an output in bf16 is rounded by 2^-8 of it.
The log of the sums: the scores' error, and 2^-18."""
import math

import pytest

import serving_window_ref as win
from test_gpu_serving import _fsa, filled_cache, gen, i32, make_table, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def far_scales(v):
    """Whether a block of 32 may have an E8M0 scale (its maximum's power of two, less two) outside 2^-23 .. 2^13."""
    top = v.unflatten(-1, (-1, 32)).abs().amax(-1)
    return bool(((top < 2.0 ** -20) | (top >= 2.0 ** 14)).any())


def check(out, lse, q, seqs, q_lens, causal, scale, window, sinks, dtype, fmt):
    for b, (k, v, live) in enumerate(seqs):
        m, n, D = q_lens[b], k.shape[0], q.shape[-1]
        want, want_lse, spread, reach = win.attention(q[b, :m], k, v, live, causal, scale, window, sinks)
        score = (D + 8) * 2.0 ** -23 * reach
        if n:
            score = score + 1.5 * 2.0 ** -29 * abs(scale) * q[b, :m].double().abs().amax(-1) * float(k.abs().sum(-1).max())
        step = 2.0 ** -8 if fmt == "E2M1" and far_scales(v) else 2.0 ** -11
        tol = spread * (2 * score + step + (n / 16 + n / 128) * 2.0 ** -23 + 2.0 ** -18)[..., None]
        tol = tol + n * 2.0 ** -31 * (float(v.abs().max()) if n else 0)
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        got = out[b, :m].double()
        bad = ~((got - want).abs() <= tol)
        assert not bool(bad.any()), (b, int(bad.sum()), float(((got - want).abs() / tol.clamp(min=1e-30)).max()))
        if lse is not None:
            none = torch.isinf(want_lse)
            assert torch.equal(none, torch.isinf(lse[b, :m]))
            off = (lse[b, :m].double() - want_lse).abs()
            assert bool((off[~none] <= (score + 2.0 ** -18 * (1 + want_lse.abs()))[~none]).all())


def run(fsa, q, cache, table, lens, q_lens=None, causal=True, scale=None, window=None, sinks=0, dtype="f32", **kw):
    """One call, its rows checked, the others left as they were."""
    B, Sq, H, D = q.shape
    real = [Sq] * B if q_lens is None else q_lens
    out = torch.full((B, Sq, H, D), 7.0, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    lse = torch.full((B, Sq, H), 7.0, device="cuda")
    got = fsa.fsa_attention_chunk(q, cache, table, i32(lens), q_lens=None if q_lens is None else i32(q_lens), causal=causal,
                                  scale=scale, window=window, sinks=sinks, out=out, lse=lse, **kw)
    assert got is out
    for b, m in enumerate(real):
        assert bool((out[b, m:] == 7.0).all()) and bool((lse[b, m:] == 7.0).all())
    fmt = {v: k for k, v in fsa.FMT_BY_NAME.items()}[cache.fmt]
    seqs = win.sequences(cache, table, lens, cache.Hkv, D, fmt)
    check(out, lse, q, seqs, real, causal, D ** -0.5 if scale is None else scale, window or 0, sinks, dtype, fmt)
    return out, lse


# lengths, rows, heads, kv heads, page: one tile and block, their edges, several of each
SHAPES = [([1], 1, 1, 1, 16), ([77], 77, 4, 1, 16), ([128], 128, 1, 1, 64), ([129], 129, 1, 1, 64), ([127, 256], 64, 4, 2, 32),
          ([700], 65, 4, 1, 128), ([300, 5, 1000], 5, 7, 1, 16), ([513, 640], 300, 2, 2, 256), ([2000], 33, 8, 8, 64),
          ([4000, 17], 17, 24, 24, 32), ([1, 1024, 90], 90, 8, 2, 1024)]


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Sq,H,Hkv,page", SHAPES)
def test_shapes(fmt, D, lens, Sq, H, Hkv, page):
    fsa = _fsa()
    g = gen(len(lens) + Sq)
    cache, table, _, _ = filled_cache(fsa, g, lens, page, Hkv, D, fmt)
    q = normal(g, len(lens), Sq, H, D)
    run(fsa, q, cache, table, lens)
    run(fsa, q, cache, table, lens, causal=False, dtype="bf16")
    run(fsa, q, cache, table, lens, window=50, sinks=3, dtype="bf16")


@pytest.mark.parametrize("fmt,D", [("E2M1", 128), ("NVFP4", 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 130), (127, 0), (128, 1), (129, 4), (500, 16), (900, 700), (2 ** 31 - 1, 0), (5, 2 ** 31 - 1)])
def test_windows(fmt, D, window, sinks):
    fsa = _fsa()
    g = gen(window % 1000 + sinks % 1000)
    lens, q_lens = [1500, 40, 0, 700, 2100], [90, 40, 0, 300, 1]
    cache, table, _, _ = filled_cache(fsa, g, lens, 32, 2, D, fmt)
    q = normal(g, len(lens), 300, 6, D) * 3
    run(fsa, q, cache, table, lens, q_lens, window=window, sinks=sinks)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_ragged_rows(fmt, causal):
    """q_lens from none to more than there are tokens (rows before the first see nothing); strided q and out; a table far wider than
    the sequences; strong scores."""
    fsa = _fsa()
    g = gen(21)
    lens, q_lens, Hkv, D, Sq, H = [100, 640, 3, 0, 2500, 31], [40, 0, 4, 2, 200, 100], 2, 128, 200, 8
    cache, table, _, _ = filled_cache(fsa, g, lens, 32, Hkv, D, fmt)
    table = torch.nn.functional.pad(table, (0, 300), value=-1)
    qkv = normal(g, len(lens), Sq, H + 2 * Hkv, D) * 4
    out, _ = run(fsa, qkv[:, :, :H], cache, table, lens, q_lens, causal)
    strided = torch.full((len(lens), H, Sq, D), 7.0, device="cuda").transpose(1, 2)
    fsa.fsa_attention_chunk(qkv[:, :, :H], cache, table, i32(lens), q_lens=i32(q_lens), causal=causal, out=strided)
    assert torch.equal(strided, out)


def test_blocks_with_and_without_a_second_tile():
    """Many short segments a CTA, some of more than 128 rows and some of fewer, none among them."""
    fsa = _fsa()
    g = gen(29)
    lens = [300, 40, 700, 260, 33, 500, 129, 9] * 5
    q_lens = [130, 3, 65, 64, 0, 128, 60, 9] * 5
    for fmt, Hkv, causal in (("E2M1", 24, True), ("NVFP4", 8, False)):
        cache, table, _, _ = filled_cache(fsa, g, lens, 16, Hkv, 64, fmt)
        table = torch.nn.functional.pad(table, (0, 3), value=-1)
        run(fsa, normal(g, len(lens), 130, 2 * Hkv, 64), cache, table, lens, q_lens, causal)
        run(fsa, normal(g, len(lens), 130, 2 * Hkv, 64), cache, table[:, :32].contiguous(), [min(n, 512) for n in lens], q_lens, causal, dtype="bf16")


def test_long_keys_over_many_ctas():
    """Few rows over many keys: parts of a segment from all CTAs, joined; rows that see none of a part."""
    fsa = _fsa()
    g = gen(5)
    for fmt, D, Hkv in (("E2M1", 128, 1), ("NVFP4", 64, 2)):
        lens = [40000, 300]
        cache, table, _, _ = filled_cache(fsa, g, lens, 64, Hkv, D, fmt)
        q = normal(g, 2, 60, 4 * Hkv, D)
        run(fsa, q, cache, table, lens)
        run(fsa, q, cache, table, lens, window=20000, sinks=200, dtype="bf16")
        run(fsa, q * 30, cache, table, lens, [7, 60], dtype="bf16")


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_scales_and_ranges(fmt):
    """Scales of every sign; values and keys far from one, a rising maximum, strong first tokens."""
    fsa = _fsa()
    g = gen(31)
    n, Hkv, D = 1300, 2, 128
    for kind in range(5):
        k, v = normal(g, 1, n, Hkv, D), normal(g, 1, n, Hkv, D)
        if kind == 0:
            v = v * torch.exp2(torch.randint(-15, 16, (1, n, 1, 1), generator=g, device="cuda").float()).to(v.dtype)
        elif kind == 1:
            v[:, 500:], k = v[:, 500:] * 2.0 ** 24, k * 2.0 ** -20
        elif kind == 2:
            v.zero_()
        elif kind == 3:
            k = k * torch.linspace(0.1, 8.0, n, device="cuda")[None, :, None, None].to(k.dtype)
            v[:, 100:200] = v[:, 100:200] * 2.0 ** -30
        else:
            k[:, 0] = k[:, 0] * 2.0 ** 30
            k[:, 1:] = k[:, 1:] * 2.0 ** 20
            v[:, 0] = v[:, 0] * 2.0 ** -12
        table, pages = make_table(g, [n], 64)
        cache = fsa.empty_cache(pages, 64, Hkv, D, fmt)
        cache.pages.fill_(0xFF)
        fsa.fsa_cache_append(cache, k, v, table, i32([n]))
        q = normal(g, 1, 70, 8, D) * (3 if kind != 4 else 2.0 ** -22)
        for scale in (None, -0.05, 0.0, 1.0):
            run(fsa, q, cache, table, [n], scale=scale)


def test_ends_of_the_key_and_value_ranges():
    """E2M1 keys of 2^100 and of 2^-100, values of both in the same sequence, scales that bring the scores back to one; a key far
    beyond all others takes no bits from the rows that do not see it, nor does a key of zeros from any."""
    fsa = _fsa()
    g = gen(37)
    n, Hkv = 500, 2
    for D, power, scale in ((128, 41, 2.0 ** -45), (64, 100, 2.0 ** -103), (128, -60, 2.0 ** 56), (64, -100, 2.0 ** 98)):
        k, v = normal(g, 1, n, Hkv, D), normal(g, 1, n, Hkv, D)
        k = torch.sign(k) * torch.linspace(1.0, 6.0, n, device="cuda")[None, :, None, None].to(k.dtype)
        k[:, ::9] = 0.0
        v[:, 200:300], v[:, 300:] = v[:, 200:300] * 2.0 ** 98, v[:, 300:] * 2.0 ** -100
        table, pages = make_table(g, [n], 64)
        cache = fsa.empty_cache(pages, 64, Hkv, D, "E2M1")
        q = normal(g, 1, 70, 8, D)
        fsa.fsa_cache_append(cache, k * 2.0 ** power, v, table, i32([n]))
        run(fsa, q, cache, table, [n], scale=scale)
        run(fsa, q, cache, table, [n], scale=-scale, window=100, sinks=3)
    k = normal(g, 1, n, Hkv, D)
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    clean = fsa.fsa_attention_chunk(q, cache, table, i32([n]))
    k[0, n - 20, 0] = -2.0 ** 100                  # rows 50 .. of head 0's queries
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    out = fsa.fsa_attention_chunk(q, cache, table, i32([n]))
    assert torch.equal(out[0, :50], clean[0, :50]) and torch.equal(out[0, :, 4:], clean[0, :, 4:])


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("wide", [0, 40])      # columns of the table that no sequence reaches: its segments are shared, and joined
def test_nan_stays_with_its_rows(fmt, wide):
    """A token with a non-finite key or value makes the rows NaN that see it, and no others; so does a
    row of q; bytes of unused places (here NaN scales) count nothing."""
    fsa = _fsa()
    g = gen(41)
    n, Hkv, D, Sq = 400, 2, 128, 150
    k, v = normal(g, 1, n, Hkv, D), normal(g, 1, n, Hkv, D)
    table, pages = make_table(g, [n], 16)
    table = torch.nn.functional.pad(table, (0, wide), value=-1)
    cache = fsa.empty_cache(pages, 16, Hkv, D, fmt)
    cache.pages.fill_(0xFF)
    q = normal(g, 1, Sq, 8, D)
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    clean = fsa.fsa_attention_chunk(q, cache, table, i32([n]))
    assert bool(torch.isfinite(clean).all())
    v[0, n - 30, 0, 40] = math.nan                 # rows Sq - 30 .. of head 0's queries
    k[0, n - 100, 1, 7] = math.inf                 # rows Sq - 100 .. of head 1's
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    out = fsa.fsa_attention_chunk(q, cache, table, i32([n]))
    for h, first in ((0, Sq - 30), (1, Sq - 100)):
        part = slice(4 * h, 4 * h + 4)
        assert torch.equal(out[0, :first, part], clean[0, :first, part]) and bool(torch.isnan(out[0, first:, part]).all())
    out = fsa.fsa_attention_chunk(q, cache, table, i32([n]), window=20, sinks=0)
    nan = torch.isnan(out[0]).all(-1)
    assert torch.equal(nan, torch.isnan(out[0]).any(-1))
    row = torch.arange(Sq, device="cuda")
    assert torch.equal(nan[:, 0], (row >= Sq - 30) & (row < Sq - 10)) and torch.equal(nan[:, 4], (row >= Sq - 100) & (row < Sq - 80))
    q[0, 60, 3, 5], q[0, 61, 2, 9] = math.nan, -math.inf
    out = fsa.fsa_attention_chunk(q, cache, table, i32([n]))
    assert bool(torch.isnan(out[0, 60, 3]).all()) and bool(torch.isnan(out[0, 61, 2]).all()) and bool(torch.isfinite(out[0, 60, 2]).all())


def test_bad_pages_and_lengths():
    """Pages outside the pool are not seen and set the status; lengths are cut to the table and at 0."""
    fsa = _fsa()
    g = gen(43)
    lens, Hkv, D, fmt = [700, 300, 90], 2, 128, "NVFP4"
    cache, table, _, _ = filled_cache(fsa, g, lens, 16, Hkv, D, fmt)
    q, status = normal(g, 3, 80, 4, D), i32([0])
    run(fsa, q, cache, table, lens, status=status)
    assert int(status) == 0
    bad = table.clone()
    bad[0, 3], bad[0, 20], bad[1, :], bad[2, 5] = cache.pages.shape[0], -5, 1 << 30, -1
    run(fsa, q, cache, bad, lens, status=status)
    assert int(status) == fsa.FSA_ERR_INVALID_ARG
    wide = fsa.fsa_attention_chunk(q, cache, table[:, :10].contiguous(), i32([1 << 30, 300, 90]))
    assert torch.equal(wide, fsa.fsa_attention_chunk(q, cache, table[:, :10].contiguous(), i32([160, 160, 90])))
    none, lse = torch.full((3, 80, 4, D), 7.0, device="cuda"), torch.zeros(3, 80, 4, device="cuda")
    fsa.fsa_attention_chunk(q, cache, table, i32([-5, -(1 << 31), 0]), out=none, lse=lse)
    assert bool((none == 0).all()) and bool((lse == -math.inf).all())


def test_workspace_streams_and_graph():
    """A given workspace with any content, another stream, a captured call that follows the lengths, the same bits
    each time."""
    fsa = _fsa()
    g = gen(61)
    Hkv, D, H, Sq = 4, 128, 16, 70
    cache, table, _, _ = filled_cache(fsa, g, [900, 4000], 64, Hkv, D, "E2M1")
    q = normal(g, 2, Sq, H, D)
    lens, q_lens = i32([900, 4000]), i32([70, 33])
    first = fsa.fsa_attention_chunk(q, cache, table, lens, q_lens=q_lens)
    ws = torch.full((fsa.fsa_attention_chunk_workspace(cache, 2, H, Sq, table.shape[1]),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        assert torch.equal(first, fsa.fsa_attention_chunk(q, cache, table, lens, q_lens=q_lens, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fsa.fsa_attention_chunk(q, cache, table, lens, q_lens=q_lens, stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    out = torch.zeros(2, Sq, H, D, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fsa.fsa_attention_chunk(q, cache, table, lens, q_lens=q_lens, out=out, workspace=ws)
    for n, m in (([900, 4000], [70, 33]), ([1, 17], [1, 17]), ([0, 3999], [5, 70]), ([640, 64], [0, 64])):
        lens.copy_(i32(n))
        q_lens.copy_(i32(m))
        out.zero_()
        graph.replay()
        assert torch.equal(out, fsa.fsa_attention_chunk(q, cache, table, lens, q_lens=q_lens))


@pytest.mark.parametrize("fmt,D", [("NVFP4", 64), ("E2M1", 128)])
def test_the_same_bits_beside_other_traffic(fmt, D):
    """Many runs with cold caches and memory busy beside them, so that copies come late and out of turn."""
    fsa = _fsa()
    g = gen(83)
    lens = [9000, 700]
    cache, table, _, _ = filled_cache(fsa, g, lens, 64, 4, D, fmt)
    q, status = normal(g, 2, 150, 16, D), i32([0])
    first, _ = run(fsa, q, cache, table, lens, status=status)
    other, side = torch.zeros(32 << 20, device="cuda"), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, bad = torch.empty_like(first), torch.zeros(1, device="cuda")
    for i in range(400):
        if i % 4 == 0:
            with torch.cuda.stream(side):
                other.add_(1.0)
        fsa.fsa_attention_chunk(q, cache, table, i32(lens), out=out, status=status)
        bad += (out != first).any()
    torch.cuda.synchronize()
    assert int(bad) == 0 and int(status) == 0


def test_as_the_decode_call():
    """The same attention as fsa_attention_cache, to both calls' rounding (bf16 2^-8, f16 2^-10 of each weight)."""
    fsa = _fsa()
    g = gen(71)
    for fmt in ("E2M1", "NVFP4"):
        lens = [1200, 77]
        cache, table, _, v = filled_cache(fsa, g, lens, 16, 2, 64, fmt)
        q = normal(g, 2, 40, 8, 64)
        for kw in ({}, dict(causal=False), dict(window=100, sinks=2)):
            a = fsa.fsa_attention_chunk(q, cache, table, i32(lens), **kw)
            b = fsa.fsa_attention_cache(q, cache, table, i32(lens), **kw)
            assert float((a - b).abs().max()) <= 2 * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12) * float(v.abs().max())
