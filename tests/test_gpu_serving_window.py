"""fsa_attention_cache with a sliding window and first tokens that stay visible, against its 64-bit
definition.  Tolerances as derived in test_gpu_serving.py."""
import math

import pytest

import serving_window_ref as win
from test_gpu_serving import _fsa, filled_cache, gen, i32, make_table, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def run(fsa, q, cache, table, lens, window, sinks, q_lens=None, dtype="f32", scale=None, **kw):
    B, Sq, H, D = q.shape
    real = [Sq] * B if q_lens is None else q_lens
    out = torch.full((B, Sq, H, D), 7.0, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
    lse = torch.full((B, Sq, H), 7.0, device="cuda")
    fsa.fsa_attention_cache(q, cache, table, i32(lens), q_lens=None if q_lens is None else i32(q_lens), window=window, sinks=sinks,
                            scale=scale, out=out, lse=lse, **kw)
    fmt = {v: k for k, v in fsa.FMT_BY_NAME.items()}[cache.fmt]
    scale = D ** -0.5 if scale is None else scale
    for b, (k, v, live) in enumerate(win.sequences(cache, table, lens, cache.Hkv, D, fmt)):
        m, n = real[b], lens[b]
        assert bool((out[b, m:] == 7.0).all()) and bool((lse[b, m:] == 7.0).all())
        want, want_lse, spread, reach = win.attention(q[b, :m], k, v, live, True, scale, window, sinks)
        score = (D + 8) * 2.0 ** -24 * reach
        # f16 weights (twice rounded with E4M3 scales), the scores' error, sums; weights below f16's range
        step = 2.0 ** -10 + 2.0 ** -22 if fmt == "NVFP4" else 2.0 ** -11
        vtop = float(v.abs().max()) if n else 0.0
        tol = spread * (2 * score + step + 2.0 ** -18)[..., None] + n * 12 * 2.0 ** -33 * vtop * max(1.0, 2 * vtop / 5.5 if fmt == "NVFP4" else 1.0)
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        bad = ~((out[b, :m].double() - want).abs() <= tol)
        assert not bool(bad.any()), (b, int(bad.sum()))
        none = torch.isinf(want_lse)
        assert torch.equal(none, torch.isinf(lse[b, :m]))
        off = (lse[b, :m].double() - want_lse).abs()
        assert bool((off[~none] <= (score + 2.0 ** -18 * (1 + want_lse.abs()))[~none]).all())
    return out, lse


WINDOWS = [(1, 0), (1, 1), (31, 0), (32, 4), (33, 40), (64, 0), (100, 7), (700, 0), (900, 64), (3, 5000), (5000, 3), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("fmt,D", [("E2M1", 128), ("NVFP4", 128), ("E2M1", 64), ("NVFP4", 64)])
def test_windows(fmt, D, window, sinks):
    """Single rows and guessed tokens, lengths around the window's ends, tables short and wide."""
    fsa = _fsa()
    g = gen(window % 1000 + sinks % 1000)
    lens = [1, 0, 33, 700, 1501, 2100, window % 2000, window % 2000 + 1, (window + sinks) % 2000 + 2]
    cache, table, _, _ = filled_cache(fsa, g, lens, 16, 2, D, fmt)
    for Sq, G, kw in ((1, 4, {}), (1, 1, dict(dtype="bf16")), (5, 3, {}), (9, 2, dict(q_lens=[1, 0, 9, 4, 7, 9, 0, 1, 2]))):
        run(fsa, normal(g, len(lens), Sq, 2 * G, D) * 2, cache, table, lens, window, sinks, **kw)
    wide = torch.nn.functional.pad(table, (0, 4000), value=-1)
    run(fsa, normal(g, len(lens), 3, 8, D), cache, wide, lens, window, sinks)


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_only_the_window_is_read(fmt):
    """Pages that no row sees may be anything: outside the pool (no status), or full of NaN."""
    fsa = _fsa()
    g = gen(3)
    n, page, window, sinks = 5000, 64, 700, 70
    cache, table, _, _ = filled_cache(fsa, g, [n], page, 2, 128, fmt)
    for Sq in (1, 4):
        q = normal(g, 1, Sq, 8, 128)
        want = fsa.fsa_attention_cache(q, cache, table, i32([n]), window=window, sinks=sinks)
        holes, status = table.clone(), i32([0])
        first = (n - Sq + 1 - window) // page                    # the first page that some window reaches
        holes[0, 2:first] = -1
        assert torch.equal(want, fsa.fsa_attention_cache(q, cache, holes, i32([n]), window=window, sinks=sinks, status=status))
        assert int(status) == 0
        holes[0, 1] = 1 << 20                                    # holds first tokens
        fsa.fsa_attention_cache(q, cache, holes, i32([n]), window=window, sinks=sinks, status=status)
        assert int(status) == fsa.FSA_ERR_INVALID_ARG
        dirty = fsa.MxCache(cache.pages.clone(), page, 2, 128, fmt)
        dirty.pages[table[0, 2:first].long()] = 0xFF
        assert torch.equal(want, fsa.fsa_attention_cache(q, dirty, table, i32([n]), window=window, sinks=sinks))


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_what_leaves_the_window_takes_no_bits(fmt):
    """Values and keys, however large or not finite, count only in rows whose window or first tokens they are in."""
    fsa = _fsa()
    g = gen(17)
    n, Sq, window, sinks, H = 1200, 6, 200, 10, 4
    k, v = normal(g, 1, n, 1, 128), normal(g, 1, n, 1, 128)
    table, pages = make_table(g, [n], 16)
    cache = fsa.empty_cache(pages, 16, 1, 128, fmt)
    cache.pages.fill_(0xFF)
    q = normal(g, 1, Sq, H, 128)
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    clean, _ = run(fsa, q, cache, table, [n], window, sinks)
    for what in (2.0 ** 60, math.nan):
        for at, rows in ((n - Sq - window, []), (n - Sq - window + 1, [0]), (n - Sq - window + 3, [0, 1, 2]), (sinks, []), (sinks - 1, range(Sq)),
                         (n - 1, [Sq - 1])):
            v2 = v.clone()
            v2[0, at] *= what
            fsa.fsa_cache_append(cache, k, v2, table, i32([n]))
            out = fsa.fsa_attention_cache(q, cache, table, i32([n]), window=window, sinks=sinks)
            for i in range(Sq):
                if i in rows:
                    # (NVFP4 saturates at 6 * 448: 2688 times a weight of about one in 200 is well over 0.1)
                    big = torch.isnan(out[0, i]).all() if math.isnan(what) else ((out[0, i] - clean[0, i]).abs() > 0.1).any()
                    assert bool(big), (at, i)
                elif math.isnan(what):
                    assert bool(torch.isfinite(out[0, i]).all()), (at, i)
                else:
                    assert float((out[0, i] - clean[0, i]).abs().max()) <= 2.0 ** -9 * float(v.abs().max()), (at, i)


def test_workspace_and_graph():
    """A captured step whose lengths pass the window's ends; the workspace query for a short window in a wide table."""
    fsa = _fsa()
    g = gen(61)
    cache, table, _, _ = filled_cache(fsa, g, [900, 4000], 64, 4, 128, "E2M1")
    q, lens = normal(g, 2, 1, 16, 128), i32([900, 4000])
    width = table.shape[1]
    assert fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, width) > 0
    assert fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, width, window=500, sinks=4) == 0
    assert fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, width, window=64 * width) == fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, width)
    for window in (500, 2000):
        out = torch.zeros(2, 1, 16, 128, device="cuda")
        ws = torch.full((fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, width, window, 4),), 0xFF, dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fsa.fsa_attention_cache(q, cache, table, lens, window=window, sinks=4, out=out, workspace=ws)
        for n in ([900, 4000], [1, 17], [0, 3999], [640, 64]):
            lens.copy_(i32(n))
            graph.replay()
            assert torch.equal(out, fsa.fsa_attention_cache(q, cache, table, lens, window=window, sinks=4))
            run(fsa, q, cache, table, n, window, 4)
        lens.copy_(i32([900, 4000]))


def test_a_window_of_everything_is_the_plain_call():
    fsa = _fsa()
    g = gen(81)
    lens = [1900, 40]
    cache, table, _, _ = filled_cache(fsa, g, lens, 32, 2, 64, "NVFP4")
    q = normal(g, 2, 3, 8, 64)
    keys = table.shape[1] * 32
    want = fsa.fsa_attention_cache(q, cache, table, i32(lens))
    assert torch.equal(want, fsa.fsa_attention_cache(q, cache, table, i32(lens), window=keys))
    assert torch.equal(want, fsa.fsa_attention_cache(q, cache, table, i32(lens), window=1, sinks=keys))
