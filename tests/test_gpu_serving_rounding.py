"""Both attention calls over the cache at the precision of their own roundings.

Tolerances as derived in test_gpu_serving.py (fsa_attention_cache) and test_gpu_serving_chunk.py (fsa_attention_chunk), but a
weight's rounding counts with the weight's own share of sum p|v| / sum p: by bf16, 2^-8, for the 32 keys of a kv head that
hold a V block with an E8M0 scale outside 2^-23 .. 2^13, by f16, 2^-11, for all others.  A block of zeros has no such scale."""
import pytest

import serving_window_ref as win
from test_gpu_serving import _fsa, gen, i32, make_table, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def far_keys(v):
    """[length, Hkv]: whether one of the key's 32 has a scale that is not exact in f16, from V's values [length, Hkv, D]."""
    top = v.unflatten(-1, (-1, 32)).abs().amax(-1)
    far = ((top > 0) & ((torch.frexp(top).exponent - 3 < -23) | (torch.frexp(top).exponent - 3 > 13))).any(-1)
    pad = torch.nn.functional.pad(far.T, (0, -len(far) % 32)).unflatten(-1, (-1, 32)).any(-1)
    return pad.repeat_interleave(32, dim=-1).T[:len(far)]


def expected(call, q, seq, causal, scale, window, sinks, fmt):
    """64-bit output of one sequence's rows, and how far `call` may be from it (fp32 output)."""
    k, v, live = seq
    n, D = k.shape[0], q.shape[-1]
    args = live, causal, scale, window, sinks
    want, _, spread, reach = win.attention(q, k, v, *args)
    top = float(v.abs().max())
    if call == "fsa_attention_chunk":
        score = (D + 8) * 2.0 ** -23 * reach + 1.5 * 2.0 ** -29 * abs(scale) * q.double().abs().amax(-1) * float(k.abs().sum(-1).max())
        step = torch.where(far_keys(v), 2.0 ** -8, 2.0 ** -11) if fmt == "E2M1" else torch.full(v.shape[:2], 2.0 ** -11, device=v.device)
        rounding = win.attention(q, k, v * step[..., None].double(), *args)[2]
        return want, rounding + spread * (2 * score + (n / 16 + n / 128) * 2.0 ** -23 + 2.0 ** -18)[..., None] + n * 2.0 ** -31 * top
    score = (D + 8) * 2.0 ** -24 * reach
    step = 2.0 ** -10 + 2.0 ** -22 if fmt == "NVFP4" else 2.0 ** -11
    least = n * 12 * 2.0 ** -33 * top * max(1.0, 2 * top / 5.5 if fmt == "NVFP4" else 1.0)
    return want, spread * (2 * score + step + 2.0 ** -18)[..., None] + least


def check(call, out, q, seq, fmt, causal=True, window=0, sinks=0):
    want, tol = expected(call, q, seq, causal, q.shape[-1] ** -0.5, window, sinks, fmt)
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), (call, float((off / tol.clamp(min=1e-30)).max()))


def cached(fsa, g, k, v, page, fmt):
    B, n, Hkv, D = k.shape
    table, pages = make_table(g, [n] * B, page)
    cache = fsa.empty_cache(pages, page, Hkv, D, fmt)
    cache.pages.fill_(0xFF)
    fsa.fsa_cache_append(cache, k, v, table, i32([n] * B))
    return cache, table


@pytest.mark.parametrize("D,dims", [(128, 96), (128, 80), (128, 32), (64, 32)])
@pytest.mark.parametrize("n,Sq", [(7, 7), (40, 40), (700, 80)])
def test_values_with_blocks_of_zeros(D, dims, n, Sq):
    """Heads padded with zeros, tokens without values among them: weights keep their f16 rounding."""
    fsa = _fsa()
    g = gen(n + dims)
    k, v = normal(g, 2, n, 2, D), normal(g, 2, n, 2, D)
    v[..., dims:] = 0.0
    v[:, 3::5] = 0.0
    cache, table = cached(fsa, g, k, v, 16, "E2M1")
    q = normal(g, 2, Sq, 32, D) * 0.25
    seqs = win.sequences(cache, table, [n, n], 2, D, "E2M1")
    for kw in ({}, dict(window=9, sinks=2), dict(causal=False)):
        out = fsa.fsa_attention_chunk(q, cache, table, i32([n, n]), **kw)
        for b in range(2):
            check("fsa_attention_chunk", out[b], q[b], seqs[b], "E2M1", **kw)
            assert bool((out[b, ..., -(-dims // 32) * 32:] == 0).all())


@pytest.mark.parametrize("call", ["fsa_attention_cache", "fsa_attention_chunk"])
@pytest.mark.parametrize("fmt,D", [("E2M1", 128), ("NVFP4", 128), ("E2M1", 64), ("NVFP4", 64)])
@pytest.mark.parametrize("n,Sq", [(12, 12), (150, 40), (1200, 40)])
def test_every_weight_by_its_own_rounding(call, fmt, D, n, Sq):
    """Values of ordinary size, and far ones in some keys: the others' weights are those of f16."""
    fsa = _fsa()
    g = gen(n + D)
    k, v = normal(g, 1, n, 2, D), normal(g, 1, n, 2, D)
    for far in (False, True):
        if far:
            v[:, n // 2 + 3] = v[:, n // 2 + 3] * 2.0 ** -26
            v[:, n // 4, 1] = v[:, n // 4, 1] * 2.0 ** -22
        cache, table = cached(fsa, g, k, v, 64, fmt)
        q = normal(g, 1, Sq, 8, D) * 0.5
        seq = win.sequences(cache, table, [n], 2, D, fmt)[0]
        for kw in ({}, dict(window=100, sinks=2), dict(causal=False)):
            out = getattr(fsa, call)(q, cache, table, i32([n]), **kw)
            check(call, out[0], q[0], seq, fmt, **kw)


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("kw", [{}, dict(window=150, sinks=4)])
def test_a_conversation_against_64_bits(fmt, kw):
    """Rows normalised, rotated, appended and attended in chunks and single tokens: each row against what its cache holds."""
    fsa = _fsa()
    g = gen(23)
    H, Hkv, D, total = 8, 2, 128, 500
    q, k, v = normal(g, 1, total, H, D), normal(g, 1, total, Hkv, D), normal(g, 1, total, Hkv, D)
    w, f = 1 + 0.2 * normal(g, D), 1.0e6 ** (-torch.arange(64, device="cuda", dtype=torch.float64) / 64)
    table, pages = make_table(g, [total], 32)
    cache = fsa.empty_cache(pages, 32, Hkv, D, fmt)
    cache.pages.fill_(0xFF)
    at = 0
    for n in (300, 1, 150, 40, *[1] * 9):
        part = slice(at, at + n)
        at += n
        r = fsa.fsa_cache_append_rope(cache, q[:, part], k[:, part], v[:, part], table, i32([at]), inv_freq=f, q_weight=w, k_weight=w)
        call = "fsa_attention_chunk" if n > 1 else "fsa_attention_cache"
        out = getattr(fsa, call)(r, cache, table, i32([at]), **kw)
        check(call, out[0], r[0], win.sequences(cache, table, [at], Hkv, D, fmt)[0], fmt, **kw)
    assert at == total


@pytest.mark.parametrize("D", [64, 128])
def test_a_block_below_the_least_scale_is_zeros(D):
    """Values all below 2^-124 count as zeros, whatever the scales beside them; the other blocks are as without them."""
    fsa = _fsa()
    g = gen(D)
    n, Sq = 200, 40
    k, v, q = normal(g, 1, n, 2, D), normal(g, 1, n, 2, D), normal(g, 1, Sq, 8, D)
    for far in (False, True):
        if far:
            v[:, ::32, :, :32] = v[:, ::32, :, :32] * 2.0 ** 40
        outs = []
        for tiny in (0.0, 2.0 ** -126):
            v[..., 32:64] = tiny
            cache, table = cached(fsa, gen(1), k, v, 64, "E2M1")
            outs.append(fsa.fsa_attention_chunk(q, cache, table, i32([n])))
        assert torch.equal(*outs) and bool((outs[1][..., 32:64] == 0).all())
