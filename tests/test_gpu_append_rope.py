"""fsa_cache_append_rope: queries as fsa_qk_norm_rope makes them, values as fsa_cache_append does, and
keys whose codes and scales are those of the exact (64-bit) norm and rotation."""
import math

import pytest

import serving_ref as ref
from test_gpu_serving import _fsa, edge_values, gen, i32, make_table, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def frequencies(half, base=1.0e6):
    return base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(half, 1))


def run(fsa, q, k, v, lens, fmt, page, new_lens=None, pos=None, inv_freq=None, sections=None, q_weight=None, k_weight=None, norm=True,
        eps=1e-6, interleaved=False, near=0.0, table=None, **kw):
    """One call; all that it writes is checked, and that it writes nothing else.  near: the share of
    codes that may differ from those of the 64-bit form (rounded otherwise in its last bits)."""
    B, S, H, D = q.shape
    Hkv = k.shape[2]
    g = gen(1)
    own, pages = make_table(g, [max(n, 0) for n in lens], page)
    table = own if table is None else table
    cache = fsa.empty_cache(pages, page, Hkv, D, fmt)
    cache.pages.fill_(0xA5)
    fresh = [S] * B if new_lens is None else [min(max(n, 0), S) for n in new_lens]
    out = torch.full_like(q, 7.0)
    got = fsa.fsa_cache_append_rope(cache, q, k, v, table, i32(lens), None if new_lens is None else i32(new_lens), pos=pos, inv_freq=inv_freq,
                                    sections=sections, q_weight=q_weight, k_weight=k_weight, norm=norm, eps=eps, interleaved=interleaved,
                                    q_out=out, **kw)
    assert got is out
    first = torch.tensor([n - m for n, m in zip(lens, fresh)], dtype=torch.int32, device="cuda")
    at = pos if pos is not None else (first[:, None] + torch.arange(S, dtype=torch.int32, device="cuda")[None, :]).contiguous()
    want_q, _ = fsa.fsa_qk_norm_rope(q.contiguous(), k.contiguous(), at, inv_freq, sections=sections, q_weight=q_weight, k_weight=k_weight,
                                     norm=norm, eps=eps, interleaved=interleaved)
    other = fsa.empty_cache(pages, page, Hkv, D, fmt)        # v by fsa_cache_append
    other.pages.fill_(0xA5)
    fsa.fsa_cache_append(other, v, v, table, i32(lens), i32(fresh))
    half = 0 if inv_freq is None else inv_freq.numel()
    secs = sections or [half]
    at3 = at[:, :, None] if at.dim() == 2 else at
    exact, _ = ref.norm_rope(k, k_weight, at3, inv_freq, secs, norm, eps, interleaved)
    kc, ks, vc, vs = ref.unpack_pages(cache.pages, page, Hkv, D, fmt)
    okc, oks, ovc, ovs = ref.unpack_pages(other.pages, page, Hkv, D, fmt)
    assert torch.equal(vc, ovc) and torch.equal(vs, ovs)
    touched = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    wrong = total = 0
    for b in range(B):
        m = fresh[b]
        assert torch.equal(out[b, :m], want_q[b, :m]) and bool((out[b, m:] == 7.0).all())
        place = torch.arange(lens[b] - m, lens[b], device="cuda")
        ok = (place >= 0) & (place // page < table.shape[1])
        ids = table[b, (place // page).clamp(0, table.shape[1] - 1)].long()
        ok &= (ids >= 0) & (ids < pages)
        ids, inside = ids[ok], (place % page)[ok]
        touched[ids, inside] = True
        codes, scales = ref.quantise(exact[b, :m][ok], fmt)
        bad = (kc[ids, inside] != codes).any(-1) | (ks[ids, inside] != scales).any(-1)
        # (zeros may have either sign where a zero is a difference)
        same = (ref.values(kc[ids, inside], ks[ids, inside], fmt) == ref.values(codes, scales, fmt)) | torch.isnan(ref.values(codes, scales, fmt))
        wrong += int((bad & ~(same.all(-1) & (ks[ids, inside] == scales).all(-1))).sum())
        total += bad.numel()
    assert wrong <= near * total, (wrong, total)
    assert torch.equal(kc[~touched], okc[~touched]) and torch.equal(ks[~touched], oks[~touched])
    return cache, out


SHAPES = [([1], 1, 1, 1, 16), ([40, 17], 17, 4, 1, 16), ([100, 3, 64], 64, 32, 8, 64), ([300], 300, 14, 2, 32), ([9000, 5, 7], 5, 3, 3, 16),
          ([130] * 40, 1, 8, 8, 128)]


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,S,H,Hkv,page", SHAPES)
def test_shapes(fmt, D, lens, S, H, Hkv, page):
    """Lengths shorter than the call's rows (dropped tokens) among them; whole, half and odd rotations, pair by pair and by halves."""
    fsa = _fsa()
    g = gen(S + H)
    q, k, v = normal(g, len(lens), S, H, D), normal(g, len(lens), S, Hkv, D), normal(g, len(lens), S, Hkv, D)
    wq, wk = 1 + 0.2 * normal(g, D), 1 + 0.2 * normal(g, D)
    for half, inter in ((D // 2, False), (D // 4, True), (4, False), (20, False), (20, True), (D // 2, True)):
        run(fsa, q, k, v, lens, fmt, page, inv_freq=frequencies(half), q_weight=wq, k_weight=wk, interleaved=inter)
    run(fsa, q, k, v, lens, fmt, page, inv_freq=frequencies(D // 2), norm=False)
    run(fsa, q, k, v, lens, fmt, page, inv_freq=frequencies(D // 4), norm=False)
    run(fsa, q, k, v, lens, fmt, page, k_weight=wk)
    run(fsa, q, k, v, lens, fmt, page, norm=False)


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_many_keys_are_the_exact_ones(fmt):
    """Four million elements far into their sequences, some channels strong: every code and scale."""
    fsa = _fsa()
    g = gen(11)
    S, Hkv, D = 2048, 16, 128
    k, v = normal(g, 1, S, Hkv, D), normal(g, 1, S, Hkv, D)
    k[..., 5] *= 16
    k[..., 70] *= 300
    run(fsa, normal(g, 1, S, 16, D), k, v, [1 << 17], fmt, 1024, inv_freq=frequencies(64))
    pos = torch.randint(0, 1 << 24, (1, S), generator=g, device="cuda", dtype=torch.int32)
    run(fsa, normal(g, 1, S, 16, D), k, v, [S], fmt, 64, pos=pos, inv_freq=frequencies(64, 1.0e4), k_weight=1 + normal(g, D))


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("norm", [True, False])
def test_edge_values(fmt, norm):
    """Ties, zeros, whole zero rows, tiny and huge values; NaN and Inf; three axes; positions 0 and below."""
    fsa = _fsa()
    g = gen(13)
    S, Hkv, D = 200, 3, 128
    k, v = edge_values(g, 2, S, Hkv, D), edge_values(g, 2, S, Hkv, D)
    q = normal(g, 2, S, 6, D)
    run(fsa, q, k, v, [S, S], fmt, 16, inv_freq=frequencies(32), norm=norm)
    pos = torch.stack([torch.arange(S, dtype=torch.int32, device="cuda") % n for n in (200, 7, 3)], dim=1).expand(2, S, 3).contiguous()
    run(fsa, q, k, v, [S, S], fmt, 16, pos=pos, inv_freq=frequencies(64), sections=[24, 20, 20], norm=norm, interleaved=True)
    run(fsa, q, k, v, [S, S], fmt, 16, pos=-pos[..., 0].contiguous(), inv_freq=frequencies(64), norm=norm, eps=0.0 if norm else 1e-6)
    k[0, 3, 1, 40], k[1, 9, 0, 7] = math.nan, math.inf
    run(fsa, q, k, v, [S, S], fmt, 16, inv_freq=frequencies(16), norm=norm)


def test_padding_drops_and_bad_pages():
    """new_lens of all kinds, tokens at negative places and past the table, pages outside the pool, strided inputs, q in place."""
    fsa = _fsa()
    g = gen(17)
    lens, fresh, S, H, Hkv, D = [50, 3, 0, 64, 20, 33], [50, 9, 4, 0, -3, 200], 60, 8, 2, 128
    qkv = normal(g, len(lens), S, H + 2 * Hkv, D)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    for fmt in ("E2M1", "NVFP4"):
        run(fsa, q, k, v, lens, fmt, 16, new_lens=fresh, inv_freq=frequencies(64))
        table, pages = make_table(gen(1), [max(n, 0) for n in lens], 16)
        status = i32([0])
        run(fsa, q, k, v, lens, fmt, 16, new_lens=fresh, inv_freq=frequencies(64), table=table[:, :3].contiguous(), status=status)
        assert int(status) == 0
        bad = table.clone()
        bad[0, 1], bad[5, 0] = pages, -7
        run(fsa, q, k, v, lens, fmt, 16, new_lens=fresh, inv_freq=frequencies(64), table=bad, status=status)
        assert int(status) == fsa.FSA_ERR_INVALID_ARG
    cache = fsa.empty_cache(30, 16, Hkv, D, "E2M1")
    want = fsa.fsa_cache_append_rope(cache, q, k, v, table, i32(lens), i32(fresh), inv_freq=frequencies(64))
    kept = q.clone()
    fsa.fsa_cache_append_rope(cache, q, k, v, table, i32(lens), i32(fresh), inv_freq=frequencies(64), q_out=q)
    for b, m in enumerate(fresh):
        m = min(max(m, 0), S)
        assert torch.equal(q[b, :m], want[b, :m]) and torch.equal(q[b, m:], kept[b, m:])


def test_streams_and_graph():
    fsa = _fsa()
    g = gen(19)
    B, S, H, Hkv, D = 3, 1, 8, 2, 128
    q, k, v = normal(g, B, S, H, D), normal(g, B, S, Hkv, D), normal(g, B, S, Hkv, D)
    table, pages = make_table(g, [200] * B, 64)
    caches = [fsa.empty_cache(pages, 64, Hkv, D, "NVFP4") for _ in range(2)]
    for c in caches:
        c.pages.zero_()
    lens, out, f = i32([1, 2, 3]), torch.zeros(B, S, H, D, dtype=torch.bfloat16, device="cuda"), frequencies(64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fsa.fsa_cache_append_rope(caches[0], q, k, v, table, lens, inv_freq=f, q_out=out)
    side = torch.cuda.Stream()
    for n in ([1, 2, 3], [63, 64, 65], [200, 0, 128]):
        lens.copy_(i32(n))
        q.copy_(normal(g, B, S, H, D))
        k.copy_(normal(g, B, S, Hkv, D))
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        got = fsa.fsa_cache_append_rope(caches[1], q, k, v, table, lens, inv_freq=f, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, out) and torch.equal(caches[0].pages, caches[1].pages)


def test_a_conversation():
    """A prompt in chunks, then single tokens, rows normalised, rotated, appended and attended, with and without a window: as one pass
    over the whole conversation."""
    fsa = _fsa()
    g = gen(23)
    H, Hkv, D, page, total = 8, 2, 128, 32, 700
    q, k, v = normal(g, 1, total, H, D), normal(g, 1, total, Hkv, D), normal(g, 1, total, Hkv, D)
    wq, wk, f = 1 + 0.2 * normal(g, D), 1 + 0.2 * normal(g, D), frequencies(64)
    table, pages = make_table(g, [total], page)
    for fmt in ("E2M1", "NVFP4"):
        for kw in ({}, dict(window=150, sinks=4)):
            once, steps = (fsa.empty_cache(pages, page, Hkv, D, fmt) for _ in range(2))
            once.pages.zero_()
            steps.pages.zero_()
            rot = fsa.fsa_cache_append_rope(once, q, k, v, table, i32([total]), inv_freq=f, q_weight=wq, k_weight=wk)
            whole = fsa.fsa_attention_chunk(rot, once, table, i32([total]), **kw)
            at, got = 0, []
            for n in (300, 1, 257, 100, *[1] * 42):
                part = slice(at, at + n)
                at += n
                r = fsa.fsa_cache_append_rope(steps, q[:, part], k[:, part], v[:, part], table, i32([at]), inv_freq=f, q_weight=wq, k_weight=wk)
                call = fsa.fsa_attention_chunk if n > 1 else fsa.fsa_attention_cache
                got.append(call(r, steps, table, i32([at]), **kw))
            assert at == total and torch.equal(once.pages, steps.pages)
            off = (torch.cat(got, dim=1) - whole).abs().max()
            assert float(off) <= 2 * (2.0 ** -8 + 2.0 ** -10 + 2.0 ** -12) * float(v.abs().max())      # both calls' rounded weights
