"""The serving operators against their 64-bit definitions: q/k norm and rotation, the
paged 4-bit cache written and read, attention over it.

Tolerances are derived, not fitted.  A rounding to a type is off by at most eps/2 of the
value: bf16 2^-8, f16 2^-11, fp32 2^-24 (torch.finfo(t).eps / 2).
  - norm and rotation: the fp32 arithmetic before the one rounding to bf16 is off by a few
    2^-24 of |a| + |b| of the pair, and the angle by 2^-24 of a turn (2^-21.3 rad), so by
    2^-20 (|a| + |b|) in all.
  - attention: each probability times its V scale is rounded to f16, 2^-11 of sum p|v| / sum p.
    E8M0 scales are powers of two, so that one rounding is all; an E4M3 scale has 4 significant
    bits, so its product with the rounded probability is rounded again:
    |f(f(p) s) - p s| <= ((1 + 2^-11)^2 - 1) p s = (2^-10 + 2^-22) p s;
    the fp32 scores are off by at most (D + 8) 2^-24 of sum |q||k| scale each way, which moves
    every weight by as much relatively, numerator and denominator; sums, exp2 and the rest
    2^-18; a probability below f16's range loses at most 2^-25 of 2^8-scaled ones (6 * 2^-33
    of the largest V block scale doubled) a key.  With E4M3 scales p itself is rounded as
    p 2^(8 - r), where r = 0 unless a scale is 8 or more, and 2^r is at most twice the largest
    scale s (s <= vtop / 5.5, as amax / 6 rounds to it): the loss of p is 2^-25 / 2^(8 - r), of
    the product 2^(r - 33) |v|, so the bound carries max(1, 2 vtop / 5.5).  bf16 output adds
    2^-8 of the value.
"""
import ctypes
import math

import pytest

import serving_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _fsa():
    import softmax_mx_block_gb300 as fsa
    return fsa


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def edge_values(g, *shape):
    """bf16 with ties of every block maximum, zeros of both signs, whole zero rows, tiny and
    huge values and strong channels."""
    x = torch.randn(*shape, generator=g, device="cuda")
    pick = torch.rand(*shape, generator=g, device="cuda")
    x = torch.where(pick < 0.2, torch.randint(-24, 25, shape, generator=g, device="cuda") / 4.0, x)
    x = torch.where((pick > 0.2) & (pick < 0.25), torch.zeros_like(x), x)
    x = torch.where((pick > 0.25) & (pick < 0.28), -torch.zeros_like(x), x)
    row = torch.rand(*shape[:-1], 1, generator=g, device="cuda")
    x = x * torch.where(row < 0.1, 1e-38, 1.0) * torch.where((row > 0.1) & (row < 0.2), 1e30, 1.0)
    x = x * torch.where((row > 0.2) & (row < 0.25), 0.0, 1.0) * torch.where((row > 0.25) & (row < 0.35), 1e-3, 1.0)
    return x.to(torch.bfloat16)


def make_table(g, lens, page, spare=2, extra=1):
    need = [-(-n // page) for n in lens]
    total = sum(need)
    order = torch.randperm(total + spare, generator=g, device="cuda")[:total].to(torch.int32).tolist()
    table = torch.full((len(lens), max(need + [1]) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), total + spare


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def filled_cache(fsa, g, lens, page, Hkv, D, fmt, make=normal, junk=0xFF):
    """A cache written by fsa_cache_append whose unused bytes are all `junk` (0xFF: NaN scales)."""
    table, pages = make_table(g, lens, page)
    cache = fsa.empty_cache(pages, page, Hkv, D, fmt)
    cache.pages.fill_(junk)
    S = max(lens + [1])
    k, v = make(g, len(lens), S, Hkv, D), make(g, len(lens), S, Hkv, D)
    fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(lens))
    return cache, table, k, v


# ------------------------------------------------------------------------ the cache itself
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page,Hkv,lens", [(16, 1, [1]), (16, 3, [17, 0, 40]), (64, 8, [5, 64, 65]), (256, 2, [300, 1])])
def test_append_writes_the_definition(fmt, D, page, Hkv, lens):
    """Codes and scales bit for bit, nothing else touched."""
    fsa = _fsa()
    g = gen(7)
    cache, table, k, v = filled_cache(fsa, g, lens, page, Hkv, D, fmt, edge_values, junk=0xA5)
    got = ref.unpack_pages(cache.pages, page, Hkv, D, fmt)
    want = [torch.full_like(x, 0x5 if i % 2 == 0 else 0xA5) for i, x in enumerate(got)]
    d = torch.arange(D, device="cuda")
    for i in (0, 2):
        want[i][:] = torch.where(d % 2 == 0, 0x5, 0xA).to(torch.uint8)
    for b, n in enumerate(lens):
        for s in range(n):
            page_id, at = int(table[b, s // page]), s % page
            for i, x in ((0, k), (2, v)):
                codes, scales = ref.quantise(x[b, s], fmt)
                want[i][page_id, at], want[i + 1][page_id, at] = codes, scales
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_append_matches_the_row_quantiser(fmt):
    """The same codes and scales as fsa_mx_quantize gives K rows (E2M1 nibbles, even element low)."""
    fsa = _fsa()
    B, S, Hkv, D, page = 1, 128, 2, 128, 64
    k = edge_values(gen(3), B, S, Hkv, D)
    cache = fsa.empty_cache(2, page, Hkv, D, fmt)
    table = i32([[0, 1]])
    fsa.fsa_cache_append(cache, k, k, table, i32([S]))
    m = fsa.fsa_mx_quantize(k.transpose(1, 2).contiguous(), fsa.FSA_MX_ROWS, fmt)
    rows = m.codes.reshape(Hkv, S, D // 2)
    codes = torch.stack((rows & 15, rows >> 4), dim=-1).flatten(-2).transpose(0, 1)
    kc, _, vc, _ = ref.unpack_pages(cache.pages, page, Hkv, D, fmt)
    assert torch.equal(kc.flatten(0, 1), codes) and torch.equal(vc.flatten(0, 1), codes)


def test_every_value_under_every_scale():
    """NVFP4 codes and scales of every finite bf16 value as a block's maximum, and of every
    significand under every scale (the divisions that the kernel does not do): as
    fsa_mx_quantize."""
    fsa = _fsa()
    bits = torch.arange(0x7F80, dtype=torch.int32, device="cuda")
    tops = (bits | (bits % 2 << 15)).to(torch.int16).view(torch.bfloat16)        # either sign
    g = gen(2)
    blocks = [tops[:, None].expand(-1, 16) * torch.rand(len(tops), 16, generator=g, device="cuda").to(torch.bfloat16)]
    blocks[0] = blocks[0].clone()
    blocks[0][:, 3] = tops
    # maxima 6 s for all scales s, with 15 values of every significand and exponent below it
    s = torch.tensor([ref.scale_values(torch.tensor([b], dtype=torch.uint8), "NVFP4").item() for b in range(1, 127)], device="cuda")
    sig = torch.arange(128, 256, device="cuda", dtype=torch.float64) / 128
    vals = (sig[None, :] * torch.exp2(torch.arange(-5, 3, device="cuda", dtype=torch.float64))[:, None]).flatten()   # x / s near 0.06 .. 8
    x = (s[:, None].double() * 1.0).log2().floor().exp2() * vals[None, :]
    x = torch.minimum(x, 6 * s[:, None].double()).reshape(len(s), -1)
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 15)).reshape(len(s), -1, 15)
    blocks.append(torch.cat(((6 * s)[:, None, None].expand(-1, x.shape[1], 1), x), dim=2).reshape(-1, 16).to(torch.bfloat16))
    flat = torch.cat([b.flatten() for b in blocks])
    n = -(-flat.numel() // (128 * 128)) * 128
    k = torch.nn.functional.pad(flat, (0, n * 128 - flat.numel())).reshape(1, n, 1, 128)
    cache = fsa.empty_cache(n // 128, 128, 1, 128, "NVFP4")
    table = torch.arange(n // 128, device="cuda", dtype=torch.int32)[None]
    fsa.fsa_cache_append(cache, k, k, table, i32([n]))
    m = fsa.fsa_mx_quantize(k.transpose(1, 2).contiguous(), fsa.FSA_MX_ROWS, "NVFP4")
    rows = m.codes.reshape(n, 64)
    codes = torch.stack((rows & 15, rows >> 4), dim=-1).flatten(-2)
    r, b = torch.arange(n, device="cuda")[:, None], torch.arange(8, device="cuda")[None]
    scales = m.scales.reshape(n // 128, 2, 512)[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4]
    kc, ks, vc, vs = ref.unpack_pages(cache.pages, 128, 1, 128, "NVFP4")
    for c, sc in ((kc, ks), (vc, vs)):
        assert torch.equal(sc.reshape(n, 8), scales) and torch.equal(c.reshape(n, 128), codes)


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_nonfinite_blocks(fmt):
    fsa = _fsa()
    D = 128
    k = normal(gen(1), 1, 4, 2, D)
    k[0, 1, 0, 5], k[0, 2, 1, 77], k[0, 3, 0, 127] = math.nan, math.inf, -math.inf
    cache = fsa.empty_cache(1, 16, 2, D, fmt)
    table = i32([[0]])
    fsa.fsa_cache_append(cache, k, k, table, i32([4]))
    for x, y in zip(fsa.fsa_cache_read(cache, table, i32([4]), 4), (k, k)):
        want = ref.rounded(y, fmt)
        assert torch.equal(torch.isnan(x), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(x.double()), torch.nan_to_num(want))
    assert int(torch.isnan(x).sum()) == 3 * ref.BLOCK[fmt]


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_in_steps_then_read(fmt, D):
    """A prompt, then chunks and single tokens, padded batches, strided sources (slices of a
    projection), destinations with heads first; rows outside stay as they were."""
    fsa = _fsa()
    g = gen(11)
    B, Hkv, page = 3, 2, 32
    total = [70, 33, 5]
    table, pages = make_table(g, total, page)
    cache = fsa.empty_cache(pages, page, Hkv, D, fmt)
    cache.pages.fill_(0xFF)
    lens = [0] * B
    kept = [[torch.zeros(0, Hkv, D, device="cuda")] * 2 for _ in range(B)]
    for S, new in ((40, [40, 20, 0]), (16, [16, 3, 4]), (1, [1, 1, 1]), (20, [13, 9, 0])):
        qkv = normal(g, B, S, 3 * Hkv, D)
        k, v = qkv[:, :, Hkv:2 * Hkv], qkv[:, :, 2 * Hkv:]
        lens = [a + n for a, n in zip(lens, new)]
        fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(new))
        for b in range(B):
            kept[b] = [torch.cat((a, x[b, :new[b]].float())) for a, x in zip(kept[b], (k, v))]
    assert lens == total
    S, start = 50, [3, -2, 0]
    base = torch.full((2, B, Hkv, S, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = base[0].transpose(1, 2), base[1].transpose(1, 2)
    fsa.fsa_cache_read(cache, table, i32(lens), start=i32(start), k_out=ko, v_out=vo)
    for b in range(B):
        for x, src in ((ko, kept[b][0]), (vo, kept[b][1])):
            want = torch.full((S, Hkv, D), 7.0, dtype=torch.float64, device="cuda")
            q = ref.rounded(src.to(torch.bfloat16), fmt)
            for i in range(S):
                if 0 <= start[b] + i < lens[b]:
                    want[i] = q[start[b] + i]
            assert torch.equal(x[b].double(), want)
    only = torch.zeros(B, 4, Hkv, D, dtype=torch.bfloat16, device="cuda")
    assert fsa.fsa_cache_read(cache, table, i32(lens), v_out=only)[0] is None
    assert torch.equal(only[0].double(), ref.rounded(kept[0][1][:4].to(torch.bfloat16), fmt))


def test_bad_pages_are_not_followed():
    """Negative and too large page numbers, lengths past the table: dropped or zero, and told."""
    fsa = _fsa()
    g = gen(5)
    Hkv, D, page = 2, 64, 16
    cache = fsa.empty_cache(3, page, Hkv, D, "E2M1")
    cache.pages.fill_(0xA5)
    table = i32([[1, 3], [-5, 0]])
    k = normal(g, 2, 40, Hkv, D)
    status = i32([0])
    fsa.fsa_cache_append(cache, k, k, table, i32([40, 32]), i32([40, 32]), status=status)
    assert int(status) == fsa.FSA_ERR_INVALID_ARG
    assert bool((cache.pages[2] == 0xA5).all())
    status.zero_()
    kb, vb = fsa.fsa_cache_read(cache, table, i32([40, 32]), 40, status=status)
    assert int(status) == fsa.FSA_ERR_INVALID_ARG
    want = torch.zeros(2, 40, Hkv, D, dtype=torch.float64, device="cuda")
    want[0, :16], want[1, 16:32] = ref.rounded(k[0, :16], "E2M1"), ref.rounded(k[1, 16:32], "E2M1")
    assert torch.equal(kb.double(), want) and torch.equal(vb.double(), want)
    # the attention does not see the keys of such pages
    q = normal(g, 2, 3, 4, D)
    status.zero_()
    out, lse = torch.empty(2, 3, 4, D, device="cuda"), torch.empty(2, 3, 4, device="cuda")
    fsa.fsa_attention_cache(q, cache, table, i32([32, 32]), out=out, lse=lse, status=status)
    assert int(status) == fsa.FSA_ERR_INVALID_ARG
    check_attention(q, cache, table, [32, 32], [3, 3], True, D ** -0.5, out, lse, torch.zeros_like(out))


def test_lengths_out_of_range():
    """Lengths and starts at the ends of int32 ask for nothing: nothing is read, written or
    attended (a row that sees nothing is zero), whatever the sum of the two would wrap to."""
    fsa = _fsa()
    g = gen(15)
    Hkv, D, page, S, top = 2, 128, 16, 5, 2 ** 31
    cache, table, k, v = filled_cache(fsa, g, [40], page, Hkv, D, "NVFP4", junk=0x11)
    before = cache.pages.clone()
    x = normal(g, 1, S, Hkv, D)
    for n, m in ((-top, S), (-1, S), (0, 0), (40, -top), (40, -1), (top - 1, S), (-top, top - 1)):
        fsa.fsa_cache_append(cache, x, x, table, i32([n]), i32([m]))
        if not (n == top - 1 or (n == 40 and m > 0)):
            assert torch.equal(cache.pages, before), (n, m)
    assert torch.equal(cache.pages, before)          # positions behind the table are dropped
    for n, start in ((-top, top - 1), (-top, 0), (0, -top), (40, top - 1), (-top + 3, top - 1), (-top + 9, top - 8), (40, -top)):
        base = torch.full((1, S, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda")
        fsa.fsa_cache_read(cache, table, i32([n]), start=i32([start]), k_out=base)
        assert bool((base == 5.0).all()), (n, start)
    q = normal(g, 1, 3, 4, D)
    for n, m in ((-top, 3), (-5, top - 1), (-top, -top), (top - 1, -1)):
        out = torch.full((1, 3, 4, D), 2.0, device="cuda")
        fsa.fsa_attention_cache(q, cache, table, i32([n]), q_lens=i32([m]), out=out)
        assert bool((out == (0.0 if m > 0 else 2.0)).all()), (n, m)


# ---------------------------------------------------------------------------- the attention
def check_attention(q, cache, table, lens, q_lens, causal, scale, out, lse, before):
    B, Sq, H, D = q.shape
    fmt = {2: "E2M1", 5: "NVFP4"}[cache.fmt]
    eps_out = 2.0 ** -8 if out.dtype == torch.bfloat16 else 2.0 ** -23
    for b in range(B):
        n = min(lens[b], table.shape[1] * cache.page_size)
        m = min(q_lens[b], Sq)
        assert torch.equal(out[b, m:], before[b, m:])
        if m <= 0:
            continue
        k, v, live = ref.sequence(cache.pages, table[b], n, cache.page_size, cache.Hkv, D, fmt)
        want, want_lse, spread, reach, total = ref.attention(q[b, :m], k, v, live, n, m, causal, scale)
        vtop = torch.nan_to_num(v[live]).abs().max() if n and bool(live.any()) else torch.zeros(())
        e_s = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -18
        round_p = 2.0 ** -11 if fmt == "E2M1" else 2.0 ** -10 + 2.0 ** -22
        tol = (round_p + 2 * e_s)[..., None] * spread * 1.01
        far = n * 12 * 2.0 ** -33 * vtop * ((vtop / 2.75).clamp(min=1.0) if fmt == "NVFP4" else 1.0)
        tol = tol + (far / total.clamp(min=1.0))[..., None] + eps_out * want.abs() + 1e-36
        got = out[b, :m].double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), b
        off = torch.nan_to_num((got - want).abs() - tol, nan=-1.0)
        assert bool((off <= 0).all()), (b, float(off.max()), float(want.abs().max()))
        if lse is not None:
            g_lse = lse[b, :m].double()
            assert torch.equal(torch.isinf(g_lse), torch.isinf(want_lse))
            fine = torch.isfinite(want_lse)
            assert bool(((g_lse - want_lse).abs()[fine] <= (e_s + 2.0 ** -22 * (want_lse.abs() + 20))[fine]).all())


def run_attention(fsa, q, cache, table, lens, q_lens=None, causal=True, scale=None, dtype="f32", seed=0, **kw):
    B, Sq, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    before = torch.full((B, Sq, H, D), 3.25, dtype=t, device="cuda")
    out, lse = before.clone(), torch.full((B, Sq, H), 9.0, device="cuda")
    fsa.fsa_attention_cache(q, cache, table, i32(lens), q_lens=None if q_lens is None else i32(q_lens), causal=causal,
                            scale=scale, out=out, lse=lse, **kw)
    check_attention(q, cache, table, lens, q_lens or [Sq] * B, causal, scale, out, lse, before)
    return out, lse


SHAPES = [
    # B-lens, Sq, H, Hkv, page
    ([1], 1, 1, 1, 16),
    ([0], 1, 8, 1, 16),
    ([0, 1, 15, 16, 17, 31, 32, 33], 1, 8, 2, 16),
    ([63, 64, 65, 127, 128, 129], 2, 4, 4, 64),
    ([1, 2, 3, 300], 5, 14, 2, 32),                 # rows before the first key, odd group
    ([2000], 1, 32, 8, 128),                        # few segments over many warps
    ([40000, 7], 1, 8, 1, 64),
    ([777] * 40, 1, 8, 4, 16),                      # many segments, shares that cross them
    ([5] * 700, 1, 2, 2, 16),                       # more segments than warps
    ([333, 90], 33, 6, 2, 1024),                    # several passes of columns
    ([1500], 70, 5, 5, 32),
]


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Sq,H,Hkv,page", SHAPES)
def test_attention_shapes(fmt, D, lens, Sq, H, Hkv, page):
    fsa = _fsa()
    g = gen(len(lens) + Sq)
    cache, table, _, _ = filled_cache(fsa, g, lens, page, Hkv, D, fmt)
    q = normal(g, len(lens), Sq, H, D)
    run_attention(fsa, q, cache, table, lens)
    run_attention(fsa, q, cache, table, lens, causal=False, dtype="bf16")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_attention_ragged_rows(fmt, causal):
    """q_lens from none to more than Sq; rows behind stay; strided q and out; strong scores."""
    fsa = _fsa()
    g = gen(21)
    lens, q_lens, Hkv, D, Sq, H = [100, 64, 3, 0, 2500, 31], [4, 0, 4, 2, 9, 1], 2, 128, 4, 8
    cache, table, _, _ = filled_cache(fsa, g, lens, 32, Hkv, D, fmt)
    qkv = normal(g, len(lens), Sq, H + 2 * Hkv, D) * 4
    out, _ = run_attention(fsa, qkv[:, :, :H], cache, table, lens, [min(x, Sq) for x in q_lens], causal)
    base = torch.full((len(lens), H, Sq, D), 3.25, device="cuda")
    strided = base.transpose(1, 2)
    fsa.fsa_attention_cache(qkv[:, :, :H], cache, table, i32(lens), q_lens=i32(q_lens), causal=causal, out=strided)
    assert torch.equal(strided, out)


def test_attention_values_with_range():
    """V blocks from 2^-30 to 2^20 times the others, whole zero V, a rising maximum, a sink."""
    fsa = _fsa()
    g = gen(31)
    n, Hkv, D = 3000, 2, 128
    for kind in range(5):
        k, v = normal(g, 1, n, Hkv, D), normal(g, 1, n, Hkv, D)
        if kind == 0:
            v = v * torch.exp2(torch.randint(-15, 16, (1, n, 1, 1), generator=g, device="cuda").float()).to(v.dtype)
        elif kind == 1:
            v[:, 1000:] = v[:, 1000:] * 2.0 ** 20
        elif kind == 2:
            v.zero_()
        elif kind == 3:
            k = k * torch.linspace(0.1, 8.0, n, device="cuda")[None, :, None, None].to(k.dtype)
            v[:, 100:200] = v[:, 100:200] * 2.0 ** -30
        else:
            k[:, 0] = k[:, 0] * 6
            v[:, 0] = v[:, 0] * 2.0 ** -12
        for fmt in ("E2M1", "NVFP4"):
            table, pages = make_table(g, [n], 64)
            cache = fsa.empty_cache(pages, 64, Hkv, D, fmt)
            cache.pages.fill_(0xFF)
            fsa.fsa_cache_append(cache, k, v, table, i32([n]))
            q = normal(g, 1, 2, 8, D) * 3
            run_attention(fsa, q, cache, table, [n])
            for scale in (-0.05, 0.0, 1.0):
                run_attention(fsa, q, cache, table, [n], scale=scale)


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_attention_nan_and_masks(fmt):
    """NaN keys and values reach the rows that see them and no others; NaN and Inf in q stay
    in their row."""
    fsa = _fsa()
    g = gen(41)
    n, Hkv, D, Sq = 200, 2, 128, 6
    k, v = normal(g, 1, n, Hkv, D), normal(g, 1, n, Hkv, D)
    v[0, n - 3, 0, 40] = math.nan                  # rows 3.. see it, in one block of V's dims
    v[0, 10, 1, 100] = math.inf                    # every row of head 1 sees it
    table, pages = make_table(g, [n], 16)
    cache = fsa.empty_cache(pages, 16, Hkv, D, fmt)
    cache.pages.fill_(0xFF)
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    q = normal(g, 1, Sq, 4, D)
    out, _ = run_attention(fsa, q, cache, table, [n])
    assert bool(torch.isfinite(out[0, :3, :2]).all()) and bool(torch.isnan(out[0, 3:, :2, 32:48]).all())
    q[0, 1, 0, 3], q[0, 2, 3, 9] = math.nan, math.inf
    out = fsa.fsa_attention_cache(q, cache, table, i32([n]))
    assert bool(torch.isnan(out[0, 1, 0]).all()) and bool(torch.isnan(out[0, 2, 3]).all())
    assert bool(torch.isfinite(out[0, 1, 1]).all()) and bool(torch.isfinite(out[0, 2, 0]).all())
    k[0, n - 2, 0, 0] = math.nan                   # a NaN key: rows 4 and 5 of head 0's queries
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    out = fsa.fsa_attention_cache(normal(g, 1, Sq, 4, D), cache, table, i32([n]))
    assert bool(torch.isnan(out[0, 4:, :2]).all()) and bool(torch.isfinite(out[0, :3, :2]).all())


def test_attention_far_pages():
    """A pool of over 4 GiB: pages whose byte offsets pass 32 bits."""
    fsa = _fsa()
    Hkv, D, page = 8, 128, 64
    per = fsa.fsa_cache_page_bytes(page, Hkv, D, "NVFP4")
    pages = (5 << 30) // per
    cache = fsa.empty_cache(pages, page, Hkv, D, "NVFP4")
    g = gen(51)
    lens = [130]
    table = i32([[pages - 1, 2, pages - 7]])
    k, v = normal(g, 1, 130, Hkv, D), normal(g, 1, 130, Hkv, D)
    fsa.fsa_cache_append(cache, k, v, table, i32(lens))
    kb, _ = fsa.fsa_cache_read(cache, table, i32(lens), 130)
    assert torch.equal(kb.double(), ref.rounded(k, "NVFP4"))
    small = fsa.MxCache(cache.pages[[pages - 1, 2, pages - 7]].contiguous(), page, Hkv, D, "NVFP4")
    q = normal(g, 1, 1, 32, D)
    out = fsa.fsa_attention_cache(q, cache, table, i32(lens))
    assert torch.equal(out, fsa.fsa_attention_cache(q, small, i32([[0, 1, 2]]), i32(lens)))
    run_attention(fsa, q, small, i32([[0, 1, 2]]), lens)


def test_attention_workspace_streams_and_graph():
    """A given workspace with any content, another stream, a captured call that follows the
    lengths and the cache, and the same bits each time."""
    fsa = _fsa()
    g = gen(61)
    Hkv, D, H = 4, 128, 16
    cache, table, _, _ = filled_cache(fsa, g, [900, 4000], 64, Hkv, D, "E2M1")
    q = normal(g, 2, 1, H, D)
    lens = i32([900, 4000])
    first = fsa.fsa_attention_cache(q, cache, table, lens)
    ws = torch.full((fsa.fsa_attention_cache_workspace(cache, 2, H, 1, table.shape[1]),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        assert torch.equal(first, fsa.fsa_attention_cache(q, cache, table, lens, workspace=ws))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fsa.fsa_attention_cache(q, cache, table, lens, stream=side)
    side.synchronize()
    assert torch.equal(first, other)
    out = torch.zeros(2, 1, H, D, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fsa.fsa_attention_cache(q, cache, table, lens, out=out, workspace=ws)
    for n in ([900, 4000], [1, 17], [0, 3999], [640, 64]):
        lens.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        check_attention(q, cache, table, n, [1, 1], True, D ** -0.5, out, None, out)


def test_calls_on_a_stream_of_their_own():
    """Outputs and workspace that a call makes for itself are made on its stream: a busy current
    stream does not write over them, nor they over its tensors."""
    fsa = _fsa()
    g = gen(65)
    Hkv, D, H = 4, 128, 16
    lens = [3000, 1999]
    cache, table, _, _ = filled_cache(fsa, g, lens, 64, Hkv, D, "E2M1")
    q, n, m = normal(g, 2, 3, H, D), i32(lens), i32([3, 1])
    want = fsa.fsa_attention_cache(q, cache, table, n, q_lens=m)
    back = fsa.fsa_cache_read(cache, table, n, 3000)
    turned = fsa.fsa_qk_norm_rope(q, q[:, :, :Hkv], None, None)
    side = torch.cuda.Stream()
    big = torch.ones(1 << 28, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        for _ in range(10):
            big.mul_(1.0)                          # about 3 ms of work
            torch.full((2, 3, H, D), 7.0, device="cuda")
            torch.full((2, 3000, Hkv, D), 7.0, device="cuda", dtype=torch.bfloat16)
            torch.full((1 << 23,), 7, device="cuda", dtype=torch.uint8)
        a = fsa.fsa_attention_cache(q, cache, table, n, q_lens=m, stream=side)
        b = fsa.fsa_cache_read(cache, table, n, 3000, stream=side)
        c = fsa.fsa_qk_norm_rope(q, q[:, :, :Hkv], None, None, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, want) and all(torch.equal(x, y) for x, y in zip(b + c, back + turned))


def test_tiny_and_large_scores():
    """q of every size that bf16 has, scales of many: the scores' factor neither vanishes nor
    overflows."""
    fsa = _fsa()
    g = gen(67)
    n, Hkv, D = 300, 1, 64
    for kexp in (-60, 0, 60):
        table, pages = make_table(g, [n], 16)
        cache = fsa.empty_cache(pages, 16, Hkv, D, "E2M1")
        cache.pages.fill_(0xFF)
        k = (torch.randn(1, n, Hkv, D, generator=g, device="cuda") * 2.0 ** kexp).to(torch.bfloat16)
        fsa.fsa_cache_append(cache, k, normal(g, 1, n, Hkv, D), table, i32([n]))
        for qexp in (-126, -60, 0, 60):
            q = (torch.randn(1, 2, 8, D, generator=g, device="cuda") * 2.0 ** qexp).to(torch.bfloat16)
            for scale in (2.0 ** -(kexp + qexp) if abs(kexp + qexp) < 99 else 1e30, 1e-12):
                if kexp + qexp + math.log2(scale) < 8:      # scores that softmax still tells apart in fp32
                    run_attention(fsa, q, cache, table, [n], scale=scale)


@pytest.mark.parametrize("seed", range(40))
def test_random_configurations(seed):
    """Seeded random shapes, lengths, formats, masks, strides and value ranges."""
    import random
    fsa = _fsa()
    r, g = random.Random(1000 + seed), gen(1000 + seed)
    D, fmt, page = r.choice((64, 128)), r.choice(("E2M1", "NVFP4")), r.choice((16, 32, 64, 128, 512))
    Hkv, G, Sq = r.choice((1, 2, 3, 8)), r.choice((1, 2, 4, 5, 7, 8, 16)), r.choice((1, 1, 2, 3, 5, 17))
    B, top = r.choice((1, 2, 5, 33, 150)), r.choice((3, 40, 500, 760, 3000))
    lens = [r.choice((0, 1, r.randint(0, top), r.randint(0, top), top)) for _ in range(B)]
    q_lens = [r.randint(0, Sq + 1) for _ in range(B)] if r.random() < 0.5 else None
    cache, table, _, _ = filled_cache(fsa, g, lens, page, Hkv, D, fmt, r.choice((normal, edge_values if top < 100 else normal)))
    wide = normal(g, B, Sq, Hkv * G + 2, D) * r.choice((0.1, 1.0, 5.0))
    run_attention(fsa, wide[:, :, 1:-1], cache, table, lens, q_lens, r.random() < 0.7, dtype=r.choice(("f32", "bf16")))


def test_two_calls_at_once():
    """Two captured calls with a workspace each, replayed on two streams together."""
    fsa = _fsa()
    g = gen(71)
    Hkv, D, H = 2, 64, 8
    made = []
    for n in ([3000, 5], [1200, 2500]):
        cache, table, _, _ = filled_cache(fsa, g, n, 16, Hkv, D, "NVFP4")
        q = normal(g, 2, 2, H, D)
        want = fsa.fsa_attention_cache(q, cache, table, i32(n))
        ws = torch.empty(fsa.fsa_attention_cache_workspace(cache, 2, H, 2, table.shape[1]), dtype=torch.uint8, device="cuda")
        out, lens = torch.zeros_like(want), i32(n)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fsa.fsa_attention_cache(q, cache, table, lens, out=out, workspace=ws)
        made.append((graph, out, want, torch.cuda.Stream(), (cache, table, q, ws, lens)))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, stream, _ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in made:
        assert torch.equal(out, want)


def test_append_of_the_longest_padding():
    """S at the end of its range, all but a few rows of it padding (a broadcast row): the count
    of the warps' units does not wrap."""
    fsa = _fsa()
    g = gen(33)
    cache, table, _, _ = filled_cache(fsa, g, [20], 16, 1, 64, "NVFP4", junk=0xA5)
    before = cache.pages.clone()
    row = normal(g, 1, 1, 1, 64)
    wide = row.expand(1, 2 ** 31 - 1, 1, 64)
    fsa.fsa_cache_append(cache, wide, wide, table, i32([12]), i32([0]))
    assert torch.equal(cache.pages, before)
    fsa.fsa_cache_append(cache, wide, wide, table, i32([12]), i32([3]))
    kb, vb = fsa.fsa_cache_read(cache, table, i32([12]), 3, start=i32([9]))
    want = ref.rounded(row, "NVFP4").expand(1, 3, 1, 64)
    assert torch.equal(kb.double(), want) and torch.equal(vb.double(), want)


def test_flags_without_a_truth_value():
    """What bool() raises for a flag is what the call raises."""
    fsa = _fsa()
    g = gen(4)
    cache, table, _, _ = filled_cache(fsa, g, [20], 16, 1, 64, "E2M1")
    q = normal(g, 1, 1, 1, 64)

    class Neither:
        def __bool__(self):
            raise ValueError("neither")

    for call in (lambda f: fsa.fsa_qk_norm_rope(q, q.clone(), None, None, norm=f),
                 lambda f: fsa.fsa_qk_norm_rope(q, q.clone(), None, None, interleaved=f),
                 lambda f: fsa.fsa_attention_cache(q, cache, table, i32([20]), causal=f)):
        with pytest.raises(ValueError, match="neither"):
            call(Neither())


def test_calls_refuse():
    """The binding's checks: devices, types, shapes, strides, buffers."""
    fsa = _fsa()
    g = gen(5)
    lens, Hkv, D, page = [40, 2500], 2, 64, 16
    cache, table, k, v = filled_cache(fsa, g, lens, page, Hkv, D, "E2M1")
    n, q = i32(lens), normal(g, 2, 3, 4, D)
    wide, host = torch.zeros(2, 3, 4, 2 * D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32)
    need = fsa.fsa_attention_cache_workspace(cache, 2, 4, 3, table.shape[1])
    assert need > 0
    pages = cache.pages

    def attn(q=q, c=cache, t=table, l=n, **kw):
        return lambda: fsa.fsa_attention_cache(q, c, t, l, **kw)

    bad = [attn(q=q.float()), attn(q=q[0]), attn(q=q.transpose(2, 3)), attn(q=q.cpu()), attn(q=normal(g, 2, 3, 3, D)),
           attn(q=normal(g, 2, 3, 4, 128)), attn(q=wide[..., 1:D + 1]), attn(q=torch.zeros(2, 3, 4, D + 4, device="cuda").bfloat16()[..., :D]),
           attn(t=table[:1]), attn(t=table.long()), attn(t=table.t()), attn(l=n[:1]), attn(l=n.long()), attn(l=host), attn(q_lens=host),
           attn(out=torch.zeros(2, 3, 4, D, device="cuda").half()), attn(out=torch.zeros(2, 3, 4, D)), attn(out=q[:, :2]),
           attn(out=torch.zeros(2, 3, 1, D, device="cuda").expand(2, 3, 4, D)), attn(out=q.float(), out_dtype="bf16"),
           attn(lse=torch.zeros(2, 4, 3, device="cuda")), attn(lse=torch.zeros(2, 3, 4, device="cuda").double()),
           attn(workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda")), attn(workspace=torch.zeros(need, dtype=torch.uint8)),
           attn(status=n), attn(timeout_ms=-1), attn(scale=float("nan")),
           attn(c=fsa.MxCache(pages[:, :-16], page, Hkv, D, "E2M1")), attn(c=fsa.MxCache(pages[::2], page, Hkv, D, "E2M1")),
           attn(c=fsa.MxCache(pages.view(torch.int8), page, Hkv, D, "E2M1")), attn(c=fsa.MxCache(pages, page, Hkv, D, "NVFP4")),
           attn(c=fsa.MxCache(pages, 24, Hkv, D, "E2M1")), attn(c=fsa.MxCache(pages.cpu(), page, Hkv, D, "E2M1")),
           lambda: fsa.fsa_cache_append(cache, k, v[:, :1], table, n), lambda: fsa.fsa_cache_append(cache, q, q, table, n),
           lambda: fsa.fsa_cache_append(cache, k.float(), v.float(), table, n), lambda: fsa.fsa_cache_append(cache, k, v, table, n, host),
           lambda: fsa.fsa_cache_read(cache, table, n), lambda: fsa.fsa_cache_read(cache, table, n, k_out=q),
           lambda: fsa.fsa_cache_read(cache, table, n, k_out=torch.empty_like(k), v_out=torch.empty_like(v[:, :1])),
           lambda: fsa.fsa_cache_read(cache, table, n, k_out=k[:, :1].expand_as(k)),
           lambda: fsa.fsa_qk_norm_rope(q, q[:1], None, None), lambda: fsa.fsa_qk_norm_rope(q, q, None, torch.ones(8, device="cuda").double()),
           lambda: fsa.fsa_qk_norm_rope(q, q, i32([[0] * 3] * 2), torch.ones(8, device="cuda")),
           lambda: fsa.fsa_qk_norm_rope(q, q, i32([[0] * 3] * 2), torch.ones(40, device="cuda").double()),
           lambda: fsa.fsa_qk_norm_rope(q, q, i32([[0] * 3] * 2), torch.ones(6, device="cuda").double()),
           lambda: fsa.fsa_qk_norm_rope(q, q, i32([[0] * 3] * 2), torch.ones(8, device="cuda").double(), sections=(4, 4)),
           lambda: fsa.fsa_qk_norm_rope(q, q, i32([[[0] * 2] * 3] * 2), torch.ones(8, device="cuda").double(), sections=(4, 5)),
           lambda: fsa.fsa_qk_norm_rope(q, q, i32([[[0] * 2] * 3] * 2), torch.ones(8, device="cuda").double()),
           lambda: fsa.fsa_qk_norm_rope(q, q, None, None, norm=False, q_weight=q[0, 0, 0]),
           lambda: fsa.fsa_qk_norm_rope(q, q, None, None, q_weight=q[0, 0, 0, :8]),
           lambda: fsa.fsa_qk_norm_rope(q, q, None, None, q_out=q[:, :1].expand_as(q))]
    for i, call in enumerate(bad):
        with pytest.raises(fsa.FsaError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: fsa.fsa_attention_cache(q, cache, None, n), lambda: fsa.fsa_cache_append(cache, k, None, table, n)):
        with pytest.raises(fsa.FsaError, match="tensor"):
            call()
    torch.cuda.synchronize()


def test_a_failed_launch_leaves_no_error_behind():
    """A launch that the runtime refuses (on the default stream, while one that waits for it is
    captured) is reported by the call, and not again to the runtime's next user."""
    fsa = _fsa()
    cache, table, k, v = filled_cache(fsa, gen(3), [20], 16, 1, 64, "E2M1")
    runtime = ctypes.CDLL("libcudart.so.13")
    stream, n, graph = ctypes.c_void_p(), i32([20]), ctypes.c_void_p()
    assert runtime.cudaStreamCreate(ctypes.byref(stream)) == 0
    torch.cuda.synchronize()
    assert runtime.cudaStreamBeginCapture(stream, 0) == 0
    try:
        with pytest.raises(fsa.FsaError) as e:
            fsa.fsa_cache_append(cache, k, v, table, n, stream=torch.cuda.default_stream())
        left = runtime.cudaPeekAtLastError()
    finally:
        runtime.cudaStreamEndCapture(stream, ctypes.byref(graph))     # it is void
        runtime.cudaGetLastError()
        runtime.cudaStreamDestroy(stream)
    assert e.value.status == fsa.FSA_ERR_LAUNCH and left == 0
    fsa.fsa_cache_append(cache, k, v, table, n)
    torch.cuda.synchronize()


# ------------------------------------------------------------------------ norm and rotation
ROPE = [
    # B, S, H, Hkv, D, rotary, sections, interleaved, norm, weights
    (1, 1, 1, 1, 64, 64, (32,), False, True, True),
    (2, 33, 5, 1, 128, 128, (64,), False, True, True),
    (2, 33, 5, 1, 128, 128, (64,), True, True, False),
    (1, 130, 14, 2, 64, 32, (16,), False, False, False),
    (3, 7, 4, 2, 128, 40, (9, 0, 11), True, True, True),
    (1, 2500, 8, 8, 128, 128, (22, 21, 21), True, True, True),
    (2, 2100, 4, 1, 128, 96, (40, 8), False, True, True),
    (1, 9, 3, 1, 128, 8, (4,), False, True, True),
    (2, 5, 2, 1, 64, 0, (0,), False, True, True),
]


@pytest.mark.parametrize("B,S,H,Hkv,D,rotary,sections,interleaved,norm,weights", ROPE)
def test_norm_rope(B, S, H, Hkv, D, rotary, sections, interleaved, norm, weights):
    fsa = _fsa()
    g = gen(S + D)
    qkv = normal(g, B, S, H + 2 * Hkv, D)
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    q[0, 0, 0] = 0.0
    half, axes = rotary // 2, len(sections)
    pos = torch.randint(-1000, 1 << 21, (B, S, axes), generator=g, device="cuda").to(torch.int32)
    inv = 1e5 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half)) if half else None
    wq, wk = (normal(g, D) if weights else None for _ in range(2))
    ko = torch.empty(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    qo, got_k = fsa.fsa_qk_norm_rope(q, k, pos if half else None, inv, sections=sections, q_weight=wq, k_weight=wk,
                                     norm=norm, eps=1e-5, interleaved=interleaved, k_out=ko.transpose(1, 2))
    for got, x, w in ((qo, q, wq), (got_k, k, wk)):
        want, size = ref.norm_rope(x, w, pos, inv, sections if half else (), norm, 1e-5, interleaved)
        assert bool(((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * size + 1e-36).all())
    fsa.fsa_qk_norm_rope(q, k, pos if half else None, inv, sections=sections, q_weight=wq, k_weight=wk, norm=norm,
                         eps=1e-5, interleaved=interleaved, q_out=q, k_out=k)          # in place
    assert torch.equal(q, qo) and torch.equal(k, got_k)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_infinities(interleaved):
    """Without the norm, Inf and NaN reach their own pair and nothing else; elements past the
    rotated ones are copied, the sign of zero with them."""
    fsa = _fsa()
    D, rotary = 128, 64
    q = normal(gen(9), 1, 3, 2, D)
    q[0, 0, 0, 5], q[0, 1, 1, 100], q[0, 2, 0, 70], q[0, 2, 1, 127] = math.inf, math.nan, -0.0, -math.inf
    inv = torch.linspace(1.0, 0.1, rotary // 2, device="cuda", dtype=torch.float64)
    out, _ = fsa.fsa_qk_norm_rope(q, q.clone(), i32([[3, 4, 5]]), inv, norm=False, interleaved=interleaved)
    got, was = out[..., rotary:].contiguous(), q[..., rotary:].contiguous()
    nan = torch.isnan(was)                          # a NaN stays one, its bits are not said
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got.view(torch.int16)[~nan], was.view(torch.int16)[~nan])
    odd = ~torch.isfinite(out[..., :rotary])
    want = torch.zeros_like(odd)
    want[0, 0, 0, [4, 5] if interleaved else [5, 5 + rotary // 2]] = True
    assert torch.equal(odd, want)


def test_norm_rope_positions():
    """The extremes of int32, and that a turn by position differs from its neighbours' as it should."""
    fsa = _fsa()
    D = 64
    q = torch.zeros(1, 6, 1, D, dtype=torch.bfloat16, device="cuda")
    q[..., : D // 2] = 1.0
    pos = i32([[0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31]])
    inv = torch.linspace(1.0, 1e-4, D // 2, device="cuda", dtype=torch.float64)
    out, _ = fsa.fsa_qk_norm_rope(q, q.clone(), pos, inv, norm=False)
    t = pos[0].double()[:, None] * inv
    want = torch.cat((torch.cos(t), torch.sin(t)), dim=-1)
    # 2^-16 of a turn at the ends of the range, 2^-24 within 2^24
    tol = torch.tensor([2.0 ** -20] * 4 + [2 * math.pi * 2.0 ** -16] * 2, device="cuda")[:, None]
    assert bool(((out[0, :, 0].double() - want).abs() <= 2.0 ** -8 * want.abs() + tol).all())


# ------------------------------------------------------------------------- a run of them all
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_prompt_then_steps(fmt):
    """A prompt and then single tokens, as a server runs them: prepare q and k, write k and v,
    attend.  The prompt's attention over the cache agrees with the prompt's own MX attention
    (fsa_attention_fwd_bf16) on the values read back, and each step with the definition."""
    fsa = _fsa()
    g = gen(81)
    B, H, Hkv, D, page, S = 2, 8, 2, 128, 64, 150
    inv = 1e4 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    w = [normal(g, D) * 0.1 + 1 for _ in range(2)]
    table, pages = make_table(g, [S + 8] * B, page)
    cache = fsa.empty_cache(pages, page, Hkv, D, fmt)
    n = 0
    for new in (S, 1, 1, 3):
        qkv = normal(g, B, new, H + 2 * Hkv, D)
        pos = (torch.arange(n, n + new, device="cuda", dtype=torch.int32)[None].expand(B, new)).contiguous()
        q, k = fsa.fsa_qk_norm_rope(qkv[:, :, :H], qkv[:, :, H:H + Hkv], pos, inv, q_weight=w[0], k_weight=w[1])
        n += new
        lens = i32([n] * B)
        fsa.fsa_cache_append(cache, k, qkv[:, :, H + Hkv:], table, lens)
        out, _ = run_attention(fsa, q, cache, table, [n] * B)
        if new == S:
            kb, vb = fsa.fsa_cache_read(cache, table, lens, n)
            heads = lambda x: x.transpose(1, 2).contiguous()  # noqa: E731
            vt = fsa.fsa_bf16_transpose_v(heads(vb))
            whole = fsa.fsa_attention_fwd_bf16(heads(q), heads(kb), vt, causal=True).transpose(1, 2)
            # the BF16 kernel rounds its probabilities to bf16: 2^-8 of sum p|v|, at most the largest |v|
            assert float((whole - out).abs().max()) <= (2.0 ** -8 + 2.0 ** -10) * float(vb.abs().max())
