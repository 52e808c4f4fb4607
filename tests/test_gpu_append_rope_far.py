"""Keys turned by large angles on their way into the cache: values within the error of fsa_qk_norm_rope."""
import pytest

import serving_ref as ref
from test_gpu_serving import _fsa, gen, i32, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("power", [10, 22, 24, 40, 60, 90])
def test_frequencies_far_over_one(fmt, norm, power):
    """Frequencies of up to 2^90 and positions 0 and 1, keys of ordinary and of far sizes: every value between the roundings of
    the exact one less and plus the error of fsa_qk_norm_rope's arithmetic."""
    fsa = _fsa()
    g = gen(power)
    S, Hkv, D, half = 64, 16, 128, 64
    k = normal(g, 1, S, Hkv, D)
    k[0, 40:48] = k[0, 40:48] * 2.0 ** -100
    k[0, 48:56] = k[0, 48:56] * 2.0 ** 100
    freq = (torch.randint(1 << 20, 1 << 21, (half,), generator=g, device="cuda").double() * 2.0 ** (power - 21)).contiguous()
    pos = (torch.arange(S, device="cuda", dtype=torch.int32) % 2)[None].contiguous()
    cache = fsa.empty_cache(1, S, Hkv, D, fmt)
    fsa.fsa_cache_append_rope(cache, normal(g, 1, S, Hkv, D), k, k, i32([[0]]), i32([S]), pos=pos, inv_freq=freq, norm=norm)
    exact, size = ref.norm_rope(k, None, pos[..., None], freq, [half], norm, 1e-6, False)
    kc, ks, _, _ = (x[0] for x in ref.unpack_pages(cache.pages, S, Hkv, D, fmt))
    exact, size = exact[0], size[0]
    # fsa_qk_norm_rope's arithmetic is off by 2^-20 (|a| + |b|), its angles (positions 0 and 1: exact products) by 2^-47 of them too, in
    # all by at most 2 (|a| + |b|); 2^-140 for what lies below fp32's range
    off = min(2.0 ** -20 + float(freq.max()) * 2.0 ** -46, 2.0) * size.amax(-1, keepdim=True) + 2.0 ** -140
    got, s = ref.values(kc, ks, fmt).unflatten(-1, (-1, ref.BLOCK[fmt])), ref.scale_values(ks, fmt)[..., None]
    assert bool(torch.isfinite(got).all())
    mags = torch.tensor(ref.MAG, dtype=torch.float64, device="cuda")

    def nearest(x):                                     # the least and the largest rounding of x / scale, ties either way
        y = torch.where(s > 0, x.unflatten(-1, (-1, ref.BLOCK[fmt])) / s.clamp(min=2.0 ** -200), 0.0).clamp(-6.0, 6.0)
        d = (y.abs()[..., None] - mags).abs()
        near = d <= d.amin(-1, keepdim=True)
        least, most = torch.where(near, mags, 9.0).amin(-1), torch.where(near, mags, -1.0).amax(-1)
        return torch.where(y < 0, -most, least) * s, torch.where(y < 0, -least, most) * s

    bad = (got < nearest(exact - off)[0]) | (got > nearest(exact + off)[1])
    assert not bool(bad.any()), int(bad.sum())
    # a scale is that of a maximum within the error
    least, most = ref.quantise((exact.abs() - off).clamp(min=0.0), fmt)[1], ref.quantise(exact.abs() + off, fmt)[1]
    assert bool(((ks >= least) & (ks <= most)).all())


@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,half", [(128, 64), (64, 16), (128, 0)])
def test_weights_and_frequencies_that_are_not_finite(fmt, interleaved, D, half):
    """Blocks with an element that a weight or an angle makes NaN or infinite are NaN as a whole, and no others."""
    fsa = _fsa()
    g = gen(D + half)
    S, Hkv = 37, 3
    k = normal(g, 2, S, Hkv, D)
    k[:, ::5, :, 3] = 0.0                               # (0 times infinity)
    pos = (torch.arange(S, device="cuda", dtype=torch.int32) % 7)[None].repeat(2, 1).contiguous()
    inf, nan = float("inf"), float("nan")
    for at, what in ((3, nan), (3, inf), (D - 2, -inf), (None, nan), (None, inf)):
        w, freq = 1 + 0.2 * normal(g, D), None
        if half:
            freq = 1.0e4 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        if at is not None:
            w[at] = what
        elif half:
            freq[half // 2] = what
        else:
            continue
        for norm in (True, False):
            weight = w if norm else None
            if at is not None and not norm:
                continue
            cache = fsa.empty_cache(6, 16, Hkv, D, fmt)
            fsa.fsa_cache_append_rope(cache, normal(g, 2, S, Hkv, D), k, k, i32([[0, 1, 2], [3, 4, 5]]), i32([S, S]), pos=pos,
                                      inv_freq=freq, k_weight=weight, norm=norm, interleaved=interleaved)
            exact, _ = ref.norm_rope(k, weight, pos[..., None], freq, [half], norm, 1e-6, interleaved)
            codes, scales = ref.quantise(exact, fmt)
            kc, ks, _, _ = (x.unflatten(0, (2, 3)).flatten(1, 2)[:, :S] for x in ref.unpack_pages(cache.pages, 16, Hkv, D, fmt))
            assert bool((scales == (255 if fmt == "E2M1" else 0x7F)).any())
            assert torch.equal(ks, scales), (at, what, norm)
            assert torch.equal(ref.values(kc, ks, fmt).nan_to_num(1e9), ref.values(codes, scales, fmt).nan_to_num(1e9)), (at, what, norm)
