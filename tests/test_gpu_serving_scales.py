"""The cache's scales and codes beside those of the framework's row quantiser."""
import pytest

import serving_ref as ref
from test_gpu_serving import _fsa, edge_values, gen, i32, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def scale_rows(scales, n, D, fmt):
    """Scale bytes [n, D/block] of a [1, 1, n, D] operand (128-row atoms of 4 scale columns)."""
    sb = D // ref.BLOCK[fmt]
    r, b = torch.arange(n, device="cuda")[:, None], torch.arange(sb, device="cuda")[None]
    return scales.reshape(-1, -(-sb // 4), 512)[r // 128, b // 4, r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


def both(fsa, k, fmt):
    """(codes, scales) of rows k [n, D] in the cache (as K, as V) and by fsa_mx_quantize."""
    n, D = k.shape
    cache = fsa.empty_cache(n // 128, 128, 1, D, fmt)
    x = k.reshape(1, n, 1, D)
    fsa.fsa_cache_append(cache, x, x, torch.arange(n // 128, device="cuda", dtype=torch.int32)[None], i32([n]))
    m = fsa.fsa_mx_quantize(k.reshape(1, 1, n, D), fsa.FSA_MX_ROWS, fmt)
    rows = m.codes.reshape(n, D // 2)
    codes = torch.stack((rows & 15, rows >> 4), dim=-1).flatten(-2)
    kc, ks, vc, vs = (x.reshape(n, -1) for x in ref.unpack_pages(cache.pages, 128, 1, D, fmt))
    return (kc, ks), (vc, vs), (codes, scale_rows(m.scales, n, D, fmt))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_scales_match_the_row_quantiser(fmt, D):
    fsa = _fsa()
    k = edge_values(gen(3), 1024, D)
    k[5, 7], k[70, 33], k[900, D - 1] = float("nan"), float("inf"), -float("inf")
    one, two, want = both(fsa, k, fmt)
    for got in (one, two):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_every_block_maximum():
    """E2M1: every finite bf16 magnitude as a block's maximum, beside values of all smaller
    sizes (ties among them), in either sign."""
    fsa = _fsa()
    g = gen(4)
    bits = torch.arange(0x7F80, dtype=torch.int32, device="cuda")
    tops = (bits | (bits % 2 << 15)).to(torch.int16).view(torch.bfloat16).double()
    steps = torch.tensor([0.125, 0.25, 0.375, 0.5, 0.625, 0.75, 0.875, 1.0], dtype=torch.float64, device="cuda")
    pick = steps[torch.randint(0, 8, (len(tops), 32), generator=g, device="cuda")]
    half = torch.rand(len(tops), 32, generator=g, device="cuda") < 0.5
    rest = torch.where(half, pick * torch.exp2(torch.floor(torch.log2(tops.abs().clamp(min=2.0 ** -133))))[:, None],
                       tops[:, None] * torch.rand(len(tops), 32, generator=g, device="cuda"))
    rest = torch.minimum(rest.abs(), tops.abs()[:, None]) * torch.where(torch.rand(len(tops), 32, generator=g, device="cuda") < 0.5, -1, 1)
    blocks = rest.to(torch.bfloat16)
    blocks[torch.arange(len(tops), device="cuda"), bits.long() % 32] = tops.to(torch.bfloat16)
    n = -(-blocks.numel() // (128 * 128)) * 128
    k = torch.nn.functional.pad(blocks.flatten(), (0, n * 128 - blocks.numel())).reshape(n, 128)
    one, two, want = both(fsa, k, "E2M1")
    for got in (one, two):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    codes, scales = ref.quantise(k, "E2M1")
    assert torch.equal(one[0], codes) and torch.equal(one[1], scales)
