"""The serving operators at the ends of what they accept: rows all of whose pages lie outside
the pool, scores near the ends of fp32 split over warps and CTAs, values near the ends of bf16,
the quantiser's scales.  Tolerances as derived in test_gpu_serving.py, or exact."""
import math

import pytest

import serving_ref as ref
from test_gpu_serving import _fsa, check_attention, edge_values, filled_cache, gen, i32, make_table, normal, run_attention

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def wide_table(table, width):
    """The table with -1 columns up to `width`: beyond 896 tokens the attention splits one list
    of tiles evenly over the CTAs, whatever the lengths."""
    return torch.nn.functional.pad(table, (0, max(0, width - table.shape[1])), value=-1)


# Lengths, kv heads and table widths (pages of 16) that end in each way of writing a row:
SPLITS = [
    pytest.param([20], 1, 4, id="one warp"),
    pytest.param([600], 2, 40, id="warps of a CTA, short table"),
    pytest.param([20, 9], 1, 100, id="one warp, list"),
    pytest.param([777] * 40, 8, 100, id="warps of a CTA, list"),
    pytest.param([5000], 1, 320, id="CTAs"),
    pytest.param([9000, 31, 4000], 2, 600, id="CTAs and warps"),
]


# ------------------------------------------------------------------- rows that see no key
@pytest.mark.parametrize("lens,Hkv,width", SPLITS)
@pytest.mark.parametrize("fmt,D,dtype", [("E2M1", 128, "f32"), ("NVFP4", 128, "bf16"), ("E2M1", 64, "bf16"), ("NVFP4", 64, "f32")])
def test_rows_all_of_whose_pages_are_outside(fmt, D, dtype, lens, Hkv, width):
    """Keys on pages outside the pool are not seen; a row that sees nothing else is zero, its
    lse -inf, however the keys are split.  Each other sequence as without them."""
    fsa = _fsa()
    g = gen(91)
    cache, table, _, _ = filled_cache(fsa, g, lens, 16, Hkv, D, fmt)
    table = wide_table(table, width)
    for which in (range(len(lens)), range(0, len(lens), 2)):
        for bad in (-1, cache.pages.shape[0]):
            t = table.clone()
            for b in which:
                t[b] = bad
            for Sq in (1, 3):
                q, status = normal(g, len(lens), Sq, 4 * Hkv, D), i32([0])
                out, lse = run_attention(fsa, q, cache, t, lens, causal=Sq == 1, dtype=dtype, status=status)
                assert int(status) == fsa.FSA_ERR_INVALID_ARG
                for b in which:
                    assert bool((out[b] == 0).all()) and bool((lse[b] == -math.inf).all())


@pytest.mark.parametrize("lens,Hkv,width", SPLITS)
def test_infinite_queries(lens, Hkv, width):
    """A row of q with an infinity has infinite scores: NaN, also where all of them are -inf;
    without a key it is zero all the same."""
    fsa = _fsa()
    g = gen(93)
    B, D, S = len(lens), 128, max(lens)
    table, pages = make_table(g, lens, 16)
    table = wide_table(table, width)
    cache = fsa.empty_cache(pages, 16, Hkv, D, "E2M1")
    k, v = normal(g, B, S, Hkv, D), normal(g, B, S, Hkv, D)
    k[..., 5] = 4.0
    fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(lens))
    q = normal(g, B, 2, 4 * Hkv, D)
    q[:, 0, 1, 5] = -math.inf
    q[:, 1, 2, 5] = math.inf
    out, lse = run_attention(fsa, q, cache, table, lens, causal=False)
    assert bool(torch.isnan(out[:, 0, 1]).all()) and bool(torch.isnan(out[:, 1, 2]).all()) and int(torch.isnan(lse).sum()) == 2 * B
    out, lse = run_attention(fsa, q, cache, torch.full_like(table, -1), lens, causal=False)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


# ---------------------------------------------------------------------------- far scores
@pytest.mark.parametrize("lens,Hkv,width", SPLITS)
@pytest.mark.parametrize("kind", ["scale", "keys", "high"])
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_far_scores_of_split_rows(fmt, kind, lens, Hkv, width):
    """All scores of a row equal and far below (or above) zero: the mean of V, however the keys
    are split.  Every weight is exactly 1, so the rounding of p times V's scale is all there is
    besides fp32 sums (2^-18)."""
    fsa = _fsa()
    if kind == "keys" and fmt == "NVFP4":
        pytest.skip("keys of 2^113 are beyond NVFP4's scales")
    g = gen(95)
    B, D, S, H = len(lens), 64, max(lens), 2 * Hkv
    table, pages = make_table(g, lens, 16)
    table = wide_table(table, width)
    cache = fsa.empty_cache(pages, 16, Hkv, D, fmt)
    k, v = torch.zeros(B, S, Hkv, D, dtype=torch.bfloat16, device="cuda"), normal(g, B, S, Hkv, D)
    k[..., 0] = 2.0 ** 113 if kind == "keys" else 4.0
    fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(lens))
    q = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0 if kind == "high" else -1.0
    scale = 1.0 if kind == "keys" else 1e30
    out, lse = torch.empty(B, 1, H, D, device="cuda"), torch.empty(B, 1, H, device="cuda")
    fsa.fsa_attention_cache(q, cache, table, i32(lens), scale=scale, out=out, lse=lse)
    score = float(q[0, 0, 0, 0]) * float(ref.rounded(k[0, 0, 0], fmt)[0]) * scale        # (NVFP4 keeps 4 as 4.125)
    for b, n in enumerate(lens):
        vq = ref.rounded(v[b, :n], fmt).repeat_interleave(2, dim=1)
        tol = (2.0 ** -10 + 2.0 ** -18) * vq.abs().mean(0)
        assert bool(((out[b, 0].double() - vq.mean(0)).abs() <= tol).all()), b
        assert bool(((lse[b, 0].double() / score - 1).abs() <= 2.0 ** -18).all())


def test_far_scores_beside_pages_outside():
    """Parts of a row without a key do not count in the join, wherever the others' scores lie."""
    fsa = _fsa()
    g = gen(97)
    n, D, page = 6000, 64, 16
    table, pages = make_table(g, [n], page)
    cache = fsa.empty_cache(pages, page, 1, D, "E2M1")
    k, v = torch.zeros(1, n, 1, D, dtype=torch.bfloat16, device="cuda"), normal(g, 1, n, 1, D)
    k[..., 0] = 4.0
    fsa.fsa_cache_append(cache, k, v, table, i32([n]))
    q = torch.zeros(1, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    for first, last in ((0, 3000), (3000, n), (16, n - 16), (0, n - 16)):
        t = table.clone()
        t[0, first // page:last // page] = -1
        live = torch.ones(n, dtype=torch.bool, device="cuda")
        live[first // page * page:last // page * page] = False
        vq = ref.rounded(v[0], "E2M1")[live]
        for sign, scale in ((-1.0, 1e30), (1.0, 1e30), (-1.0, 1e-30), (-1.0, 0.125)):
            q[..., 0] = sign
            out = fsa.fsa_attention_cache(q, cache, t, i32([n]), scale=scale)
            tol = (2.0 ** -10 + 2.0 ** -18) * vq.abs().mean(0)
            assert bool(((out[0, 0].double() - vq.mean(0)).abs() <= tol).all()), (first, last, sign, scale)


@pytest.mark.parametrize("lens,Hkv,width", SPLITS)
@pytest.mark.parametrize("scale", [0.6, 0.125, 1e-3])
def test_tiny_queries_huge_keys(scale, lens, Hkv, width):
    """q at the least normal bf16 number, keys at 2^115: the factor of the scores (below fp32's
    normal range) is the scale's."""
    fsa = _fsa()
    g = gen(99)
    B, D, S = len(lens), 128, max(lens)
    table, pages = make_table(g, lens, 16)
    table = wide_table(table, width)
    cache = fsa.empty_cache(pages, 16, Hkv, D, "E2M1")
    way = torch.where(torch.rand(B, S, Hkv, 1, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    k = (way * 2.0 ** 115).expand(B, S, Hkv, D).to(torch.bfloat16)
    v = (way + 0.25 * torch.randn(B, S, Hkv, D, generator=g, device="cuda")).to(torch.bfloat16)
    fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(lens))
    q = torch.full((B, 2, 4 * Hkv, D), 1.984375 * 2.0 ** -126, device="cuda").to(torch.bfloat16)
    q[:, 1] *= 2.0 ** -4
    run_attention(fsa, q, cache, table, lens, causal=False, scale=scale)


def test_queries_beyond_the_range_stay_alone():
    """Where scale times q leaves fp32 a row may be NaN; the rows beside it are not touched."""
    fsa = _fsa()
    g = gen(101)
    for lens, width in (([300], 20), ([5000], 320)):
        cache, table, _, _ = filled_cache(fsa, g, lens, 16, 1, 64, "E2M1")
        table = wide_table(table, width)
        q = normal(g, 1, 1, 8, 64) * 1e-30
        want = fsa.fsa_attention_cache(q, cache, table, i32(lens), scale=1e30)
        q[0, 0, 3] = q[0, 0, 3] * 1e30 * 1e30
        out = fsa.fsa_attention_cache(q, cache, table, i32(lens), scale=1e30)
        keep = torch.arange(8, device="cuda") != 3
        assert torch.equal(out[:, :, keep], want[:, :, keep]) and bool(torch.isfinite(want).all())


# ---------------------------------------------------------------------------- far values
@pytest.mark.parametrize("top", [90, 100, 120, 127])
@pytest.mark.parametrize("lens,width", [([600], 40), ([20000], 1300)])
def test_huge_values_beside_small_weights(lens, width, top):
    """One key of weight 1, all others of 2^-15 or so, V at 2^top: the small weights count in the
    sum and in the product."""
    fsa = _fsa()
    g = gen(103)
    n, D, Hkv = lens[0], 128, 2
    table, pages = make_table(g, lens, 16)
    table = wide_table(table, width)
    cache = fsa.empty_cache(pages, 16, Hkv, D, "E2M1")
    k = torch.zeros(1, n, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = (-torch.rand(1, n, Hkv, D, generator=g, device="cuda") * 2.0 ** top).to(torch.bfloat16)
    q = torch.zeros(1, 1, 8, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    for sink in (0, n // 2, n - 1):
        k.zero_()
        k[0, sink, :, 0] = 1.0
        vs = v.clone()
        vs[0, sink] = 1.5 * 2.0 ** top
        fsa.fsa_cache_append(cache, k, vs, table, i32(lens))
        run_attention(fsa, q, cache, table, lens, scale=math.log(min(n, 16384)))
        run_attention(fsa, q, cache, table, lens, scale=16.0, dtype="bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,Hkv,width", SPLITS)
@pytest.mark.parametrize("kind", ["rising", "falling", "any", "after zeros"])
def test_values_of_every_size(kind, lens, Hkv, width, D):
    """V from 2^-80 to 2^127, a size a token, in every order: the running offset of V's scales
    moves over its whole range without losing the sum of the weights."""
    fsa = _fsa()
    g = gen(105)
    B, S = len(lens), max(lens)
    table, pages = make_table(g, lens, 16)
    table = wide_table(table, width)
    cache = fsa.empty_cache(pages, 16, Hkv, D, "E2M1")
    at = torch.linspace(-80, 126.9, S, device="cuda")
    at = {"rising": at, "falling": at.flip(0), "any": at[torch.randperm(S, generator=g, device="cuda")],
          "after zeros": torch.where(torch.arange(S, device="cuda") < S // 2, -200.0, 126.0)}[kind]
    size = torch.exp2(at.double())[None, :, None, None]
    v = (size * (1 + torch.rand(B, S, Hkv, D, generator=g, device="cuda"))).clamp(max=3.3e38)
    v = v * torch.where(torch.rand(B, S, Hkv, D, generator=g, device="cuda") < 0.5, -1, 1)
    k = normal(g, B, S, Hkv, D)
    fsa.fsa_cache_append(cache, k, v.to(torch.bfloat16), table, i32(lens), i32(lens))
    for Sq in (1, 4):
        run_attention(fsa, normal(g, B, Sq, 4 * Hkv, D), cache, table, lens)
    run_attention(fsa, normal(g, B, 1, 4 * Hkv, D) * 4, cache, table, lens, dtype="bf16")


@pytest.mark.parametrize("fmt,D,top", [("E2M1", 128, 30), ("E2M1", 128, 127), ("E2M1", 64, 80), ("NVFP4", 128, 11), ("NVFP4", 64, 11)])
@pytest.mark.parametrize("lens,Hkv,width", SPLITS + [pytest.param([33, 5], 1, 4, id="two tiles"), pytest.param([96], 2, 100, id="a tile a CTA")])
def test_values_behind_a_row(lens, Hkv, width, fmt, D, top):
    """Values at positions behind a row, however large, do not change the row: it is held to
    the bounds of the keys that it sees."""
    fsa = _fsa()
    g = gen(107)
    B, S = len(lens), max(lens)
    table, pages = make_table(g, lens, 16)
    table = wide_table(table, width)
    cache = fsa.empty_cache(pages, 16, Hkv, D, fmt)
    for G, Sq in ((4, 2), (4, 5), (1, 17)):
        k, v = normal(g, B, S, Hkv, D), normal(g, B, S, Hkv, D) * 2.0 ** -6
        for b, n in enumerate(lens):
            for i in range(1, min(n, Sq)):             # each new position larger than the one before
                v[b, n - Sq + i if n >= Sq else i] *= 2.0 ** (6 + top * i / Sq)
        fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(lens))
        q, scale = normal(g, B, Sq, G * Hkv, D), D ** -0.5
        out, lse = torch.empty(B, Sq, G * Hkv, D, device="cuda"), torch.empty(B, Sq, G * Hkv, device="cuda")
        fsa.fsa_attention_cache(q, cache, table, i32(lens), out=out, lse=lse)
        for i in range(Sq):
            rows = slice(i, i + 1)
            check_attention(q[:, rows], cache, table, [max(0, n - Sq + 1 + i) for n in lens], [1] * B, True, scale, out[:, rows],
                            lse[:, rows], out[:, rows])


@pytest.mark.parametrize("seed", range(30))
def test_random_ranges(seed):
    """Seeded random shapes with pages outside the pool here and there, values of random sizes,
    rows that see different keys."""
    import random
    fsa = _fsa()
    r, g = random.Random(500 + seed), gen(500 + seed)
    D, fmt, page = r.choice((64, 128)), r.choice(("E2M1", "NVFP4")), r.choice((16, 32, 128))
    Hkv, G, Sq = r.choice((1, 2, 5)), r.choice((1, 3, 8)), r.choice((1, 2, 5, 17))
    B, top = r.choice((1, 4, 40)), r.choice((40, 500, 3000))
    lens = [r.choice((0, 1, r.randint(0, top), top)) for _ in range(B)]
    q_lens = [r.randint(0, Sq) for _ in range(B)] if r.random() < 0.5 else None
    table, pages = make_table(g, lens, page)
    table = wide_table(table, r.choice((0, 1000 // page + 1)))
    cache = fsa.empty_cache(pages, page, Hkv, D, fmt)
    cache.pages.fill_(0xFF)
    S = max(lens + [1])
    low, high = (-60, 126) if fmt == "E2M1" else (-6, 10)
    size = torch.exp2(torch.randint(low, high, (B, S, 1, 1), generator=g, device="cuda").double())
    v = (normal(g, B, S, Hkv, D).double() * (size if r.random() < 0.7 else 1.0)).clamp(-3.3e38, 3.3e38).to(torch.bfloat16)
    fsa.fsa_cache_append(cache, normal(g, B, S, Hkv, D), v, table, i32(lens), i32(lens))
    gone = torch.rand(table.shape, generator=g, device="cuda") < r.choice((0.0, 0.1, 0.6))
    table = torch.where(gone, torch.where(torch.rand(table.shape, generator=g, device="cuda") < 0.5, -1, pages).int(), table)
    q = normal(g, B, Sq, Hkv * G, D) * r.choice((1.0, 4.0))
    run_attention(fsa, q, cache, table, lens, q_lens, r.random() < 0.8, scale=r.choice((None, -0.1, 0.3)), dtype=r.choice(("f32", "bf16")))


@pytest.mark.parametrize("width", [512, 2048])
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_a_captured_step_goes_on(fmt, width):
    """A decode step (prepare, write, attend) captured once and replayed: it follows positions,
    lengths and contents on the device, with the bits of the same calls made one by one."""
    fsa = _fsa()
    g = gen(109)
    B, H, Hkv, D, page = 3, 8, 2, 128, 16
    lens = [300, 17, 1]
    table, pages = make_table(g, [n + 8 for n in lens], page)
    table = wide_table(table, width // page)
    inv = 1e4 ** (-torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
    w = normal(g, D)
    caches = [fsa.empty_cache(pages, page, Hkv, D, fmt) for _ in range(2)]
    k, v = normal(g, B, 300, Hkv, D), normal(g, B, 300, Hkv, D)
    for cache in caches:
        cache.pages.fill_(0xFF)
        fsa.fsa_cache_append(cache, k, v, table, i32(lens), i32(lens))
    qkv, pos, n = normal(g, B, 1, H + 2 * Hkv, D), i32([[x] for x in lens]), i32(lens)

    def step(cache, qkv, pos, n):
        q, k = fsa.fsa_qk_norm_rope(qkv[:, :, :H], qkv[:, :, H:H + Hkv], pos, inv, q_weight=w, k_weight=w)
        n = n + 1
        fsa.fsa_cache_append(cache, k, qkv[:, :, H + Hkv:], table, n)
        return fsa.fsa_attention_cache(q, cache, table, n, out_dtype="bf16")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kept = caches[0].pages.clone()
    with torch.cuda.stream(side):
        step(caches[0], qkv, pos, n)                   # warm
    torch.cuda.current_stream().wait_stream(side)
    caches[0].pages.copy_(kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0], qkv, pos, n)
    for _ in range(6):
        fresh = normal(g, *qkv.shape)
        want = step(caches[1], fresh, pos.clone(), n.clone())
        qkv.copy_(fresh)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(caches[0].pages, caches[1].pages)
        pos += 1
        n += 1
