"""Cases of the serving operators around the MX attention: queries and keys normalised and
rotated (fsa_qk_norm_rope), a paged 4-bit key/value cache written and read back
(fsa_cache_append, fsa_cache_read), and attention over that cache (fsa_attention_cache).

`run` computes a case in elementary torch operations, or, with `own` true, by the calls a
user of the package makes.  `exact` gives the operator's definition in 64 bits.

The cache holds K and V of whole tokens.  A page is [Hkv][page/16] groups of 16 tokens; a
group is 16 rows of K codes, 16 rows of V codes (D/2 bytes each), 16 rows of K scales and
16 rows of V scales (one byte per block).  The codes are E2M1, two to a byte, the even
element in the low nibble; byte t*(D/8) + 2s + h of a K row holds elements 16s + 4t + 2h
and the next, byte g*(D/16) + i of a V row elements 16i + 2g and the next.  "E2M1" has an
E8M0 scale for each 32 elements, "NVFP4" an E4M3 scale for each 16."""
import math
import random

import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- the cases
def _attn(name, B, Sq, H, Hkv, D, longest, page, fmt, shortest=None, ragged_q=False, lse=False):
    return dict(name=name, op="attention", B=B, Sq=Sq, H=H, Hkv=Hkv, D=D, longest=longest,
                shortest=longest if shortest is None else shortest, page=page, fmt=fmt, ragged_q=ragged_q, lse=lse)


def _cache(name, op, B, S, Hkv, D, longest, page, fmt, shortest=None):
    return dict(name=name, op=op, B=B, S=S, Hkv=Hkv, D=D, longest=longest,
                shortest=longest if shortest is None else shortest, page=page, fmt=fmt)


def _rope(name, B, S, H, Hkv, D, rotary, axes, interleaved, far, heads_first, norm=True):
    return dict(name=name, op="norm_rope", B=B, S=S, H=H, Hkv=Hkv, D=D, rotary=rotary, axes=axes,
                interleaved=interleaved, far=far, heads_first=heads_first, norm=norm)


def listed():
    return [
        # one conversation that has just begun: a single new token, where latency is all there is
        _attn("attn_one", 1, 1, 32, 8, 128, 333, 16, "E2M1"),
        # a server's decode step: many conversations of uneven length
        _attn("attn_batch", 64, 1, 32, 8, 128, 8192, 64, "NVFP4", shortest=17),
        # one long document of 128K tokens, as in the long causal workloads: few rows, one long axis
        _attn("attn_long", 1, 1, 32, 8, 128, 131072, 64, "E2M1", lse=True),
        # guessed tokens checked together, up to five for each conversation, every head with its own keys
        _attn("attn_verify", 16, 5, 24, 24, 128, 8201, 32, "E2M1", shortest=2, ragged_q=True, lse=True),
        # small heads, an odd group of seven query heads, many short conversations
        _attn("attn_small_heads", 256, 2, 14, 2, 64, 1500, 16, "NVFP4", shortest=1),
        # a decode step writes one token for each conversation, and the values cached are read back
        _cache("write_step", "append", 128, 1, 8, 128, 4096, 64, "NVFP4", shortest=1),
        # prompts of uneven length written into the cache, the prefill workload's sizes
        _cache("write_prompts", "append", 4, 4096, 8, 128, 6001, 64, "E2M1", shortest=1500),
        # a cached document of 128K tokens read back as the operands of a prompt's attention
        _cache("read_long", "read", 1, 131072, 8, 128, 131072, 64, "NVFP4"),
        # the decode step's queries and keys, far into their sequences
        _rope("rope_step", 64, 1, 32, 8, 128, 128, 1, False, 1 << 20, False),
        # a 16K prompt on its way to the attention, which takes heads before positions
        _rope("rope_prompt", 1, 16384, 32, 8, 128, 128, 1, False, 1 << 15, True),
        # the video workload: 21 x 45 x 80 latent patches, an axis each for time, height and width
        _rope("rope_video", 1, 75600, 40, 40, 128, 128, 3, True, 21 * 45 * 80, True),
        # small heads turned in half of their dimensions, a batch of odd length
        _rope("rope_partial", 3, 1531, 14, 2, 64, 32, 1, False, 1 << 13, False),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))


def draw(rng):
    largest = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("attention", "attention", "append", "read", "norm_rope", "norm_rope"))
        D = rng.choice((64, 128, 128))
        Hkv = rng.choice((1, 2, 4, 8, 8, 24))
        group = rng.choice((1, 4, 4, 5, 7, 8))
        page, fmt = rng.choice((16, 32, 64, 128)), rng.choice(("E2M1", "NVFP4"))
        if op == "attention":
            longest = _spread(rng, 1, 131072)
            case = _attn("", _spread(rng, 1, 256), rng.choice((1, 1, 1, 2, 3, 4, 8)), Hkv * group, Hkv, D, longest, page,
                         fmt, rng.choice((None, max(1, longest // 64), 1)), rng.random() < 0.4, rng.random() < 0.5)
        elif op == "norm_rope":
            axes = rng.choice((1, 1, 3))
            case = _rope("", _spread(rng, 1, 128), _spread(rng, 1, 65536), Hkv * group, Hkv, D,
                         D if axes > 1 else rng.choice((D, D, D // 2, D // 4)), axes, rng.random() < 0.5,
                         _spread(rng, 4096, 1 << 20), rng.random() < 0.5, rng.random() < 0.8)
        else:
            S = _spread(rng, 1, 131072)
            longest = S + _spread(rng, 1, 8192)
            case = _cache("", op, _spread(rng, 1, 256), S, Hkv, D, longest, page, fmt, rng.choice((None, 1, max(1, S // 2))))
        padded = case["B"] * case["longest"] * Hkv * D if op != "norm_rope" else 0
        if _cost(case) <= largest and padded <= 6e8:        # the plain form unpacks every sequence to the longest
            del case["name"]
            return case


def _lengths(case):
    """The sequences' lengths (tokens in the cache, the new ones among them), spread over shortest..longest."""
    rng = random.Random("%(B)d %(longest)d %(shortest)d" % case)
    lens = [_spread(rng, case["shortest"], case["longest"]) for _ in range(case["B"])]
    lens[0] = case["longest"]
    return lens


def _news(case, lens):
    """How many of each sequence's tokens are new: its queries, or what the call writes or reads."""
    S = case["Sq"] if case["op"] == "attention" else case["S"]
    if case.get("ragged_q"):
        rng = random.Random(7)
        return [rng.randint(1, S) for _ in lens]
    if case["op"] == "attention":
        return [S for _ in lens]
    return [min(S, n) for n in lens]


def _code_bytes(case):
    D = case["D"]
    return D // 2 + D // (32 if case["fmt"] == "E2M1" else 16)


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.0e15


def work(case):
    B, D = case["B"], case["D"]
    if case["op"] == "norm_rope":
        x = B * case["S"] * (case["H"] + case["Hkv"]) * D
        return {"bytes": 4.0 * x + 4.0 * B * case["S"] * case["axes"], "flops": 7.0 * x}
    lens = _lengths(case)
    news = _news(case, lens)
    if case["op"] == "attention":
        rows, H, Hkv = sum(news), case["H"], case["Hkv"]
        seen = sum(max(0, n - m + i + 1) for n, m in zip(lens, news) for i in range(m))
        cached = sum(lens) * Hkv * 2 * _code_bytes(case)
        return {"bytes": cached + 4.0 * rows * H * D + (4.0 * rows * H if case["lse"] else 0) + 12.0 * B, "flops": 4.0 * seen * H * D}
    rows = sum(news) * case["Hkv"] * 2
    codes = rows * _code_bytes(case)
    values = 2.0 * rows * D
    return {"bytes": codes + (2 if case["op"] == "append" else 1) * values, "flops": 3.0 * rows * D}


# ------------------------------------------------------------------------------ the inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _keys(g, *shape):
    """Keys with four strong channels a head, as trained models have them."""
    k = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
    gain = torch.ones(shape[-2:], device="cuda")
    gain[:, torch.randperm(shape[-1], generator=g, device="cuda")[:4]] = 4.0
    return k * gain


def _table(case, g, lens):
    """Pages of a pool in random order, with some to spare; -1 behind each sequence's last."""
    P = case["page"]
    need = torch.tensor([-(-n // P) for n in lens], device="cuda")
    width = int(need.max()) + 1
    used = torch.arange(width, device="cuda")[None, :] < need[:, None]
    total = int(need.sum())
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
    table[used] = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    return table, total + 3


def prepare(case, seed):
    g = _generator(seed)
    B, D, Hkv = case["B"], case["D"], case["Hkv"]
    st = {"case": case}
    if case["op"] == "norm_rope":
        S, H, n = case["S"], case["H"], case["rotary"] // 2
        qkv = _normal(g, B, S, H + 2 * Hkv, D)             # the projection's output: q, k and v side by side
        qkv *= torch.exp(0.5 * torch.randn(1, 1, H + 2 * Hkv, 1, generator=g, device="cuda")).to(qkv.dtype)
        st["q"], st["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        if case["norm"]:
            st["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
            st["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        else:
            st["q_weight"] = st["k_weight"] = None
        if case["axes"] == 1:
            first = torch.randint(0, max(1, case["far"] - S), (B, 1), generator=g, device="cuda")
            st["pos"] = (first + torch.arange(S, device="cuda")).to(torch.int32)[:, :, None].contiguous()
            st["sections"] = (n,)
            st["inv_freq"] = 1.0e6 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n)
        else:                                               # patches of a film, frame by frame
            at = torch.arange(S, device="cuda") + torch.randint(0, 3600, (B, 1), generator=g, device="cuda")
            st["pos"] = torch.stack((at // 3600, at // 80 % 45, at % 80), dim=2).to(torch.int32).contiguous()
            other = n // 3
            st["sections"] = (n - 2 * other, other, other)
            st["inv_freq"] = torch.cat([1.0e4 ** (-torch.arange(m, device="cuda", dtype=torch.float64) / m) for m in st["sections"]])
        shape = lambda h: (B, h, S, D) if case["heads_first"] else (B, S, h, D)  # noqa: E731
        st["q_out"] = torch.empty(shape(H), dtype=torch.bfloat16, device="cuda")
        st["k_out"] = torch.empty(shape(Hkv), dtype=torch.bfloat16, device="cuda")
        return st
    lens = _lengths(case)
    news = _news(case, lens)
    st["table"], pages = _table(case, g, lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["news"] = torch.tensor(news, dtype=torch.int32, device="cuda")
    st["first"] = st["lens"] - st["news"]
    P = case["page"]
    if case["op"] == "append":
        S = case["S"]
        st["pages"] = torch.zeros(pages, Hkv * P * 2 * _code_bytes(case), dtype=torch.uint8, device="cuda")
        st["k"] = _keys(g, B, S, Hkv, D).to(torch.bfloat16)
        st["v"] = _normal(g, B, S, Hkv, D)
    else:
        st["pages"] = torch.cat([_encode_pages(case, _keys(g, m, P, Hkv, D).to(torch.bfloat16), _normal(g, m, P, Hkv, D))
                                 for m in [min(2048, pages - i) for i in range(0, pages, 2048)]])
    if case["op"] == "attention":
        st["q"] = _normal(g, B, case["Sq"], case["H"], D)
        st["out"] = torch.zeros(B, case["Sq"], case["H"], D, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros(B, case["Sq"], case["H"], dtype=torch.float32, device="cuda") if case["lse"] else None
    else:
        st["k_back"] = torch.zeros(B, case["S"], Hkv, D, dtype=torch.bfloat16, device="cuda")
        st["v_back"] = torch.zeros(B, case["S"], Hkv, D, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------- the cache's format, in torch
def _codes(y):
    """E2M1 code of each y: the nearest magnitude, ties to the even code, saturating."""
    a = y.abs()
    m = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    return m | (torch.signbit(y).to(torch.uint8) << 3)


def _power(e):
    """2^e for whole e in -127..127, exactly (exp2 may be off in the last place)."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).view(torch.float32)


def _quantise(x, fmt):
    """x [..., D] as (codes [..., D], scale bytes [..., D/block])."""
    block = 32 if fmt == "E2M1" else 16
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // block, block)
    amax = b.abs().amax(-1)
    if fmt == "E2M1":
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
        y, scales = b * _power(-e)[..., None], (e + 127).to(torch.uint8)
    else:
        s8 = (amax / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float()[..., None]
        y, scales = torch.where(s > 0, b / s, torch.zeros_like(b)), s8.view(torch.uint8)
    return _codes(y).reshape(x.shape), scales


def _rows(codes, key):
    """Codes [..., D] as the bytes of cache rows, in the order of K rows or of V rows."""
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    order = (4, 2) if key else (8,)
    return b.unflatten(-1, (-1, *order)).movedim(-1 - len(order), -len(order) if key else -1).flatten(-2 - key)


def _encode_pages(case, k, v):
    """K and V [pages, page, Hkv, D] as pages of the pool."""
    n, P, Hkv, D = k.shape
    (ck, sk), (cv, sv) = _quantise(k, case["fmt"]), _quantise(v, case["fmt"])
    parts = [x.transpose(1, 2).reshape(n, Hkv, P // 16, -1) for x in (_rows(ck, True), _rows(cv, False), sk, sv)]
    return torch.cat(parts, dim=3).reshape(n, -1)


def _table_of_bytes(dtype):
    m = torch.tensor(MAGNITUDES + tuple(-x for x in MAGNITUDES), dtype=dtype, device="cuda")
    i = torch.arange(256, device="cuda")
    return torch.stack((m[i & 15], m[i >> 4]), dim=1)


def _decode(case, pages, dtype=torch.float32):
    """Pages [..., page_bytes] as K and V values [..., page, Hkv, D]."""
    lead, P, Hkv, D = pages.shape[:-1], case["page"], case["Hkv"], case["D"]
    block = 32 if case["fmt"] == "E2M1" else 16
    sb = D // block
    g = pages.reshape(-1, Hkv, P // 16, 16 * (D + 2 * sb))
    lut = _table_of_bytes(dtype)

    def values(codes, scales, key):
        n = codes.shape[0]
        if key:                                             # bytes [t][s][h] -> [s][t][h]
            codes = codes.reshape(n, Hkv, P, 4, D // 16, 2).transpose(3, 4)
        else:                                               # bytes [g][i] -> [i][g]
            codes = codes.reshape(n, Hkv, P, 8, D // 16).transpose(3, 4)
        x = lut[codes.reshape(n, Hkv, P, D // 2).int()].reshape(n, Hkv, P, sb, block)
        if case["fmt"] == "E2M1":
            s = _power(scales.int() - 127).to(dtype)
        else:
            s = scales.contiguous().view(torch.float8_e4m3fn).to(dtype)
        x = x * s.reshape(n, Hkv, P, sb, 1)
        return x.reshape(n, Hkv, P, D).transpose(1, 2).reshape(*lead, P, Hkv, D)

    k = values(g[..., :8 * D], g[..., 16 * D:16 * (D + sb)], True)
    v = values(g[..., 8 * D:16 * D], g[..., 16 * (D + sb):], False)
    return k, v


# -------------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import softmax_mx_block_gb300 as fsa
    case = st["case"]
    if case["op"] == "norm_rope":
        swap = (lambda x: x.transpose(1, 2)) if case["heads_first"] else (lambda x: x)
        fsa.fsa_qk_norm_rope(st["q"], st["k"], st["pos"], st["inv_freq"], sections=st["sections"],
                             q_weight=st["q_weight"], k_weight=st["k_weight"], norm=case["norm"], eps=1e-6,
                             interleaved=case["interleaved"], q_out=swap(st["q_out"]), k_out=swap(st["k_out"]))
        return {"q": st["q_out"], "k": st["k_out"]}
    cache = fsa.MxCache(st["pages"], case["page"], case["Hkv"], case["D"], case["fmt"])
    if case["op"] == "attention":
        fsa.fsa_attention_cache(st["q"], cache, st["table"], st["lens"], q_lens=st["news"], causal=True,
                                scale=case["D"] ** -0.5, out=st["out"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if case["op"] == "append":
        fsa.fsa_cache_append(cache, st["k"], st["v"], st["table"], st["lens"], new_lens=st["news"])
    fsa.fsa_cache_read(cache, st["table"], st["lens"], start=st["first"], k_out=st["k_back"], v_out=st["v_back"])
    return {"k": st["k_back"], "v": st["v_back"]}


def _plain(st):
    case = st["case"]
    if case["op"] == "norm_rope":
        angle = _angles(st)
        cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
        back = (0, 2, 1, 3) if case["heads_first"] else (0, 1, 2, 3)
        return {"q": _turned(st["q"], st["q_weight"], cos, sin, case).permute(back).contiguous(),
                "k": _turned(st["k"], st["k_weight"], cos, sin, case).permute(back).contiguous()}
    if case["op"] == "attention":
        return _attended(st)
    at = torch.arange(case["S"], device="cuda")[None, :]
    live = (at < st["news"][:, None])[:, :, None, None]
    place = (st["first"][:, None] + at).clamp(max=int(case["longest"]) - 1)
    if case["op"] == "append":
        page = st["table"].gather(1, (place // case["page"]).long())
        k, v = _written(case, st["k"], st["v"])
        _store(case, st["pages"], page, place % case["page"], live[:, :, 0, 0], k, v)
        return {"k": torch.where(live, k[2], st["k_back"]), "v": torch.where(live, v[2], st["v_back"])}
    pool_k, pool_v = (x.to(torch.bfloat16) for x in _decode(case, st["pages"]))
    page = st["table"].gather(1, (place // case["page"]).long()).clamp(min=0).long()
    inside = (place % case["page"]).long()
    return {"k": torch.where(live, pool_k[page, inside], st["k_back"]), "v": torch.where(live, pool_v[page, inside], st["v_back"])}


def _written(case, *xs):
    """(codes, scale bytes, the values they stand for) of each x [..., D]."""
    got = []
    m = torch.tensor(MAGNITUDES + tuple(-x for x in MAGNITUDES), device="cuda")
    for x in xs:
        codes, scales = _quantise(x, case["fmt"])
        s = _power(scales.int() - 127) if case["fmt"] == "E2M1" else scales.view(torch.float8_e4m3fn).float()
        values = (m[codes.int()].reshape(*scales.shape, -1) * s[..., None]).reshape(x.shape).to(torch.bfloat16)
        got.append((codes, scales, values))
    return got


def _store(case, pages, page, inside, live, k, v):
    """Puts the codes and scales of tokens [B, S, Hkv] into their places of the pool."""
    Hkv, P, D = case["Hkv"], case["page"], case["D"]
    sb = k[1].shape[-1]
    groups = pages.view(pages.shape[0], Hkv, P // 16, 16 * (D + 2 * sb))
    page, inside = page[live].long(), inside[live].long()
    group, row = inside // 16, inside % 16

    def rows(first, width, x):
        groups[:, :, :, first:first + 16 * width].unflatten(3, (16, width))[page, :, group, row] = x

    for (codes, scales, _), at, scale_at, key in ((k, 0, 16 * D, True), (v, 8 * D, 16 * (D + sb), False)):
        rows(at, D // 2, _rows(codes[live], key))
        rows(scale_at, sb, scales[live])


def _angles(st):
    axis = torch.repeat_interleave(torch.arange(len(st["sections"]), device="cuda"),
                                   torch.tensor(st["sections"], device="cuda"), output_size=st["inv_freq"].numel())
    return st["pos"].double()[:, :, axis] * st["inv_freq"]


def _turned(x, weight, cos, sin, case):
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    r = case["rotary"]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., r:]), dim=-1).to(torch.bfloat16)


def _attended(st):
    case = st["case"]
    B, Sq, H, Hkv, D = case["B"], case["Sq"], case["H"], case["Hkv"], case["D"]
    k, v = _decode(case, st["pages"][st["table"].clamp(min=0).long()])
    k, v = k.flatten(1, 2).transpose(1, 2), v.flatten(1, 2).transpose(1, 2)          # [B, Hkv, L, D]
    q = st["q"].float().reshape(B, Sq, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5                                # [B, Hkv, Sq*G, L]
    row = torch.arange(Sq, device="cuda")[None, :]
    last = (st["first"][:, None] + row).repeat_interleave(H // Hkv, dim=1)           # the last key a row sees
    seen = torch.arange(k.shape[2], device="cuda") <= last[:, None, :, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    o = o.reshape(B, Hkv, Sq, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Sq, H, D)
    live = row < st["news"][:, None]
    out = torch.where(live[:, :, None, None], o.to(torch.bfloat16), st["out"])
    if st["lse"] is None:
        return {"out": out, "lse": None}
    lse = (top + torch.log(total)).reshape(B, Hkv, Sq, H // Hkv).permute(0, 2, 1, 3).reshape(B, Sq, H)
    return {"out": out, "lse": torch.where(live[:, :, None], lse, st["lse"])}


# ---------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_norm_rope(st, case)
    if case["op"] == "append":
        live = torch.arange(case["S"], device="cuda")[None, :] < st["news"][:, None]
        return {n: torch.where(live[:, :, None, None], _exact_rounded(st[n], case["fmt"]), 0.0) for n in ("k", "v")}
    if case["op"] == "read":
        got = {n: torch.zeros(case["B"], case["S"], case["Hkv"], case["D"], dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for b, (length, new) in enumerate(zip(_lengths(case), st["news"].tolist())):
            for n, x in zip(("k", "v"), _exact_sequence(st, case, b, length)):
                got[n][b, :new] = x[length - new:]
        return got
    return _exact_attention(st, case)


def _exact_norm_rope(st, case):
    S, r, half = case["S"], case["rotary"], case["rotary"] // 2
    got = {}
    for n in ("q", "k"):
        x = st[n]
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        for i in range(0, S, 4096):                         # positions in turn: the whole would be large
            c = x[:, i:i + 4096].double()
            if case["norm"]:
                c = c / (c.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6).sqrt() * st[n + "_weight"].double()
            z = c.clone()
            pair = 0
            for axis, count in enumerate(st["sections"]):
                for j in range(pair, pair + count):
                    one, two = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
                    t = (st["pos"][:, i:i + 4096, axis].double() * st["inv_freq"][j])[:, :, None]
                    z[..., one] = c[..., one] * t.cos() - c[..., two] * t.sin()
                    z[..., two] = c[..., two] * t.cos() + c[..., one] * t.sin()
                pair += count
            y[:, i:i + 4096] = z
        got[n] = y.transpose(1, 2).contiguous() if case["heads_first"] else y
    return got


def _double_power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _binade(x):
    """The largest power of two that is not over x, as its exponent."""
    return torch.frexp(x).exponent - 1


def _exact_rounded(x, fmt):
    """The value that each element of x is cached as."""
    size = 32 if fmt == "E2M1" else 16
    b = x.double().unflatten(-1, (-1, size))
    top = b.abs().max(-1, keepdim=True).values
    if fmt == "E2M1":
        scale = _double_power(_binade(top.clamp(min=2.0 ** -125)) - 2)
    else:
        t = (top / 6.0).clamp(max=448.0)
        step = _double_power(_binade(t.clamp(min=2.0 ** -6)) - 3)
        scale = torch.round(t / step) * step                # ties to even, as torch.round has them
    y = torch.where(scale > 0, b / scale, torch.zeros_like(b)).clamp(-6.0, 6.0)
    step = _double_power(_binade(y.abs().clamp(min=1.0)) - 1)
    return (torch.round(y / step) * step * scale).flatten(-2)


def _exact_sequence(st, case, b, length):
    """K and V [length, Hkv, D] of one sequence, element by element from the format's description."""
    Hkv, D, P = case["Hkv"], case["D"], case["page"]
    size = 32 if case["fmt"] == "E2M1" else 16
    sb = D // size
    raw = st["pages"][st["table"][b, :-(-length // P)].long()].reshape(-1, Hkv, P // 16, 16 * (D + 2 * sb))
    raw = raw.permute(0, 2, 1, 3).flatten(0, 1)             # [groups of 16 tokens, Hkv, bytes]
    d = torch.arange(D, device="cuda")
    s, t, h = d // 16, d % 16 // 4, d % 4 // 2
    i, g = d // 16, d % 16 // 2
    mag = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
    got = []
    for at, scale_at, byte in ((0, 16 * D, t * (D // 8) + 2 * s + h), (8 * D, 16 * (D + sb), g * (D // 16) + i)):
        rows = raw[..., at:at + 8 * D].unflatten(2, (16, D // 2))
        code = (rows[..., byte].int() >> (4 * (d % 2)).int()) & 15
        value = mag[(code & 7).long()] * (1.0 - 2.0 * (code >> 3).double())
        sc = raw[..., scale_at:scale_at + 16 * sb].unflatten(2, (16, sb)).int()
        if case["fmt"] == "E2M1":
            sc = _double_power(sc - 127)
        else:
            e, m = (sc >> 3) & 15, (sc & 7).double()
            sc = torch.where(e > 0, (8.0 + m) * _double_power(e - 10), m * 2.0 ** -9)
        x = value * sc[..., d // size]
        got.append(x.transpose(1, 2).reshape(-1, Hkv, D)[:length])
    return got


def _exact_attention(st, case):
    B, Sq, H, Hkv, D = case["B"], case["Sq"], case["H"], case["Hkv"], case["D"]
    out = torch.zeros(B, Sq, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Sq, H, dtype=torch.float64, device="cuda")
    for b, (length, new) in enumerate(zip(_lengths(case), st["news"].tolist())):
        k, v = _exact_sequence(st, case, b, length)
        for i in range(new):
            sees = length - new + i + 1
            if sees <= 0:
                lse[b, i] = -math.inf
                continue
            q = st["q"][b, i].double().reshape(Hkv, H // Hkv, D)
            s = torch.einsum("hgd,lhd->hgl", q, k[:sees]) / math.sqrt(D)
            lse[b, i] = torch.logsumexp(s, -1).reshape(H)
            out[b, i] = torch.einsum("hgl,lhd->hgd", torch.softmax(s, -1), v[:sees]).reshape(H, D)
    return {"out": out, "lse": lse if case["lse"] else None}
