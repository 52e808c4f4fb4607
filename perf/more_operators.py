"""Cases of the serving operators that take prompts in chunks and long conversations through a
window, over the paged 4-bit key/value cache: queries and keys normalised and rotated on the
way into the cache (fsa_cache_append_rope), attention of a chunk of new tokens over the cache
(fsa_attention_chunk), and attention of few rows that see a sliding window and the first
tokens (fsa_attention_cache with window and sinks).

`run` computes a case in elementary torch operations, or, with `own` true, by the calls a
user of the package makes.  `exact` gives the operator's definition in 64 bits.

The cache holds K and V of whole tokens.  A page is [Hkv][page/16] groups of 16 tokens; a
group is 16 rows of K codes, 16 rows of V codes (D/2 bytes each), 16 rows of K scales and
16 rows of V scales (one byte per block).  The codes are E2M1, two to a byte, the even
element in the low nibble; byte t*(D/8) + 2s + h of a K row holds elements 16s + 4t + 2h
and the next, byte g*(D/16) + i of a V row elements 16i + 2g and the next.  "E2M1" has an
E8M0 scale for each 32 elements, "NVFP4" an E4M3 scale for each 16.

A row at position p sees key j where j <= p and, with a window, j > p - window or j < sinks."""
import math
import random

import numpy as np
import torch

own = False

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- the cases
def _attn(name, op, B, Sq, H, Hkv, D, longest, page, fmt, shortest=None, window=0, sinks=0, ragged_q=False, lse=False):
    return dict(name=name, op=op, B=B, Sq=Sq, H=H, Hkv=Hkv, D=D, longest=longest,
                shortest=longest if shortest is None else shortest, page=page, fmt=fmt, window=window, sinks=sinks,
                ragged_q=ragged_q, lse=lse)


def _append(name, B, S, H, Hkv, D, longest, page, fmt, rotary, shortest=None, interleaved=False, norm=True):
    return dict(name=name, op="append", B=B, S=S, H=H, Hkv=Hkv, D=D, longest=longest,
                shortest=longest if shortest is None else shortest, page=page, fmt=fmt, rotary=rotary,
                interleaved=interleaved, norm=norm)


def listed():
    return [
        # a decode step: one token of each conversation, far into some of them
        _append("append_step", 64, 1, 32, 8, 128, 65536, 64, "NVFP4", 128, shortest=1),
        # prompts of uneven length on their way into the cache, the prefill workload's sizes
        _append("append_prompts", 4, 4096, 32, 8, 128, 6001, 64, "E2M1", 128, shortest=1500),
        # one 16K chunk of a long document
        _append("append_long", 1, 16384, 32, 8, 128, 131072, 64, "NVFP4", 128),
        # small heads turned in half of their dimensions, pair by pair, without a norm, a batch of odd length
        _append("append_partial", 3, 1531, 14, 2, 64, 1777, 16, "E2M1", 32, shortest=900, interleaved=True, norm=False),
        # a short question at the start of a conversation, where latency counts
        _attn("chunk_first", "chunk", 1, 77, 32, 8, 128, 77, 16, "E2M1"),
        # a server's mixed step: the next turns of eight conversations, up to 500 tokens each
        _attn("chunk_turns", "chunk", 8, 500, 32, 8, 128, 8192, 64, "NVFP4", shortest=600, ragged_q=True, lse=True),
        # the last chunk of a 128K document, as in the long causal workloads
        _attn("chunk_long", "chunk", 1, 2048, 32, 8, 128, 131072, 64, "E2M1", lse=True),
        # a layer of small heads with a window: a large chunk in the middle of a document
        _attn("chunk_window", "chunk", 1, 8192, 14, 2, 64, 32768, 64, "NVFP4", window=4096, sinks=4),
        # a decode step of a windowed layer: many conversations, few of them shorter than the window
        _attn("window_step", "window", 64, 1, 32, 8, 128, 32768, 64, "NVFP4", shortest=700, window=4096, sinks=4),
        # one long conversation in such a layer: latency, whatever its length
        _attn("window_one", "window", 1, 1, 32, 8, 128, 131072, 64, "E2M1", window=1024, sinks=4, lse=True),
        # guessed tokens checked together, up to five for each conversation, every head with its own keys
        _attn("window_verify", "window", 16, 5, 24, 24, 128, 16411, 32, "E2M1", shortest=3, window=2048, sinks=16, ragged_q=True, lse=True),
        # small heads, an odd group of seven query heads, a short odd window and no first tokens
        _attn("window_small", "window", 256, 2, 14, 2, 64, 3001, 16, "NVFP4", shortest=1, window=509),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))


def draw(rng):
    largest = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(("append", "append", "chunk", "chunk", "window", "window"))
        D = rng.choice((64, 128, 128))
        Hkv = rng.choice((1, 2, 4, 8, 8, 24))
        H = Hkv * rng.choice((1, 4, 4, 5, 7, 8))
        page, fmt = rng.choice((16, 32, 64, 128)), rng.choice(("E2M1", "NVFP4"))
        if op == "append":
            S = rng.choice((1, _spread(rng, 2, 16384), _spread(rng, 2, 16384)))
            longest = S + _spread(rng, 1, 65536)
            case = _append("", _spread(rng, 1, 256), S, H, Hkv, D, longest, page, fmt, rng.choice((D, D, D // 2, D // 4)),
                           rng.choice((None, 1, max(1, S // 2))), rng.random() < 0.3, rng.random() < 0.8)
        else:
            window = rng.choice((0, 0, _spread(rng, 64, 8192))) if op == "chunk" else _spread(rng, 32, 8192)
            Sq = _spread(rng, 33, 8192) if op == "chunk" else rng.choice((1, 1, 1, 2, 3, 4, 8))
            longest = _spread(rng, max(Sq, 64), 131072)
            case = _attn("", op, _spread(rng, 1, 32 if op == "chunk" else 256), Sq, H, Hkv, D, longest, page, fmt,
                         rng.choice((None, max(1, longest // 64), 1)), window, rng.choice((0, 1, 4, 64)) if window else 0,
                         rng.random() < 0.4, rng.random() < 0.5)
        if _cost(case) <= largest and _held(case) <= 6e8 and (op == "append" or _scores(case) <= 9e9):
            del case["name"]
            return case


def _held(case):
    """Elements of the pool and of the inputs."""
    rows = case["B"] * case["S"] * (case["H"] + 2 * case["Hkv"]) if case["op"] == "append" else 0
    return (sum(_lengths(case)) * case["Hkv"] + rows) * case["D"]


def _width(case):
    """Keys of a sequence that the plain form takes up."""
    if not case["window"]:
        return case["longest"]
    return case["sinks"] + case["window"] - 1 + case["Sq"]


def _scores(case):
    return case["B"] * case["Sq"] * case["H"] * _width(case)


def _lengths(case):
    """The sequences' lengths (tokens in the cache, the new ones among them), spread over shortest..longest."""
    rng = random.Random("%(B)d %(longest)d %(shortest)d" % case)
    lens = [_spread(rng, case["shortest"], case["longest"]) for _ in range(case["B"])]
    lens[0] = case["longest"]
    return lens


def _news(case, lens):
    """How many of each sequence's tokens are new: those written, or the query rows."""
    S = case["S"] if case["op"] == "append" else case["Sq"]
    rng = random.Random(7)
    return [min(n, rng.randint(1, S) if case.get("ragged_q") else S) for n in lens]


def _code_bytes(case):
    D = case["D"]
    return D // 2 + D // (32 if case["fmt"] == "E2M1" else 16)


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.0e15


def work(case):
    B, D, H, Hkv = case["B"], case["D"], case["H"], case["Hkv"]
    lens = _lengths(case)
    news = _news(case, lens)
    rows = sum(news)
    if case["op"] == "append":      # q, k and v read, q, the codes and the values read back written
        kv = 2 * rows * Hkv
        return {"bytes": 4.0 * rows * H * D + 4.0 * kv * D + kv * _code_bytes(case) + 12.0 * B, "flops": 7.0 * rows * (H + Hkv) * D + 3.0 * kv * D}
    w, first = case["window"] or 1 << 30, case["sinks"]
    used, seen = 0, 0
    for n, m in zip(lens, news):
        used += min(n, first + w - 1 + m)
        p = np.arange(n - m, n, dtype=np.int64) + 1
        seen += int((np.minimum(p, w) + np.clip(p - w, 0, first)).sum())
    return {"bytes": used * Hkv * 2.0 * _code_bytes(case) + 4.0 * rows * H * D + (4.0 * rows * H if case["lse"] else 0) + 12.0 * B,
            "flops": 4.0 * seen * H * D}


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
    B, D, H, Hkv, P = case["B"], case["D"], case["H"], case["Hkv"], case["page"]
    lens = _lengths(case)
    news = _news(case, lens)
    st = {"case": case}
    st["table"], pages = _table(case, g, lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["news"] = torch.tensor(news, dtype=torch.int32, device="cuda")
    st["first"] = st["lens"] - st["news"]
    if case["op"] == "append":
        S, half = case["S"], case["rotary"] // 2
        qkv = _normal(g, B, S, H + 2 * Hkv, D)             # the projection's output: q, k and v side by side
        qkv *= torch.exp(0.5 * torch.randn(1, 1, H + 2 * Hkv, 1, generator=g, device="cuda")).to(qkv.dtype)
        st["q"], st["k"], st["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        st["q_weight"] = st["k_weight"] = None
        if case["norm"]:
            st["q_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
            st["k_weight"] = (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        st["inv_freq"] = 1.0e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        st["pages"] = torch.zeros(pages, Hkv * P * 2 * _code_bytes(case), dtype=torch.uint8, device="cuda")
        st["q_out"] = torch.zeros(B, S, H, D, dtype=torch.bfloat16, device="cuda")
        st["k_back"] = torch.zeros(B, S, Hkv, D, dtype=torch.bfloat16, device="cuda")
        st["v_back"] = torch.zeros(B, S, Hkv, D, dtype=torch.bfloat16, device="cuda")
        return st
    st["pages"] = torch.cat([_encode_pages(case, _keys(g, m, P, Hkv, D).to(torch.bfloat16), _normal(g, m, P, Hkv, D))
                             for m in [min(4096, pages - i) for i in range(0, pages, 4096)]])
    st["q"] = _normal(g, B, case["Sq"], H, D)
    st["out"] = torch.zeros(B, case["Sq"], H, D, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros(B, case["Sq"], H, dtype=torch.float32, device="cuda") if case["lse"] else None
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
    """x [..., D] as (codes [..., D], scale bytes [..., D/block], the scales), in x's type."""
    block = 32 if fmt == "E2M1" else 16
    b = x.reshape(*x.shape[:-1], x.shape[-1] // block, block)
    amax = b.abs().amax(-1)
    if fmt == "E2M1":
        e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
        s, scales = _power(e).to(x.dtype), (e + 127).to(torch.uint8)
        y = b * _power(-e).to(x.dtype)[..., None]
    else:
        t = (amax / 6.0).clamp(max=448.0)
        step = _power(torch.frexp(t.clamp(min=2.0 ** -6)).exponent - 4).to(x.dtype)      # E4M3: eight steps a binade
        s = torch.round(t / step) * step
        scales = s.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
        y = torch.where(s[..., None] > 0, b / s[..., None], torch.zeros_like(b))
    return _codes(y).reshape(x.shape), scales, s


def _rows(codes, key):
    """Codes [..., D] as the bytes of cache rows, in the order of K rows or of V rows."""
    b = codes[..., 0::2] | (codes[..., 1::2] << 4)
    order = (4, 2) if key else (8,)
    return b.unflatten(-1, (-1, *order)).movedim(-1 - len(order), -len(order) if key else -1).flatten(-2 - key)


def _encode_pages(case, k, v):
    """K and V [pages, page, Hkv, D] as pages of the pool."""
    n, P, Hkv, D = k.shape
    (ck, sk, _), (cv, sv, _) = _quantise(k.float(), case["fmt"]), _quantise(v.float(), case["fmt"])
    parts = [x.transpose(1, 2).reshape(n, Hkv, P // 16, -1) for x in (_rows(ck, True), _rows(cv, False), sk, sv)]
    return torch.cat(parts, dim=3).reshape(n, -1)


def _magnitudes(dtype):
    return torch.tensor(MAGNITUDES + tuple(-x for x in MAGNITUDES), dtype=dtype, device="cuda")


def _tokens(case, pages, page, inside):
    """K and V values [B, L, Hkv, D] in 32 bits of the tokens [B, L] at `inside` of their pages."""
    Hkv, P, D = case["Hkv"], case["page"], case["D"]
    B, L = page.shape
    sb = D // (32 if case["fmt"] == "E2M1" else 16)
    groups = pages.view(pages.shape[0], Hkv, P // 16, 16 * (D + 2 * sb))
    m, i = _magnitudes(torch.float32), torch.arange(256, device="cuda")
    pairs = torch.stack((m[i & 15], m[i >> 4]), dim=1)
    got = []
    for at, scale_at, key in ((0, 16 * D, True), (8 * D, 16 * (D + sb), False)):
        codes = groups[..., at:at + 8 * D].unflatten(3, (16, D // 2))[page, :, inside // 16, inside % 16]
        scales = groups[..., scale_at:scale_at + 16 * sb].unflatten(3, (16, sb))[page, :, inside // 16, inside % 16]
        if key:                                             # bytes [t][s][h] -> [s][t][h]
            codes = codes.reshape(B, L, Hkv, 4, D // 16, 2).transpose(3, 4)
        else:                                               # bytes [g][i] -> [i][g]
            codes = codes.reshape(B, L, Hkv, 8, D // 16).transpose(3, 4)
        x = pairs[codes.reshape(B, L, Hkv, D // 2).int()].reshape(B, L, Hkv, sb, -1)
        s = _power(scales.int() - 127) if case["fmt"] == "E2M1" else scales.contiguous().view(torch.float8_e4m3fn).float()
        got.append((x * s[..., None]).reshape(B, L, Hkv, D))
    return got


# -------------------------------------------------------------------------------- one pass
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import softmax_mx_block_gb300 as fsa
    case = st["case"]
    cache = fsa.MxCache(st["pages"], case["page"], case["Hkv"], case["D"], case["fmt"])
    if case["op"] == "append":
        fsa.fsa_cache_append_rope(cache, st["q"], st["k"], st["v"], st["table"], st["lens"], st["news"], inv_freq=st["inv_freq"],
                                  q_weight=st["q_weight"], k_weight=st["k_weight"], norm=case["norm"], eps=1e-6,
                                  interleaved=case["interleaved"], q_out=st["q_out"])
        fsa.fsa_cache_read(cache, st["table"], st["lens"], start=st["first"], k_out=st["k_back"], v_out=st["v_back"])
        return {"q": st["q_out"], "k": st["k_back"], "v": st["v_back"]}
    attend = fsa.fsa_attention_chunk if case["op"] == "chunk" else fsa.fsa_attention_cache
    attend(st["q"], cache, st["table"], st["lens"], q_lens=st["news"], window=case["window"] or None, sinks=case["sinks"],
           scale=case["D"] ** -0.5, out=st["out"], lse=st["lse"])
    return {"out": st["out"], "lse": st["lse"]}


def _plain(st):
    return _written(st) if st["case"]["op"] == "append" else _attended(st)


def _written(st):
    case = st["case"]
    D, Hkv, P = case["D"], case["Hkv"], case["page"]
    at = torch.arange(case["S"], device="cuda")[None, :]
    live = at < st["news"][:, None]
    place = (st["first"][:, None] + at).clamp(max=case["longest"] - 1)
    angle = place.double()[:, :, None] * st["inv_freq"]
    cos, sin = angle.cos()[:, :, None], angle.sin()[:, :, None]
    q = _turned(st["q"].float(), st["q_weight"], cos.float(), sin.float(), case).to(torch.bfloat16)
    k = _turned(st["k"].double(), st["k_weight"], cos, sin, case)              # 64 bits: values next to a border
    sb = D // (32 if case["fmt"] == "E2M1" else 16)
    groups = st["pages"].view(st["pages"].shape[0], Hkv, P // 16, 16 * (D + 2 * sb))
    page = st["table"].gather(1, (place // P).long())[live].long()
    inside = (place % P)[live].long()
    values = []

    def put(x, code_at, scale_at, key):
        codes, scales, s = _quantise(x, case["fmt"])
        for first, width, rows in ((code_at, D // 2, _rows(codes[live], key)), (scale_at, sb, scales[live])):
            groups[..., first:first + 16 * width].unflatten(3, (16, width))[page, :, inside // 16, inside % 16] = rows
        v = _magnitudes(x.dtype)[codes.int()].reshape(*scales.shape, -1) * s[..., None]
        values.append(v.reshape(x.shape).to(torch.bfloat16))

    put(k, 0, 16 * D, True)
    put(st["v"].float(), 8 * D, 16 * (D + sb), False)
    live = live[:, :, None, None]
    return {"q": torch.where(live, q, st["q_out"]), "k": torch.where(live, values[0], st["k_back"]),
            "v": torch.where(live, values[1], st["v_back"])}


def _turned(x, weight, cos, sin, case):
    if case["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.to(x.dtype)
    r = case["rotary"]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., r:]), dim=-1)


def _attended(st):
    case = st["case"]
    B, Sq, H, Hkv, D, P, W, first = (case[n] for n in ("B", "Sq", "H", "Hkv", "D", "page", "window", "sinks"))
    G, L = H // Hkv, _width(case)
    # the keys taken up, by position: all, or the first ones and those that some row's window reaches
    j = torch.arange(L, device="cuda")[None, :]
    low = st["first"][:, None] - (W - 1) if W else torch.zeros_like(st["first"])[:, None]
    key = torch.where(j < first, j, low + j - first)
    there = (key >= 0) & (key < st["lens"][:, None]) & ((j < first) | (key >= first))
    key = torch.where(there, key, 0)
    page = st["table"].gather(1, (key // P).long()).clamp(min=0).long()
    k, v = (x.transpose(1, 2) for x in _tokens(case, st["pages"], page, (key % P).long()))      # [B, Hkv, L, D]
    q = st["q"].float().reshape(B, Sq, Hkv, G, D).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5)                          # [B, Hkv, Sq*G, L]
    row = torch.arange(Sq, device="cuda")[None, :]
    at = (st["first"][:, None] + row).repeat_interleave(G, dim=1)[:, :, None]      # a row's position
    seen = there[:, None, :] & (key[:, None, :] <= at)
    if W:
        seen &= (key[:, None, :] > at - W) | (key[:, None, :] < first)
    s.masked_fill_(~seen[:, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    o = o.reshape(B, Hkv, Sq, G, D).permute(0, 2, 1, 3, 4).reshape(B, Sq, H, D)
    live = row < st["news"][:, None]
    out = torch.where(live[:, :, None, None], o.to(torch.bfloat16), st["out"])
    if st["lse"] is None:
        return {"out": out, "lse": None}
    lse = (top + torch.log(total)).reshape(B, Hkv, Sq, G).permute(0, 2, 1, 3).reshape(B, Sq, H)
    return {"out": out, "lse": torch.where(live[:, :, None], lse, st["lse"])}


# ---------------------------------------------------------------- the definitions, 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st, case) if case["op"] == "append" else _exact_attention(st, case)


def _double_power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _binade(x):
    """The largest power of two that is not over x, as its exponent."""
    return torch.frexp(x).exponent - 1


def _exact_append(st, case):
    B, S, r, half = case["B"], case["S"], case["rotary"], case["rotary"] // 2
    got = {n: torch.zeros(B, S, case["H"] if n == "q" else case["Hkv"], case["D"], dtype=torch.float64, device="cuda") for n in "qkv"}
    for b, (n, m) in enumerate(zip(_lengths(case), st["news"].tolist())):
        for i in range(0, m, 4096):                         # positions in turn: the whole would be large
            rows = slice(i, min(m, i + 4096))
            at = (torch.arange(n - m, n, device="cuda")[rows]).double()
            for name in "qk":
                c = st[name][b, rows].double()
                if case["norm"]:
                    c = c / (c.pow(2).sum(-1, keepdim=True) / case["D"] + 1e-6).sqrt() * st[name + "_weight"].double()
                z = c.clone()
                for j in range(half):
                    one, two = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
                    t = (at * st["inv_freq"][j])[:, None]
                    z[..., one] = c[..., one] * t.cos() - c[..., two] * t.sin()
                    z[..., two] = c[..., two] * t.cos() + c[..., one] * t.sin()
                got[name][b, rows] = z if name == "q" else _exact_rounded(z, case["fmt"])
            got["v"][b, rows] = _exact_rounded(st["v"][b, rows].double(), case["fmt"])
    return got


def _exact_rounded(x, fmt):
    """The value that each element of x is cached as."""
    size = 32 if fmt == "E2M1" else 16
    b = x.unflatten(-1, (-1, size))
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


def _exact_sequence(st, case, b, length, head):
    """K and V [length, D] of one head of one sequence, element by element from the format's description."""
    D, P = case["D"], case["page"]
    size = 32 if case["fmt"] == "E2M1" else 16
    sb = D // size
    raw = st["pages"].view(-1, case["Hkv"], P // 16, 16 * (D + 2 * sb))[st["table"][b, :-(-length // P)].long(), head].flatten(0, 1)
    d = torch.arange(D, device="cuda")
    s, t, h = d // 16, d % 16 // 4, d % 4 // 2
    i, g = d // 16, d % 16 // 2
    mag = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
    got = []
    for at, scale_at, byte in ((0, 16 * D, t * (D // 8) + 2 * s + h), (8 * D, 16 * (D + sb), g * (D // 16) + i)):
        code = (raw[:, at:at + 8 * D].unflatten(1, (16, D // 2))[..., byte].int() >> (4 * (d % 2)).int()) & 15
        value = mag[(code & 7).long()] * (1.0 - 2.0 * (code >> 3).double())
        sc = raw[:, scale_at:scale_at + 16 * sb].unflatten(1, (16, sb)).int()
        if case["fmt"] == "E2M1":
            sc = _double_power(sc - 127)
        else:
            e, m = (sc >> 3) & 15, (sc & 7).double()
            sc = torch.where(e > 0, (8.0 + m) * _double_power(e - 10), m * 2.0 ** -9)
        got.append((value * sc[..., d // size]).reshape(-1, D)[:length])
    return got


def _exact_attention(st, case):
    B, Sq, H, Hkv, D, W = (case[n] for n in ("B", "Sq", "H", "Hkv", "D", "window"))
    out = torch.zeros(B, Sq, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, Sq, H, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(_lengths(case), st["news"].tolist())):
        for h in range(H):
            if h % (H // Hkv) == 0:
                k, v = _exact_sequence(st, case, b, n, h // (H // Hkv))
            for i in range(0, m, 2048):                     # rows in turn: the scores would be large
                c = min(2048, m - i)
                low = max(0, n - m + i + 1 - W) if W else 0
                keys = torch.cat((torch.arange(min(case["sinks"], low), device="cuda"), torch.arange(low, n, device="cuda")))
                p = (n - m + i + torch.arange(c, device="cuda"))[:, None]
                e = st["q"][b, i:i + c, h].double() @ k[keys].T / math.sqrt(D)
                hidden = keys > p
                if W:
                    hidden |= (keys <= p - W) & (keys >= case["sinks"])
                e[hidden] = -math.inf
                z = torch.logsumexp(e, dim=1)
                out[b, i:i + c, h] = torch.exp(e - z[:, None]) @ v[keys]
                lse[b, i:i + c, h] = z
    return {"out": out, "lse": lse if case["lse"] else None}
