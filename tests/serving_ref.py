"""Plain 64-bit forms of the serving operators (include/fsa.h), element by element from
their definitions, for the tests: torch on the tensors' own device, nothing of the library."""
import math

import torch

MAG = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"E2M1": 32, "NVFP4": 16}


def pow2(e):
    """2^e in fp64 for a tensor of whole numbers within -1022..1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantise(x, fmt):
    """(codes, scale bytes) of x [..., D]: blocks along D, round to nearest even, saturating."""
    b = x.double().unflatten(-1, (-1, BLOCK[fmt]))
    finite = torch.isfinite(b).all(-1)
    top = torch.where(finite[..., None], b.abs(), 0.0).amax(-1)
    if fmt == "E2M1":
        e = torch.where(top > 0, torch.frexp(top.clamp(min=2.0 ** -1000)).exponent - 3, -127).clamp(-127, 127)
        scale, byte = pow2(e), torch.where(finite, e + 127, 255)
    else:
        t = (top / 6).clamp(max=448.0)
        ex = (torch.frexp(t.clamp(min=2.0 ** -6)).exponent - 1).clamp(min=-6)
        n = torch.round(t / pow2(ex - 3))                      # 8..16 of 2^(ex-3), or 0..8 when subnormal
        scale = n * pow2(ex - 3)
        byte = torch.where(scale < 2.0 ** -6, n, (ex + 7) * 8 + n - 8)      # n = 16 carries into the exponent
        byte = torch.where(finite, byte.long(), 0x7F)
    y = torch.where((scale > 0)[..., None] & finite[..., None], b / scale[..., None].clamp(min=2.0 ** -200), 0.0)
    a = y.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    sign = torch.signbit(b) & finite[..., None] & (scale > 0)[..., None]
    return (code + 8 * sign).flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def scale_values(byte, fmt):
    byte = byte.long()
    if fmt == "E2M1":
        return torch.where(byte == 255, math.nan, pow2(byte - 127))
    e, m = byte >> 3 & 15, (byte & 7).double()
    return torch.where(byte == 0x7F, math.nan, torch.where(e > 0, (8 + m) * pow2(e - 10), m * 2.0 ** -9))


def values(codes, byte, fmt):
    """fp64 values of codes [..., D] under scale bytes [..., D/block]."""
    m = torch.tensor(MAG, dtype=torch.float64, device=codes.device)[(codes & 7).long()]
    v = torch.where((codes & 8) > 0, -m, m).unflatten(-1, (-1, BLOCK[fmt]))
    return (v * scale_values(byte, fmt)[..., None]).flatten(-2)


def rounded(x, fmt):
    return values(*quantise(x, fmt), fmt)


def unpack_pages(pages, page_size, Hkv, D, fmt):
    """Codes and scale bytes of a pool: k_codes [pages, page, Hkv, D], k_scales, v_codes, v_scales."""
    n, sb = pages.shape[0], D // BLOCK[fmt]
    g = pages.reshape(n, Hkv, page_size // 16, 16 * (D + 2 * sb))
    d = torch.arange(D, device=pages.device)
    kbyte = (d % 16 // 4) * (D // 8) + 2 * (d // 16) + d % 4 // 2
    vbyte = (d % 16 // 2) * (D // 16) + d // 16
    out = []
    for at, sat, byte in ((0, 16 * D, kbyte), (8 * D, 16 * (D + sb), vbyte)):
        rows = g[..., at:at + 8 * D].unflatten(3, (16, D // 2))[..., byte]
        codes = (rows >> (4 * (d % 2)).to(torch.uint8)) & 15
        out += [codes, g[..., sat:sat + 16 * sb].unflatten(3, (16, sb))]
    return [x.flatten(2, 3).transpose(1, 2) for x in out]


def sequence(pages, table_row, length, page_size, Hkv, D, fmt):
    """fp64 K and V [length, Hkv, D] of one sequence; a bad page's tokens are NaN."""
    need = -(-length // page_size)
    ids = table_row[:need].long()
    good = (ids >= 0) & (ids < pages.shape[0])
    kc, ks, vc, vs = unpack_pages(pages[ids.clamp(0, pages.shape[0] - 1)], page_size, Hkv, D, fmt)
    live = good.repeat_interleave(page_size)[:length]
    k, v = (values(c.flatten(0, 1), s.flatten(0, 1), fmt)[:length] for c, s in ((kc, ks), (vc, vs)))
    return k, v, live


def attention(q, k, v, live, length, q_len, causal, scale):
    """fp64 attention of one sequence: q [q_len, H, D], k, v [length, Hkv, D].  Returns
    out, lse and, per row and head, what error bounds need: sum p|v| [.., D], sum |q||k|
    max over seen keys, and the number of seen keys."""
    H, D = q.shape[1:]
    Hkv = k.shape[1]
    G = H // Hkv
    q = q.double()
    pos = torch.arange(length, device=q.device)
    row = torch.arange(q_len, device=q.device)
    seen = live[None, :] & ((pos[None, :] <= (length - q_len + row)[:, None]) if causal else torch.ones_like(pos[None, :], dtype=torch.bool))
    kh, vh = k.repeat_interleave(G, dim=1), v.repeat_interleave(G, dim=1)
    s = torch.einsum("ihd,lhd->ihl", q, kh) * scale
    s = torch.where(seen[:, None, :], s, -math.inf)
    some = seen.any(-1)[:, None]
    top = torch.where(some, s.amax(-1) if length else torch.zeros_like(some, dtype=torch.float64), 0.0)
    p = torch.where(seen[:, None, :], torch.exp(s - top[..., None]), 0.0)
    total = p.sum(-1)
    vz = torch.where(live[:, None, None], vh, 0.0)
    mul = lambda w, x: torch.einsum("ihl,lhd->ihd", w, x)  # noqa: E731
    # 0 * NaN of keys that a row does not see must not count: zero NaN V there, add them back where seen
    nan = torch.isnan(vz)
    o = mul(p, torch.where(nan, 0.0, vz))
    o = torch.where(mul(seen[:, None, :].double().expand_as(p), nan.double()) > 0, math.nan, o)
    div = torch.where(total > 0, total, 1.0)[..., None]
    out = torch.where(some[..., None], o / div, 0.0)
    lse = torch.where(some, top + torch.log(torch.where(some, total, 1.0)), -math.inf)
    spread = mul(p, torch.where(nan, 0.0, vz).abs()) / div
    kz = torch.where(torch.isnan(kh), 0.0, kh).abs()
    reach = torch.einsum("ihd,lhd->ihl", q.abs(), kz) * abs(scale)
    reach = torch.where(seen[:, None, :], reach, 0.0).amax(-1) if length else torch.zeros_like(top)
    return out, lse, spread, reach, total


def norm_rope(x, weight, pos, inv_freq, sections, norm, eps, interleaved):
    """fp64 norm and rotation of x [B,S,H,D]; also |a| + |b| of each element's pair (for bounds)."""
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    out, size = y.clone(), y.abs()
    half = 0 if inv_freq is None else inv_freq.numel()
    i = 0
    for axis, count in enumerate(sections):
        for j in range(i, i + count):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
            t = (pos[:, :, axis].double() * inv_freq[j])[:, :, None]
            out[..., a] = y[..., a] * torch.cos(t) - y[..., b] * torch.sin(t)
            out[..., b] = y[..., a] * torch.sin(t) + y[..., b] * torch.cos(t)
            size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
        i += count
    return out, size
