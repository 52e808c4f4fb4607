"""Attention over the cache in 64 bits with a sliding window and first tokens that stay visible,
and what the tests' error bounds need of it: torch on the tensors' own device, nothing of the library."""
import math

import torch

import serving_ref as ref


def seen_keys(length, q_len, causal, window, sinks, device):
    """[q_len, length]: whether row i sees key j."""
    j = torch.arange(length, device=device)[None, :]
    p = (length - q_len + torch.arange(q_len, device=device))[:, None]
    if not causal:
        return torch.ones(q_len, length, dtype=torch.bool, device=device)
    seen = j <= p
    if window:
        seen = seen & ((j > p - window) | (j < sinks))
    return seen


def attention(q, k, v, live, causal, scale, window=0, sinks=0):
    """q [rows, H, D], k and v [length, Hkv, D] (fp64), live [length]: out, lse, and for bounds
    sum p|v| / sum p and the largest scale * sum |q||k| of the keys a row sees."""
    rows, H, D = q.shape
    length, Hkv = k.shape[:2]
    G = H // Hkv
    seen = seen_keys(length, rows, causal, window, sinks, q.device) & live[None, :]
    out = torch.zeros(rows, H, D, dtype=torch.float64, device=q.device)
    lse = torch.full((rows, H), -math.inf, dtype=torch.float64, device=q.device)
    spread, reach = torch.zeros_like(out), torch.zeros_like(lse)
    if length == 0 or rows == 0:
        return out, lse, spread, reach
    some = seen.any(-1)
    for h in range(H):
        qh, kh, vh = q[:, h].double(), k[:, h // G], v[:, h // G]
        s = torch.where(seen, qh @ kh.T * scale, -math.inf)
        top = torch.where(some, s.amax(-1), 0.0)
        p = torch.where(seen, torch.exp(s - top[:, None]), 0.0)
        total = torch.where(some, p.sum(-1), 1.0)
        out[:, h] = torch.where(some[:, None], p @ vh / total[:, None], 0.0)
        lse[:, h] = torch.where(some, top + torch.log(total), -math.inf)
        spread[:, h] = p @ vh.abs() / total[:, None]
        reach[:, h] = torch.where(seen, qh.abs() @ kh.abs().T * abs(scale), 0.0).amax(-1)
    return out, lse, spread, reach


def sequences(cache, table, lens, Hkv, D, fmt):
    """fp64 K, V and which tokens lie on pages of the pool, of each sequence."""
    got = []
    for b, n in enumerate(lens):
        k, v, live = ref.sequence(cache.pages, table[b], n, cache.page_size, Hkv, D, fmt)
        zero = live[:, None, None]
        got.append((torch.where(zero, k, 0.0), torch.where(zero, v, 0.0), live))
    return got
