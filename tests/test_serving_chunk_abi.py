"""Refusals of fsa_cache_append_rope, fsa_attention_chunk and the window of fsa_attention_cache before any
launch: the C ABI's checks on made-up pointers, the binding's on tensors, and the last shapes accepted."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import softmax_mx_block_gb300 as fsa  # noqa: E402
from softmax_mx_block_gb300 import _binding as b  # noqa: E402

BAD, FMT = fsa.FSA_ERR_INVALID_ARG, fsa.FSA_ERR_UNSUPPORTED_FMT
CACHE_BAD = [dict(pages=0), dict(pages=72), dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=24), dict(Hkv=0), dict(D=96),
             dict(fmt=0), dict(fmt=3)]


def strides(*v):
    return b.fsa_strides(*(v or (8 * 128, 4 * 128, 128)))


def cache(**kw):
    return b.fsa_cache(*(dict(pages=64, num_pages=4, page_size=16, Hkv=2, D=128, fmt=2) | kw).values())


def test_append_rope_refuses():
    def call(c=None, v=64, vs=None, table=64, width=5, lens=64, which=0, status=0, **kw):
        a = b.fsa_norm_rope(64, 64, 64, 0, strides(), strides(), strides(), strides(), 0, 0, 64, 64, 2, 3, 4, 2, 128, 128, 1,
                            (ctypes.c_int32 * 3)(64, 0, 0), 1, 0, 1e-6)
        for n, x in kw.items():
            setattr(a, n, x)
        c, vs = c or cache(), vs or strides()
        return fsa.load().fsa_cache_append_rope(ctypes.byref(a), ctypes.byref(c), v, ctypes.byref(vs), table, width, lens, which, status, None)

    sec = lambda *v: (ctypes.c_int32 * 3)(*v)  # noqa: E731
    for kw in CACHE_BAD:
        assert call(cache(**kw)) == (FMT if "fmt" in kw else BAD), kw
    for kw in (dict(q=0), dict(k=0), dict(k=8), dict(q_out=0), dict(q_out=72), dict(k_out=64), dict(v=0), dict(v=24), dict(q_weight=8), dict(pos=66),
               dict(inv_freq=0), dict(inv_freq=68), dict(B=0), dict(S=0), dict(H=0), dict(Hkv=0), dict(Hkv=3), dict(D=64), dict(D=96), dict(rotary=4),
               dict(rotary=136), dict(n_axes=0), dict(n_axes=4), dict(sections=sec(63, 0, 0)), dict(n_axes=3, pos=0, sections=sec(24, 20, 20)),
               dict(norm=2), dict(interleaved=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(norm=0, k_weight=64), dict(q_strides=strides(1, 512, 128)),
               dict(k_strides=strides(1024, 4, 128)), dict(vs=strides(-1024, 512, 128)), dict(q_out_strides=strides(1024, 0, 128)), dict(table=0),
               dict(table=66), dict(width=0), dict(width=(1 << 30) // 16 + 1), dict(lens=0), dict(lens=65), dict(which=2), dict(status=3),
               dict(B=1 << 20, S=1 << 20)):
        assert call(**kw) == BAD, kw
    f = fsa.load().fsa_cache_append_rope
    assert f(None, ctypes.byref(cache()), 64, ctypes.byref(strides()), 64, 5, 64, 0, 0, None) == BAD


@pytest.mark.parametrize("name,window", [("fsa_attention_chunk", 0), ("fsa_attention_chunk", 9), ("fsa_attention_cache_window", 9)])
def test_attention_refuses(name, window):
    f = getattr(fsa.load(), name)

    def call(c=None, window=window, sinks=0, **kw):
        c = c or cache()
        a = b.fsa_cache_attn(64, 64, 0, ctypes.pointer(c), 64, 64, 0, 64, 1 << 40, 0, strides(), strides(), 2, 4, 3, 5, 1, 1, 0.1, 0)
        for n, x in kw.items():
            setattr(a, n, x)
        return f(ctypes.byref(a), window, sinks, None)

    for kw in CACHE_BAD:
        assert call(cache(**kw)) == (FMT if "fmt" in kw else BAD), kw
    for kw in (dict(q=0), dict(q=72), dict(out=0), dict(out=8), dict(lse=2), dict(block_table=0), dict(lens=0), dict(q_lens=2), dict(workspace=8),
               dict(status=1), dict(B=0), dict(H=3), dict(H=0), dict(Sq=0), dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(causal=2),
               dict(out_dtype=2), dict(scale=float("inf")), dict(scale=float("nan")), dict(q_strides=strides(1024, 512, 4)),
               dict(out_strides=strides(1024, 512, 0)), dict(B=1 << 20, Sq=1 << 10), dict(window=-1), dict(sinks=-1), dict(window=9, causal=0)):
        assert call(**kw) == BAD, kw
    assert (call(window=0, sinks=1) == BAD) and f(None, window, 0, None) == BAD
    if name == "fsa_attention_cache_window":
        assert call(window=0) == BAD


def test_workspace_queries():
    n, lib = ctypes.c_size_t(), fsa.load()
    for v in ((0, 4, 1, 5), (1, 3, 1, 5), (1, 4, 0, 5), (1, 4, 1, 0), (1, 4, 1, 1 << 30)):
        assert lib.fsa_attention_chunk_workspace(ctypes.byref(cache()), *v, ctypes.byref(n)) == BAD
        assert lib.fsa_attention_cache_window_workspace(ctypes.byref(cache()), *v, 8, 0, ctypes.byref(n)) == BAD
    for w in ((0, 0), (-1, 0), (8, -1)):
        assert lib.fsa_attention_cache_window_workspace(ctypes.byref(cache()), 1, 4, 1, 5, *w, ctypes.byref(n)) == BAD
    assert lib.fsa_attention_chunk_workspace(ctypes.byref(cache(fmt=4)), 1, 4, 1, 5, ctypes.byref(n)) == FMT
    assert lib.fsa_attention_chunk_workspace(ctypes.byref(cache()), 1, 4, 1, 5, None) == BAD
    # B * Hkv * ceil(Sq * H/Hkv / 256) * (ceil(max_pages * page_size / 128) + 4) below 2^31, and at it
    ok = (fsa.FSA_OK, fsa.FSA_ERR_NO_DEVICE)
    one = cache(Hkv=1, page_size=128)
    assert lib.fsa_attention_chunk_workspace(ctypes.byref(one), 1 << 16, 1, 1, (1 << 15) - 5, ctypes.byref(n)) in ok
    assert lib.fsa_attention_chunk_workspace(ctypes.byref(one), 1 << 16, 1, 257, (1 << 14) - 4, ctypes.byref(n)) == BAD


def test_binding_refuses():
    x = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    n = fsa.fsa_cache_page_bytes(16, 4, 128, "E2M1")
    c = fsa.MxCache(torch.zeros(3, n, dtype=torch.uint8), 16, 4, 128, "E2M1")
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fsa.fsa_cache_append_rope(c, x, x, x, i[None], i), lambda: fsa.fsa_attention_chunk(x, c, i[None], i),
                 lambda: fsa.fsa_attention_cache(x, c, i[None], i, window=4)):
        with pytest.raises(fsa.FsaError, match="CUDA tensor"):
            call()
    with pytest.raises(fsa.FsaError):
        fsa.fsa_attention_chunk(x, c, i[None], i, out=torch.zeros_like(x), out_dtype="f32")
