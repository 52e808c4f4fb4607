"""Refusals of the serving entry points before any launch: the C ABI's argument checks on
made-up pointers, the binding's checks on tensors, and the page layout's sizes."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import softmax_mx_block_gb300 as fsa  # noqa: E402
from softmax_mx_block_gb300 import _binding as b  # noqa: E402

OK_STRIDES = (8 * 128, 4 * 128, 128)


@pytest.fixture(scope="module")
def lib():
    return fsa.load()


def strides(*v):
    return b.fsa_strides(*(v or OK_STRIDES))


def cache(**kw):
    return b.fsa_cache(*(dict(pages=64, num_pages=4, page_size=16, Hkv=2, D=128, fmt=2) | kw).values())


@pytest.mark.parametrize("page,Hkv,D,fmt,want", [(16, 1, 128, 2, 16 * 136), (64, 8, 128, 5, 64 * 8 * 144),
                                                 (32, 2, 64, 2, 32 * 2 * 68), (1024, 1, 64, 5, 1024 * 72)])
def test_page_bytes(lib, page, Hkv, D, fmt, want):
    assert fsa.fsa_cache_page_bytes(page, Hkv, D, fmt) == want


@pytest.mark.parametrize("page,Hkv,D,fmt,want", [(8, 1, 128, 2, -1), (48, 1, 128, 2, -1), (2048, 1, 128, 2, -1), (16, 0, 128, 2, -1),
                                                 (16, 1, 96, 2, -1), (16, 1, 128, 0, -2), (16, 1, 128, 3, -2)])
def test_page_bytes_refuses(lib, page, Hkv, D, fmt, want):
    with pytest.raises(fsa.FsaError) as e:
        fsa.fsa_cache_page_bytes(page, Hkv, D, fmt)
    assert e.value.status == want


CACHE_BAD = [dict(pages=0), dict(pages=72), dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=24), dict(Hkv=0),
             dict(D=96), dict(fmt=0), dict(fmt=3)]


@pytest.mark.parametrize("fn", ["fsa_cache_append", "fsa_cache_read"])
def test_cache_io_refuses(lib, fn):
    f = getattr(lib, fn)

    def call(c=None, k=64, v=64, ks=None, vs=None, B=2, S=3, table=64, width=5, lens=64, which=0, status=0):
        c, ks, vs = c or cache(), ks or strides(), vs or strides()
        return f(ctypes.byref(c), k, v, ctypes.byref(ks), ctypes.byref(vs), B, S, table, width, lens, which, status, None)

    for kw in CACHE_BAD:
        assert call(c=cache(**kw)) == (fsa.FSA_ERR_UNSUPPORTED_FMT if "fmt" in kw else fsa.FSA_ERR_INVALID_ARG), kw
    for kw in (dict(k=8), dict(v=24), dict(B=0), dict(S=-1), dict(table=0), dict(table=66), dict(width=0),
               dict(width=(1 << 30) // 16 + 1), dict(lens=0), dict(lens=65), dict(which=2), dict(status=3),
               dict(ks=strides(1024, 4, 128)), dict(vs=strides(-1024, 512, 128)), dict(B=1 << 30, S=1 << 30)):
        assert call(**kw) == fsa.FSA_ERR_INVALID_ARG, kw
    assert f(None, 64, 64, None, None, 1, 1, 64, 1, 64, 0, 0, None) == fsa.FSA_ERR_INVALID_ARG
    assert call(k=0, v=0) == fsa.FSA_ERR_INVALID_ARG
    if fn == "fsa_cache_append":
        assert call(v=0) == fsa.FSA_ERR_INVALID_ARG
    else:
        assert call(ks=strides(1024, 0, 128)) == fsa.FSA_ERR_INVALID_ARG     # rows of an output on one another


def test_norm_rope_refuses(lib):
    def call(**kw):
        a = b.fsa_norm_rope(64, 64, 64, 64, strides(), strides(), strides(), strides(), 0, 0, 64, 64, 2, 3, 4, 2, 128, 128,
                            1, (ctypes.c_int32 * 3)(64, 0, 0), 1, 0, 1e-6)
        for n, x in kw.items():
            setattr(a, n, x)
        return lib.fsa_qk_norm_rope(ctypes.byref(a), None)

    sec = lambda *v: (ctypes.c_int32 * 3)(*v)  # noqa: E731
    for kw in (dict(q=0), dict(k=8), dict(q_out=0), dict(k_out=72), dict(q_weight=8), dict(pos=0), dict(pos=66),
               dict(inv_freq=0), dict(inv_freq=68), dict(B=0), dict(S=0), dict(H=0), dict(Hkv=0), dict(D=96), dict(rotary=4),
               dict(rotary=136), dict(rotary=-8), dict(n_axes=0), dict(n_axes=4), dict(sections=sec(63, 0, 0)),
               dict(n_axes=3, sections=sec(65, -1, 0)), dict(norm=2), dict(interleaved=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(norm=0, q_weight=64), dict(q_strides=strides(1, 512, 128)),
               dict(k_out_strides=strides(1024, 0, 128)), dict(B=1 << 20, S=1 << 20)):
        assert call(**kw) == fsa.FSA_ERR_INVALID_ARG, kw
    assert lib.fsa_qk_norm_rope(None, None) == fsa.FSA_ERR_INVALID_ARG


def test_attention_cache_refuses(lib):
    def call(c=None, **kw):
        c = c or cache()
        a = b.fsa_cache_attn(64, 64, 0, ctypes.pointer(c), 64, 64, 0, 64, 1 << 40, 0, strides(), strides(), 2, 4, 3, 5, 1, 1,
                             0.1, 0)
        for n, x in kw.items():
            setattr(a, n, x)
        return lib.fsa_attention_cache(ctypes.byref(a), None)

    for kw in CACHE_BAD:
        assert call(cache(**kw)) == (fsa.FSA_ERR_UNSUPPORTED_FMT if "fmt" in kw else fsa.FSA_ERR_INVALID_ARG), kw
    for kw in (dict(q=0), dict(q=72), dict(out=0), dict(out=8), dict(lse=2), dict(block_table=0), dict(lens=0), dict(q_lens=2),
               dict(workspace=8), dict(status=1), dict(B=0), dict(H=3), dict(H=0), dict(Sq=0),
               dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(causal=2), dict(out_dtype=2),
               dict(scale=float("inf")), dict(scale=float("nan")), dict(q_strides=strides(1024, 512, 4)),
               dict(out_strides=strides(1024, 512, 0)), dict(B=1 << 20, Sq=1 << 10)):
        assert call(**kw) == fsa.FSA_ERR_INVALID_ARG, kw
    assert lib.fsa_attention_cache(None, None) == fsa.FSA_ERR_INVALID_ARG
    n = ctypes.c_size_t()
    for v in ((0, 4, 1, 5), (1, 3, 1, 5), (1, 4, 0, 5), (1, 4, 1, 0), (1, 4, 1, 1 << 30)):
        assert lib.fsa_attention_cache_workspace(ctypes.byref(cache()), *v, ctypes.byref(n)) == fsa.FSA_ERR_INVALID_ARG
    assert lib.fsa_attention_cache_workspace(ctypes.byref(cache(fmt=4)), 1, 4, 1, 5, ctypes.byref(n)) == fsa.FSA_ERR_UNSUPPORTED_FMT
    assert lib.fsa_attention_cache_workspace(ctypes.byref(cache()), 1, 4, 1, 5, None) == fsa.FSA_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(lib):
    x = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    n = fsa.fsa_cache_page_bytes(16, 4, 128, "E2M1")
    c = fsa.MxCache(torch.zeros(3, n, dtype=torch.uint8), 16, 4, 128, "E2M1")
    i = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: fsa.fsa_qk_norm_rope(x, x, None, None), lambda: fsa.fsa_cache_append(c, x, x, i[None], i),
                 lambda: fsa.fsa_cache_read(c, i[None], i, 2), lambda: fsa.fsa_attention_cache(x, c, i[None], i)):
        with pytest.raises(fsa.FsaError, match="CUDA tensor"):
            call()
