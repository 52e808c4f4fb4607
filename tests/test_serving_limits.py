"""The serving calls take what their header says they take, to the last shape: seen by the
workspace query, which launches nothing (without a device its answer is that there is none)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import softmax_mx_block_gb300 as fsa  # noqa: E402
from softmax_mx_block_gb300 import _binding as b  # noqa: E402


def workspace(B, H, Sq, max_pages, Hkv, page_size=16):
    c, n = b.fsa_cache(64, 4, page_size, Hkv, 64, fsa.FSA_FMT_E2M1), ctypes.c_size_t()
    return fsa.load().fsa_attention_cache_workspace(ctypes.byref(c), B, H, Sq, max_pages, ctypes.byref(n))


@pytest.mark.parametrize("B,H,Sq", [(256, 32, 16384), (1, 1, 1 << 27), (1 << 27, 1, 1), (1, 1 << 14, 1 << 13), (3, 7, (1 << 27) // 21)])
def test_rows_up_to_the_limit(B, H, Sq):
    Hkv = H if H < 4 else 1
    assert workspace(B, H, Sq, 1, Hkv) in (fsa.FSA_OK, fsa.FSA_ERR_NO_DEVICE)
    assert workspace(B, H, Sq + 1, 1, Hkv) == fsa.FSA_ERR_INVALID_ARG


def test_tiles_up_to_the_limit():
    # B * Hkv * (Sq * H/Hkv / 8 + 1) * (max_pages * page_size / 32 + 9) below 2^31, and at it
    assert workspace((1 << 27) - 1, 1, 1, 15, 1) in (fsa.FSA_OK, fsa.FSA_ERR_NO_DEVICE)
    assert workspace(1 << 27, 1, 1, 15, 1) == fsa.FSA_ERR_INVALID_ARG


def test_heads_up_to_the_limit():
    assert fsa.fsa_cache_page_bytes(16, 65535, 64, "E2M1") == 16 * 65535 * 68
    assert workspace(1, 65535, 1, 1, 65535) in (fsa.FSA_OK, fsa.FSA_ERR_NO_DEVICE)
    with pytest.raises(fsa.FsaError) as e:
        fsa.fsa_cache_page_bytes(16, 65536, 64, "E2M1")
    assert e.value.status == fsa.FSA_ERR_INVALID_ARG
    assert workspace(1, 65536, 1, 1, 65536) == fsa.FSA_ERR_INVALID_ARG
