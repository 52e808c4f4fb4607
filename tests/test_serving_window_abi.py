"""The workspace query of a window takes the numbers that the call itself takes."""
import pytest

torch = pytest.importorskip("torch")

import softmax_mx_block_gb300 as fsa  # noqa: E402

LARGE = [(2 ** 31, 0), (2 ** 32, 4), (2 ** 32 + 5, 0), (2 ** 40, 2 ** 40), (9, 2 ** 32), (9, 2 ** 31)]


def query(cache, window, sinks):
    """The bytes, or the error's status."""
    try:
        return fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, 4096, window=window, sinks=sinks)
    except fsa.FsaError as e:
        return f"status {e.status}"


@pytest.mark.parametrize("window,sinks", LARGE)
def test_windows_beyond_32_bits(window, sinks):
    """As the call does, larger numbers count as the largest (without a GPU: the same answer as for that one)."""
    page = fsa.fsa_cache_page_bytes(16, 4, 128, "E2M1")
    cache = fsa.MxCache(torch.zeros(3, page, dtype=torch.uint8), 16, 4, 128, "E2M1")
    most = 2 ** 31 - 1
    assert query(cache, window, sinks) == query(cache, min(window, most), min(sinks, most))
    for w, s in ((-2 ** 32 + 5, 0), (-2 ** 31 - 1, 0), (9, -2 ** 32), (0, 0), (None, 2 ** 32)):
        assert query(cache, w, s) == f"status {fsa.FSA_ERR_INVALID_ARG}", (w, s)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", LARGE)
def test_the_call_takes_the_workspace_of_the_query(window, sinks):
    page = fsa.fsa_cache_page_bytes(16, 4, 128, "E2M1")
    cache = fsa.MxCache(torch.zeros(3, page, dtype=torch.uint8, device="cuda"), 16, 4, 128, "E2M1")
    q = torch.ones(2, 1, 16, 128, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 4096, dtype=torch.int32, device="cuda")
    lens = torch.tensor([7, 900], dtype=torch.int32, device="cuda")
    ws = torch.empty(fsa.fsa_attention_cache_workspace(cache, 2, 16, 1, 4096, window, sinks), dtype=torch.uint8, device="cuda")
    got = fsa.fsa_attention_cache(q, cache, table, lens, window=window, sinks=sinks, workspace=ws)
    assert torch.equal(got, fsa.fsa_attention_cache(q, cache, table, lens, window=window, sinks=sinks))
