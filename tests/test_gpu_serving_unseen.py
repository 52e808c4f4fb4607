"""Keys that no row sees, before a window and behind the first tokens: their pages are not looked up, and neither these
nor their tokens change a bit."""
import pytest

from test_gpu_serving import _fsa, filled_cache, gen, i32, normal

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

WINDOWS = [(700, 4), (333, 1), (50, 17), (129, 0), (16, 33), (1, 4), (401, 200)]      # and first tokens
LENS = [2100, 1507, 333, 40]


def unseen(n, rows, window, sinks):
    """The keys [first, last) between the first tokens and the first row's window."""
    return sinks, max(sinks, n - rows + 1 - window)


def check_pages(call, shapes, page, fmt, D):
    """Pages without a key that some row sees, as holes and as another sequence's pages (far scales, NaN, zeros)."""
    fsa = _fsa()
    g = gen(page + D)
    cache, table, _, _ = filled_cache(fsa, g, LENS, page, 2, D, fmt)
    pool = torch.cat((cache.pages, torch.zeros_like(cache.pages[:1])))
    other = fsa.MxCache(pool, page, 2, D, fmt)
    for Sq, G in shapes:
        q = normal(g, len(LENS), Sq, 2 * G, D)
        for window, sinks in WINDOWS:
            def run(cache, table, status=None):
                lse = torch.zeros(len(LENS), Sq, 2 * G, device="cuda")
                return call(q, cache, table, i32(LENS), window=window, sinks=sinks, lse=lse, status=status), lse

            want, status, holes, n_holes = run(cache, table), i32([0]), table.clone(), 0
            for b, n in enumerate(LENS):
                first, last = unseen(n, Sq, window, sinks)
                first, last = -(-first // page), last // page
                n_holes += max(0, last - first)
                holes[b, first:max(first, last)] = -1
            assert n_holes > 0
            got = run(cache, holes, status)
            assert int(status) == 0, (Sq, window, sinks)
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]), (Sq, window, sinks)
            foreign = torch.where((holes == -1) & (table >= 0), pool.shape[0] - 1, table).to(torch.int32)
            for byte in (0x60, 0xFF, 0x00):
                pool[-1] = byte
                got = run(other, foreign, status)
                assert int(status) == 0
                assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]), (Sq, window, sinks, byte)
            # a page that one row sees one key of is still asked for
            for b, at in ((0, LENS[0] - Sq + 1 - window), (1, LENS[1] - 1), (0, sinks - 1)):
                if at >= 0:
                    hole = holes.clone()
                    hole[b, at // page] = -1
                    status.zero_()
                    run(cache, hole, status)
                    assert int(status) == fsa.FSA_ERR_INVALID_ARG, (Sq, window, sinks, at)
            status.zero_()


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("fmt,D", [("E2M1", 128), ("NVFP4", 64)])
def test_pages_of_few_rows(fmt, D, page):
    """One row and several, in one block of rows and in three."""
    check_pages(_fsa().fsa_attention_cache, [(1, 4), (5, 1), (9, 4)], page, fmt, D)


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("fmt,D", [("E2M1", 128), ("NVFP4", 64)])
def test_pages_of_chunks(fmt, D, page):
    """Rows of one block, of two tiles, and of three blocks."""
    check_pages(_fsa().fsa_attention_chunk, [(5, 4), (40, 4), (150, 4)], page, fmt, D)


@pytest.mark.parametrize("name", ["fsa_attention_cache", "fsa_attention_chunk"])
@pytest.mark.parametrize("fmt", ["E2M1", "NVFP4"])
def test_tokens_beside_the_seen_ones(fmt, name):
    """Tokens that no row sees, on the pages of seen ones: far scales, zeros, NaN."""
    fsa = _fsa()
    call, g, page, D = getattr(fsa, name), gen(5), 64, 128
    cache, table, k, v = filled_cache(fsa, g, LENS, page, 2, D, fmt)
    for Sq in (1, 6):
        q = normal(g, len(LENS), Sq, 4, D)
        for window, sinks in WINDOWS:
            fsa.fsa_cache_append(cache, k, v, table, i32(LENS), i32(LENS))
            want = call(q, cache, table, i32(LENS), window=window, sinks=sinks)
            for what in (2.0 ** 60, 2.0 ** -40, 0.0, float("nan")):
                k2, v2 = k.clone(), v.clone()
                for b, n in enumerate(LENS):
                    part = slice(*unseen(n, Sq, window, sinks))
                    k2[b, part] *= what
                    v2[b, part] *= what
                fsa.fsa_cache_append(cache, k2, v2, table, i32(LENS), i32(LENS))
                assert torch.equal(want, call(q, cache, table, i32(LENS), window=window, sinks=sinks)), (Sq, window, sinks, what)
