"""gdn_pages_evict's refusals on the CPU: sizes whose places would not fit 32 bits."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE, WS = P(0x10000), P(0x20000)  # never dereferenced
MOST = 2 ** 31 - 2 ** 14


@pytest.fixture(scope="module")
def crg():
    from chunked_recurrence_gb300 import build as b
    b.build()
    import chunked_recurrence_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("mass_len,max_keep,status", [
    (2 ** 31 - 1, 10, 2), (MOST + 1, 10, 2), (100, 2 ** 31 - 1, 2), (100, MOST + 1, 2), (MOST, 10, 0), (100, MOST, 0)])
def test_lists_past_32_bits(crg, mass_len, max_keep, status):
    """A thread's place in a list goes up to 8191 past its end.  (With no rows listed a call that is not refused does nothing.)"""
    lib = crg.load()
    t = crg.GdnPageTables(page_table=0x1000, seq_lens=0x1000, refs=0x1000, n_rows=4, max_pages=8, n_pages=20, page_size=16)
    h = crg.GdnPageHeads(mass=0x1000, n_layers=1, heads=1, mass_len=mass_len, row_bytes=32)
    p = crg.GdnPagePools(pools=None, n_pools=0, page_bytes=512, page_stride=512)
    assert lib.gdn_pages_evict(ctypes.byref(t), FAKE, FAKE, 0, max_keep, 2, ctypes.byref(h), ctypes.byref(p), None, WS, 1 << 62,
                               None) == status
