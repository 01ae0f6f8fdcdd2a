"""Where the paged calls keep their status and scratch, on the CPU: nothing is launched."""
import ctypes

import pytest

P = ctypes.c_void_p
FAKE, WS = P(0x10000), P(0x20000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from chunked_recurrence_gb300 import build as b
    b.build()
    import chunked_recurrence_gb300 as crg
    return crg.load()


def test_status_words_are_words(lib):
    import chunked_recurrence_gb300 as crg
    assert lib.gdn_status_words(None) == 1
    for status in (0x1001, 0x1002):
        sh = crg.GdnCacheShape(n_seqs=2, n_tok=2, Hq=4, Hkv=2, D=128, dtype=1, page_size=16, n_pages=10, max_pages=5,
                               status=status)
        assert lib.gdn_paged_attn(FAKE, FAKE, FAKE, FAKE, FAKE, None, ctypes.byref(sh), 1, 0.1, 0, 0, FAKE, None, WS,
                                  1 << 40, None) == 1
        assert lib.gdn_kv_append(None, FAKE, FAKE, None, None, 0, 1.0, 0, FAKE, FAKE, None, ctypes.byref(sh), None, FAKE,
                                 FAKE, WS, 256, None) == 1
        t = crg.GdnPageTables(page_table=0x1000, seq_lens=0x2000, refs=0x3000, n_rows=4, max_pages=8, n_pages=32,
                              page_size=16, status=status)
        assert lib.gdn_pages_free(ctypes.byref(t), FAKE, 2, WS, 1 << 20, None) == 1
