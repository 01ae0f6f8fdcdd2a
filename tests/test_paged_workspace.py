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


@pytest.fixture
def recorded(monkeypatch):
    """The binding on CPU tensors: every library call is handed to `calls.hook` instead (name, scratch, its bytes)."""
    from types import SimpleNamespace
    from chunked_recurrence_gb300 import paged
    calls = SimpleNamespace(hook=None)

    def entry(name):
        return lambda *a: calls.hook(name, a[-3], a[-2]) or 0
    for name, to in (("_entry", entry), ("_need_cuda", lambda *t: None), ("_handle", lambda t, stream: 0), ("_plans", {}),
                     ("_status_words", lambda index: 0x1000)):
        monkeypatch.setattr(paged, name, to)
    return calls


def _a_call(kind, big):
    import torch
    import chunked_recurrence_gb300 as crg
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    if kind == "attn":
        cache, n = torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16), 300 if big else 2
        q = torch.zeros(n, 4, 128, dtype=torch.bfloat16)
        return lambda: crg.gdn_paged_attn(q, cache, cache, i32(n, 4), i32(n), max_new=n)
    rows, pages = (50, 900) if big else (5, 8)
    tables = (i32(rows, 4), i32(rows), i32(pages))
    return {"free": lambda: crg.gdn_pages_free(*tables, i32(2), 16),
            "grow": lambda: crg.gdn_pages_grow(*tables, i32(2), i32(2), 16),
            "fork": lambda: crg.gdn_pages_fork(*tables, i32(2), i32(2), [i32(pages, 4)], 16),
            "compact": lambda: crg.gdn_pages_compact(*tables, [i32(pages, 4)], 16)}[kind]


@pytest.mark.parametrize("kind", ["attn", "grow", "free", "fork", "compact"])
def test_no_call_brings_scratch_of_another(lib, recorded, kind):
    """The binding holds no scratch: a second thread's call, between a first one's launches, must not write to the
    first one's, nor a later call let go of what a graph was captured with."""
    seen = []
    recorded.hook = lambda name, buf, nbytes: seen.append((buf, nbytes))
    for big in (False, True, False):
        _a_call(kind, big)()
    assert [b for b, _ in seen] == [None] * 3  # the call's own, from the allocator
    small, large, again = (n for _, n in seen)
    assert 256 <= small == again < large
