"""The paged cache on the CPU: the index arithmetic that the kernels use, compiled for the host;
the frequencies of the rotary step; and the refusals of every entry point (nothing is launched)."""
import ctypes
import math
import os
import random
import subprocess
from fractions import Fraction

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("paged") / "paged_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-static-libubsan", "-I", os.path.join(ROOT, "chunked_recurrence_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "host_emulation", "paged_host.cpp")], check=True)
    lib = ctypes.CDLL(so)
    lib.host_slots.restype = lib.host_share.restype = ctypes.c_int64
    lib.host_slots.argtypes = [ctypes.c_int64] + [ctypes.c_int32] * 3
    lib.host_share.argtypes = [ctypes.c_int64] + [ctypes.c_int32] * 2
    return lib


def _i32(a):
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _item(host, lens, cu, n_tok, most, slot, G, R, KT, window):
    la, lp = _i32(lens)
    ca, cp = _i32(cu) if cu is not None else (None, None)
    out = (ctypes.c_int32 * 11)()
    host.host_item(lp, cp, len(lens), n_tok, most, slot, G, R, KT, window, out)
    return dict(zip("s t0 first row0 rows lo hi tile0 n_tiles ok units".split(), out))


@pytest.mark.parametrize("G,R", [(1, 128), (3, 128), (4, 256), (8, 256), (7, 4), (300, 128), (1, 4)])
@pytest.mark.parametrize("window", [0, 1, 130])
def test_items_cover_every_row_once(host, G, R, window):
    """Every query row lies in exactly one slot, and an item's positions and tiles hold what its rows see."""
    rng = random.Random(G * 1000 + R + window)
    for _ in range(12):
        n = rng.randint(1, 9)
        new = [rng.choice([0, 0, 1, 1, rng.randint(1, 300)]) for _ in range(n)]
        lens = [max(0, k + rng.choice([0, 0, 1, rng.randint(0, 700), -rng.randint(0, 3)])) for k in new]
        cu = np.concatenate([[0], np.cumsum(new)])
        n_tok = int(cu[-1])
        rows = {}
        for slot in range(host.host_slots(n_tok, n, G, R)):
            it = _item(host, lens, cu, n_tok, 1 << 20, slot, G, R, 128, window)
            if it["rows"] <= 0:
                assert it["units"] == 0
                continue
            assert it["ok"] and it["rows"] <= R and it["t0"] == cu[it["s"]]
            seen = []
            for r in range(it["row0"], it["row0"] + it["rows"]):
                assert (it["s"], r) not in rows
                rows[(it["s"], r)] = slot
                p = lens[it["s"]] - new[it["s"]] + r // G
                seen += [(max(0, p - window + 1) if window else 0, p + 1)] if p >= 0 else []
            assert it["units"] == it["n_tiles"] + 1
            if not seen:
                assert it["lo"] == it["hi"] == it["n_tiles"] == 0
                continue
            assert it["lo"] == min(a for a, _ in seen) and it["hi"] == max(b for _, b in seen)
            assert it["hi"] <= lens[it["s"]]
            assert it["tile0"] * 128 <= it["lo"] < it["tile0"] * 128 + 128
            assert (it["tile0"] + it["n_tiles"] - 1) * 128 < it["hi"] <= (it["tile0"] + it["n_tiles"]) * 128
        assert len(rows) == sum(k * G for k in new)


def test_one_token_each_without_offsets(host):
    for slot in range(host.host_slots(5, 5, 4, 128)):
        it = _item(host, [0, 1, 129, 7, 3], None, 5, 1000, slot, 4, 128, 128, 0)
        if it["rows"]:
            assert it["rows"] == 4 and it["t0"] == it["s"]
    assert sum(_item(host, [0, 1, 129, 7, 3], None, 5, 1000, s, 4, 128, 128, 0)["rows"] for s in range(5)) == 20


def test_lying_lengths_and_offsets_are_clamped(host):
    """Offsets that fall or leave the tokens, negative or too long lengths: flagged, and nothing past the
    declared tokens or the table is addressed."""
    for lens, cu in (([50, 5000], [0, 3, 6]), ([-4, 10], [0, 3, 6]), ([10, 10], [0, 9, 6]), ([10, 10], [0, 3, 900]),
                     ([10, 10], [-5, 3, 6]), ([10, 10], [0, 6, 3])):
        flagged = False
        for slot in range(host.host_slots(6, 2, 4, 128)):
            it = _item(host, lens, cu, 6, 64, slot, 4, 128, 128, 0)
            assert 0 <= it["s"] < 2 and 0 <= it["t0"] <= 6 and 0 <= it["rows"] <= 128
            if it["rows"]:
                assert it["row0"] >= 0 and it["t0"] + (it["row0"] + it["rows"] - 1) // 4 < 6
            assert 0 <= it["lo"] <= it["hi"] <= 64
            flagged |= not it["ok"]
        assert flagged, (lens, cu)


@pytest.mark.parametrize("total", [1, 3, 151, 152, 153, 10 ** 6 + 7, 2 ** 40 + 12345])
def test_shares_cover_the_work(host, total):
    blocks = min(152, total)
    at = [host.host_share(total, b, blocks) for b in range(blocks + 1)]
    assert at[0] == 0 and at[-1] == total
    sizes = [b - a for a, b in zip(at, at[1:])]
    assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1


def test_pages_outside_the_cache_are_not_followed(host):
    row, p = _i32([5, -1, 99, 100, 2 ** 31 - 1, -2 ** 31])
    page = lambda pos: host.host_page(p, pos, 16, 6, 100)  # noqa: E731
    assert [page(16 * i) for i in range(6)] == [5, -1, 99, -1, -1, -1]
    assert page(15) == 5 and page(47) == 99 and page(-1) == -1 and page(16 * 6) == -1 and page(2 ** 31 - 1) == -1


# ------------------------------------------------------- rotary frequencies

def test_rope_frequencies():
    import chunked_recurrence_gb300 as crg
    plain = [10000.0 ** (-2 * i / 64) for i in range(32)]
    near = lambda a, b: all(abs(x - y) <= 1e-14 * abs(y) for x, y in zip(a.tolist(), b))  # noqa: E731
    assert near(crg.gdn_rope_inv_freq(64), plain)
    assert near(crg.gdn_rope_inv_freq(64, scaling="linear", factor=4.0), [x / 4 for x in plain])
    big = 10000.0 * 4.0 ** (64 / 62)
    assert near(crg.gdn_rope_inv_freq(64, scaling="base", factor=4.0), [big ** (-2 * i / 64) for i in range(32)])
    parts = crg.gdn_rope_inv_freq(64, scaling="parts", factor=8.0, orig_len=4096)
    for x, got in zip(plain, parts.tolist()):
        turns = 4096 * x / (2 * math.pi)
        g = min(1.0, max(0.0, (turns - 1) / 31))
        assert abs(got - ((1 - g) * x / 8 + g * x)) <= 1e-14 * x
    assert parts[0] == plain[0] and abs(parts[-1] - plain[-1] / 8) < 1e-18


def test_rope_table_is_the_fraction_of_a_turn():
    """Each word is inv / 2 pi as a 64-bit fraction to double precision, whatever the sign or size."""
    import torch
    import chunked_recurrence_gb300 as crg
    inv = [1.0, 1e-4, 0.3, math.pi, -math.pi, 7.0, -0.25, 0.0, 2 * math.pi]
    words = crg.gdn_rope_freqs(torch.tensor(inv, dtype=torch.float64), device="cpu").tolist()
    for x, w in zip(inv, words):
        turns = Fraction(x / (2 * math.pi))
        off = (Fraction(w % 2 ** 64, 2 ** 64) - turns) % 1
        assert min(off, 1 - off) <= Fraction(1, 2 ** 63) + abs(turns) / 2 ** 52, x


# ------------------------------------------------------------------ refusals

P = ctypes.c_void_p
FAKE, WS = P(0x10000), P(0x20000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from chunked_recurrence_gb300 import build as b
    b.build()
    import chunked_recurrence_gb300 as crg
    return crg.load()


def _shape(**kw):
    import chunked_recurrence_gb300 as crg
    d = dict(n_seqs=2, n_tok=6, Hq=4, Hkv=2, D=128, dtype=1, page_size=16, n_pages=10, max_pages=5)
    d.update(kw)
    return crg.GdnCacheShape(**d)


def test_rope_refusals(lib):
    out = (ctypes.c_double * 64)()
    f = lib.gdn_rope_inv_freq
    assert f(64, 1e4, 0, 1, 0, 1, 32, out) == 0
    for bad in ((63, 1e4, 0, 1, 0, 1, 32), (0, 1e4, 0, 1, 0, 1, 32), (64, 0, 0, 1, 0, 1, 32), (64, 1e4, 4, 1, 0, 1, 32),
                (64, 1e4, 1, 0, 0, 1, 32), (2, 1e4, 2, 2, 0, 1, 32), (64, 1e4, 3, 2, 0, 1, 32), (64, 1e4, 3, 2, 9, 2, 2)):
        assert f(*bad, out) == 1, bad
    assert f(64, 1e4, 0, 1, 0, 1, 32, None) == 1
    words = (ctypes.c_uint64 * 4)()
    nan = (ctypes.c_double * 1)(float("nan"))
    assert lib.gdn_rope_freqs(nan, 1, words) == 1 and lib.gdn_rope_freqs(None, 1, words) == 1
    assert lib.gdn_rope_freqs(None, 0, None) == 0

    def call(q=FAKE, k=FAKE, pos=FAKE, fr=FAKE, dt=1, n=3, Hq=4, Hk=2, D=64, rd=64, qs=0, ks=0, qos=0, kos=0, flags=0,
             qo=FAKE, ko=FAKE):
        return lib.gdn_rope(q, k, pos, fr, dt, n, Hq, Hk, D, rd, qs, ks, qos, kos, 1.0, flags, qo, ko, None)
    for kw in (dict(dt=2), dict(n=-1), dict(Hq=-1), dict(D=0), dict(D=257), dict(rd=65), dict(rd=3), dict(rd=-2),
               dict(qs=255), dict(ks=1), dict(qos=255), dict(kos=127), dict(flags=1), dict(q=None), dict(k=None),
               dict(qo=None), dict(ko=None), dict(pos=None), dict(fr=None), dict(qs=512)):  # in place, another stride
        assert call(**kw) == 1, kw
    assert call(n=0, q=None, k=None, pos=None, fr=None, qo=None, ko=None) == 0


def test_append_and_attention_refusals(lib):
    def append(shape=None, q=FAKE, k=FAKE, v=FAKE, fr=FAKE, rd=128, flags=0, tb=FAKE, ln=FAKE, cu=FAKE, qo=P(0x30000),
               kc=FAKE, vc=FAKE, ws=WS, nbytes=256):
        sh = shape or _shape()
        return lib.gdn_kv_append(q, k, v, None, fr, rd, 1.0, flags, tb, ln, cu, ctypes.byref(sh), qo, kc, vc, ws, nbytes,
                                 None)

    def attn(shape=None, q=FAKE, kc=FAKE, vc=FAKE, tb=FAKE, ln=FAKE, cu=FAKE, new=3, window=0, flags=0, o=FAKE, ws=WS,
             nbytes=1 << 40):
        sh = shape or _shape()
        return lib.gdn_paged_attn(q, kc, vc, tb, ln, cu, ctypes.byref(sh), new, 0.1, window, flags, o, None, ws, nbytes,
                                  None)
    for bad, want in ((dict(n_seqs=-1), 1), (dict(n_tok=-1), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(D=0), 1),
                      (dict(dtype=2), 1), (dict(page_size=0), 1), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1),
                      (dict(table_stride=4), 1), (dict(head_stride=64, slot_stride=256, page_stride=4096), 1),
                      (dict(head_stride=128, slot_stride=64, page_stride=4096), 1),
                      (dict(head_stride=128, slot_stride=256), 1), (dict(q_stride=511), 1), (dict(k_stride=255), 1),
                      (dict(v_stride=255), 1), (dict(D=257), 2), (dict(Hq=1 << 17, Hkv=1 << 17), 2)):
        assert append(_shape(**bad)) == want, bad
        assert attn(_shape(**bad)) == want, bad
        assert lib.gdn_paged_attn_workspace_bytes(ctypes.byref(_shape(**bad)), 3) == 0
    assert append(cu=None) == 1 and attn(cu=None) == 1      # one token each needs n_tok = n_seqs
    for kw in (dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(tb=None), dict(ln=None), dict(qo=None),
               dict(fr=None), dict(rd=130), dict(rd=3), dict(flags=256), dict(flags=2)):
        assert append(**kw) == 1, kw
    assert append(_shape(q_stride=1024), qo=FAKE) == 1      # in place needs a dense q
    for kw in (dict(ws=None), dict(ws=P(0x20004)), dict(nbytes=255)):
        assert append(**kw) == 5, kw
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(tb=None), dict(ln=None), dict(o=None), dict(new=-1),
               dict(window=-1), dict(flags=1)):
        assert attn(**kw) == 1, kw
    need = lib.gdn_paged_attn_workspace_bytes(ctypes.byref(_shape()), 3)
    for kw in (dict(ws=None), dict(ws=P(0x20004)), dict(nbytes=need - 1)):
        assert attn(**kw) == 5, kw
    assert lib.gdn_paged_attn_workspace_bytes(None, 3) == 0
    none = dict(q=None, kc=None, vc=None, tb=None, ln=None)
    assert attn(_shape(n_tok=0), **none, o=None) == 0       # nothing to do
    assert append(_shape(n_tok=0, n_seqs=0), k=None, v=None, **none) == 0


def test_pages_refusals(lib):
    import chunked_recurrence_gb300 as crg
    T = lambda **kw: crg.GdnPageTables(**{**dict(page_table=0x1000, seq_lens=0x2000, refs=0x3000, n_rows=4,  # noqa: E731
                                                 max_pages=8, table_stride=0, n_pages=32, page_size=16), **kw})
    one = (ctypes.c_void_p * 1)(0x9000)
    pools = lambda **kw: crg.GdnPagePools(**{**dict(pools=one, n_pools=1, page_bytes=64, page_stride=64), **kw})  # noqa: E731
    need = lib.gdn_pages_workspace_bytes(32, 4)
    assert need >= 256 and lib.gdn_pages_workspace_bytes(-1, 4) == 0 == lib.gdn_pages_workspace_bytes(4, -1)
    b = ctypes.byref
    calls = {"grow": lambda t, w=WS, n=need, k=2, ls=FAKE: lib.gdn_pages_grow(b(t), ls, ls, k, w, n, None),
             "free": lambda t, w=WS, n=need, k=2, ls=FAKE: lib.gdn_pages_free(b(t), ls, k, w, n, None),
             "fork": lambda t, w=WS, n=need, k=2, ls=FAKE, p=pools(): lib.gdn_pages_fork(b(t), ls, ls, k, b(p), w, n, None),
             "compact": lambda t, w=WS, n=need, p=pools(): lib.gdn_pages_compact(b(t), b(p), w, n, None)}
    for name, f in calls.items():
        for bad in (dict(n_rows=-1), dict(max_pages=-1), dict(n_pages=-1), dict(page_size=0), dict(table_stride=7),
                    dict(page_table=None), dict(seq_lens=None), dict(refs=None), dict(n_pages=1 << 21)):
            assert f(T(**bad)) == 1, (name, bad)
        assert f(T(), w=None) == 5 and f(T(), w=P(0x20004)) == 5 and f(T(), n=need - 1) == 5, name
        if name != "compact":
            assert f(T(), k=-1) == 1 and f(T(), ls=None) == 1 and f(T(), k=0, ls=None) == 0, name
    assert calls["grow"](T(), k=5) == 1 and calls["fork"](T(), k=5) == 1  # a row twice
    null = (ctypes.c_void_p * 1)(None)
    for bad, want in ((dict(n_pools=-1), 1), (dict(page_bytes=-1), 1), (dict(page_stride=63), 1), (dict(pools=null), 1),
                      (dict(n_pools=crg.GDN_MAX_POOLS + 1), 2)):
        assert calls["fork"](T(), p=pools(**bad)) == want and calls["compact"](T(), p=pools(**bad)) == want, bad
        assert lib.gdn_pages_copy(FAKE, FAKE, 2, 32, b(pools(**bad)), WS, 256, None) == want
    assert lib.gdn_pages_copy(None, FAKE, 2, 32, b(pools()), WS, 256, None) == 1
    assert lib.gdn_pages_copy(FAKE, FAKE, 2, 32, b(pools()), WS, 255, None) == 5
    assert lib.gdn_pages_copy(None, None, 0, 32, b(pools()), WS, 256, None) == 0
    assert calls["compact"](T(n_pages=0, refs=None)) == 0


def test_python_layer_refuses():
    """Wrong dtypes, layouts and devices raise before the library is called."""
    import torch
    import chunked_recurrence_gb300 as crg
    q = torch.zeros(2, 4, 64)
    cache = torch.zeros(8, 16, 2, 64)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        crg.gdn_paged_attn(q, cache, cache, table, lens)
    shape = lambda **kw: crg.cache_shape(**{**dict(q=q, k_cache=cache, v_cache=cache, page_table=table,  # noqa: E731
                                                   seq_lens=lens), **kw})
    assert (shape().Hq, shape().Hkv, shape().page_size, shape().max_pages) == (4, 2, 16, 4)
    assert shape(k_cache=cache.permute(0, 2, 1, 3), v_cache=cache.permute(0, 2, 1, 3), q=torch.zeros(2, 16, 64)).Hkv == 16
    for kw, err in ((dict(page_table=table.long()), TypeError), (dict(seq_lens=lens.long()), TypeError),
                    (dict(v_cache=cache.bfloat16()), TypeError), (dict(v_cache=cache[:4]), ValueError),
                    (dict(q=torch.zeros(3, 4, 64)), ValueError), (dict(q=torch.zeros(2, 3, 64)), ValueError),
                    (dict(q=torch.zeros(2, 64, 4).transpose(1, 2)), ValueError),
                    (dict(seq_lens=lens[:1]), ValueError), (dict(k=torch.zeros(2, 1, 64)), ValueError),
                    (dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)), ValueError),
                    (dict(k_cache=torch.zeros(8, 16, 2, 128)[..., ::2], v_cache=torch.zeros(8, 16, 2, 128)[..., ::2]),
                     ValueError)):
        with pytest.raises(err):
            shape(**kw)
