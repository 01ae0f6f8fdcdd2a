"""Attention over shared prefixes and eviction on the CPU: the index arithmetic that the kernels use, compiled for the
host, and the refusals of the entry points (nothing is launched)."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("groups") / "paged_groups_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-static-libubsan", "-I", os.path.join(ROOT, "chunked_recurrence_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "host_emulation", "paged_groups_host.cpp")], check=True)
    lib = ctypes.CDLL(so)
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    lib.host_shared_slots.restype = lib.host_share_begin.restype = i64
    lib.host_shared_slots.argtypes = [i64, i32, i32, i32, i32]
    lib.host_share_begin.argtypes = [i64, i32, i32]
    lib.host_share_of.argtypes = [i64, i64, i32]
    return lib


def _i32(a):
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


class Call:
    def __init__(self, host, lens, cu, groups, prefix, G, R, KT, over=2, n_tok=None, most=1 << 20):
        self.host, self.n, self.ng = host, len(lens), len(prefix)
        self.n_tok = n_tok if n_tok is not None else len(lens) if cu is None else int(cu[-1])
        self._keep = [_i32(x) if x is not None else (None, None) for x in (lens, cu, groups, prefix)]
        self.args = (G, R, KT, over)
        self.G, self.R, self.most = G, R, most
        self.slots = host.host_shared_slots(self.n_tok, self.n, self.ng, G, R)

    def item(self, slot):
        (_, lens), (_, cu), (_, groups), (_, prefix) = self._keep
        out, ends = (ctypes.c_int32 * 13)(), (ctypes.c_int32 * self.R)()
        self.host.host_shared_item(lens, cu, self.n, self.n_tok, self.most, groups, prefix, self.ng, slot, *self.args, out,
                                   ends)
        it = dict(zip("s t0 first row0 rows lo hi tile0 n_tiles ok units g own".split(), out))
        it["ends"] = list(ends)
        return it


def _random_call(rng, one):
    ng = rng.randint(1, 5)
    sizes = [rng.choice([0, 1, 2, rng.randint(1, 9)]) for _ in range(ng)]
    if sum(sizes) == 0:
        sizes[-1] = 1
    groups = np.concatenate([[0], np.cumsum(sizes)])
    prefix, lens, new = [], [], []
    for m in sizes:
        p = rng.choice([0, 1, 63, rng.randint(0, 500)]) if m else 0  # a group of none names no tokens
        prefix.append(p)
        for _ in range(m):
            k = 1 if one else rng.choice([0, 1, 1, rng.randint(1, 150)])
            own = rng.choice([0, k, rng.randint(0, 300)])  # new tokens may lie in the prefix
            lens.append(max(p + own, k))
            new.append(k)
    cu = None if one else np.concatenate([[0], np.cumsum(new)])
    return groups, prefix, lens, new, cu


@pytest.mark.parametrize("one", [False, True])
@pytest.mark.parametrize("G,R,KT", [(1, 128, 128), (4, 256, 128), (7, 126, 64), (8, 512, 128), (3, 16, 1), (300, 4, 1)])
def test_items_cover_every_row_and_position_once(host, one, G, R, KT):
    """Each row meets each position that it sees in exactly one of its group's prefix item and its own item."""
    rng = random.Random(G * 1000 + R + one)
    for _ in range(15):
        groups, prefix, lens, new, cu = _random_call(rng, one)
        call = Call(host, lens, cu, groups, prefix, G, R, KT)
        first = [0 if cu is None else 0] + np.cumsum(new).tolist()
        seen = {}
        for slot in range(call.slots):
            it = call.item(slot)
            assert it["units"] == (it["n_tiles"] + 2 if it["rows"] > 0 and it["n_tiles"] else 0)
            if it["rows"] <= 0:
                continue
            assert it["ok"] and it["rows"] <= R and it["row0"] % R == 0
            if it["n_tiles"]:
                assert it["tile0"] * KT <= it["lo"] < it["tile0"] * KT + KT
                assert (it["tile0"] + it["n_tiles"] - 1) * KT < it["hi"] <= (it["tile0"] + it["n_tiles"]) * KT
            for r in range(it["rows"]):
                t, head = it["t0"] + (it["row0"] + r) // G, (it["row0"] + r) % G
                s = next(i for i in range(len(lens)) if first[i] <= t < first[i + 1])
                g = max(i for i in range(len(prefix)) if groups[i] <= s < groups[i + 1])
                assert it["g"] == g
                p = lens[s] - new[s] + t - first[s]
                if it["own"]:
                    assert it["s"] == s
                    span = (it["lo"], min(p + 1, it["hi"]))
                else:
                    assert it["s"] == groups[g] and it["lo"] == 0
                    span = (0, it["ends"][r])
                assert (t, head, bool(it["own"])) not in seen
                seen[(t, head, bool(it["own"]))] = span if span[0] < span[1] else (0, 0)
        for s, (k, m) in enumerate(zip(new, lens)):
            g = max(i for i in range(len(prefix)) if groups[i] <= s < groups[i + 1])
            for i in range(k):
                p = m - k + i
                for head in range(G):
                    a, b = seen[(first[s] + i, head, False)], seen[(first[s] + i, head, True)]
                    assert a == ((0, min(p + 1, prefix[g])) if prefix[g] else (0, 0))
                    assert b == ((prefix[g], p + 1) if p + 1 > prefix[g] else (0, 0))
        assert len(seen) == 2 * sum(new) * G


def test_lying_groups_are_clamped(host):
    """Offsets that fall, leave the sequences or miss some, prefixes longer than a sequence: flagged, and nothing past the
    tokens, the sequences or a sequence's length is addressed."""
    lens, cu = [50, 60, 70], [0, 3, 6, 10]
    for groups, prefix in (([0, 2, 9], [10, 10]), ([0, -4, 3], [10, 10]), ([1, 2, 3], [10, 10]), ([0, 1, 2], [10, 10]),
                           ([0, 3, 3], [55, 0]), ([0, 2, 3], [-5, 10]), ([3, 1, 0], [10, 10]), ([0, 2, 3], [10, 2 ** 31 - 1]),
                           ([2 ** 31 - 1, -2 ** 31, 5], [10, 10])):
        call = Call(host, lens, cu, groups, prefix, 4, 128, 128, most=1 << 10)
        flagged = False
        for slot in range(call.slots):
            it = call.item(slot)
            assert 0 <= it["s"] < 3 and 0 <= it["g"] < 2 and 0 <= it["t0"] <= 10 and 0 <= it["rows"] <= 128
            if it["rows"]:
                assert it["row0"] >= 0 and it["t0"] + (it["row0"] + it["rows"] - 1) // 4 < 10
            assert 0 <= it["lo"] <= it["hi"] <= lens[it["s"]]
            assert all(0 <= e <= it["hi"] for e in it["ends"][: it["rows"]])
            flagged |= not it["ok"]
        assert flagged, (groups, prefix)


@pytest.mark.parametrize("blocks", [1, 76, 152])
@pytest.mark.parametrize("over", [2, 4])
def test_pieces_are_where_the_join_looks(host, blocks, over):
    """An item's pieces lie in the shares from the one that holds its first tile's unit to the one that holds its last, the
    first of them the one that begins it, and every share between has one."""
    rng = random.Random(blocks + over)
    for _ in range(30):
        units = [rng.choice([1, 2, 3, rng.randint(1, 300)]) + over for _ in range(rng.randint(1, 40))]
        total = sum(units)
        shares = min(blocks, total)
        bounds = [host.host_share_begin(total, b, shares) for b in range(shares + 1)]
        for u in rng.sample(range(total), min(total, 50)):
            b = host.host_share_of(total, u, shares)
            assert bounds[b] <= u < bounds[b + 1]
        at = 0
        for n in units:
            pieces = []
            for b in range(shares):
                a, e = max(bounds[b], at) - at, min(bounds[b + 1], at + n) - at
                if a < e:  # as a block cuts its share
                    j = host.host_unit_tile(a, over)
                    if host.host_unit_tile(e, over) > j:
                        pieces.append((b, j))
            f, last = (host.host_share_of(total, u, shares) for u in (at + over, at + n - 1))
            assert [b for b, _ in pieces] == list(range(f, last + 1))
            assert pieces[0][1] == 0 and all(j > 0 for _, j in pieces[1:])
            at += n
    lib = host.host_shares_agree
    lib.argtypes = [ctypes.c_int64, ctypes.c_int32]
    assert all(lib(t, min(blocks, t)) for t in (1, 2, 151, 152, 153, 10 ** 6 + 7, (1 << 40) + 12345))
    big = (1 << 40) + 12345
    for u in (0, 1, big // 2, big - 1):
        b = host.host_share_of(big, u, 152)
        assert host.host_share_begin(big, b, 152) <= u < host.host_share_begin(big, b + 1, 152)


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


BAD_SHAPES = ((dict(n_seqs=-1), 1), (dict(n_tok=-1), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(dtype=2), 1),
              (dict(page_size=0), 1), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1), (dict(table_stride=4), 1),
              (dict(head_stride=64, slot_stride=256, page_stride=4096), 1), (dict(q_stride=511), 1), (dict(D=257), 2),
              (dict(Hq=1 << 17, Hkv=1 << 17), 2))


def test_shared_attention_refusals(lib):
    def attn(shape=None, q=FAKE, kc=FAKE, vc=FAKE, tb=FAKE, ln=FAKE, cu=FAKE, gr=FAKE, pr=FAKE, ng=1, most=3, flags=0,
             o=FAKE, ws=WS, nbytes=1 << 40):
        sh = shape or _shape()
        return lib.gdn_paged_attn_shared(q, kc, vc, tb, ln, cu, gr, pr, ng, ctypes.byref(sh), most, 0.1, flags, o, None, ws,
                                         nbytes, None)
    need = lib.gdn_paged_attn_shared_workspace_bytes
    for bad, want in BAD_SHAPES:
        assert attn(_shape(**bad)) == want, bad
        assert need(ctypes.byref(_shape(**bad)), 1, 3) == 0
    assert attn(cu=None) == 1
    for kw in (dict(q=None), dict(kc=None), dict(vc=None), dict(tb=None), dict(ln=None), dict(o=None), dict(gr=None),
               dict(pr=None), dict(ng=0), dict(ng=-1), dict(most=-1), dict(flags=1)):
        assert attn(**kw) == 1, kw
    assert attn(ng=(1 << 28) + 1) == 2
    nbytes = need(ctypes.byref(_shape()), 1, 3)
    assert nbytes > 256 and need(None, 1, 3) == 0 and need(ctypes.byref(_shape()), -1, 3) == 0
    assert need(ctypes.byref(_shape()), 1, -1) == 0
    for kw in (dict(ws=None), dict(ws=P(0x20004)), dict(nbytes=nbytes - 1)):
        assert attn(**kw) == 5, kw
    none = dict(q=None, kc=None, vc=None, tb=None, ln=None, gr=None, pr=None, o=None)
    assert attn(_shape(n_tok=0), **none) == 0 == attn(_shape(n_tok=0, n_seqs=0), ng=0, **none)


def test_evict_refusals(lib):
    import chunked_recurrence_gb300 as crg
    b = ctypes.byref
    T = lambda **kw: crg.GdnPageTables(**{**dict(page_table=0x1000, seq_lens=0x2000, refs=0x3000, n_rows=4,  # noqa: E731
                                                 max_pages=8, table_stride=0, n_pages=32, page_size=16), **kw})
    two = (ctypes.c_void_p * 2)(0x9000, 0xa000)
    pools = lambda **kw: crg.GdnPagePools(**{**dict(pools=two, n_pools=2, page_bytes=16 * 2 * 64,  # noqa: E731
                                                    page_stride=4096), **kw})
    H = lambda **kw: crg.GdnPageHeads(**{**dict(mass=0x5000, n_layers=1, heads=2, mass_len=100, row_bytes=64), **kw})  # noqa: E731
    need = lib.gdn_pages_evict_workspace_bytes(b(T()), 2, 50, 1, 2)
    assert need >= 256 + 2 * 2 * 50 * 8

    def call(t=None, h=None, p=None, sq=FAKE, kp=FAKE, n=2, most=50, recent=3, w=WS, nbytes=need):
        return lib.gdn_pages_evict(b(t or T()), sq, kp, n, most, recent, b(h or H()), b(p or pools()), None, w, nbytes, None)
    for bad in (dict(n_rows=-1), dict(max_pages=-1), dict(n_pages=-1), dict(page_size=0), dict(table_stride=7),
                dict(page_table=None), dict(seq_lens=None), dict(refs=None), dict(n_pages=1 << 21)):
        assert call(t=T(**bad)) == 1, bad
    for bad in (dict(n_layers=0), dict(heads=0), dict(mass_len=-1), dict(row_bytes=0), dict(mass=None),
                dict(layer_stride=1, row_stride=100, head_stride=100, n_layers=2), dict(row_stride=99, head_stride=100),
                dict(row_stride=200, head_stride=99), dict(slot_stride=63, slot_head_stride=64),
                dict(slot_stride=128, slot_head_stride=63), dict(row_bytes=65),           # 16 slots of two heads' rows do not fit
                dict(slot_stride=1 << 62, slot_head_stride=64), dict(slot_stride=128, slot_head_stride=1 << 62),
                dict(slot_stride=64, slot_head_stride=-64), dict(n_layers=3)):            # two pools of three layers
        assert call(h=H(**bad)) == 1, bad
    assert call(h=H(row_bytes=1 << 17), p=pools(page_bytes=1 << 24, page_stride=1 << 24)) == 2
    null = (ctypes.c_void_p * 2)(0x9000, None)
    for bad, want in ((dict(n_pools=-1), 1), (dict(page_bytes=-1), 1), (dict(page_stride=63), 1), (dict(pools=null), 1),
                      (dict(n_pools=crg.GDN_MAX_POOLS + 1), 2)):
        assert call(p=pools(**bad)) == want, bad
    for kw in (dict(n=-1), dict(n=5), dict(most=-1), dict(recent=-1), dict(sq=None), dict(kp=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(w=None), dict(w=P(0x20004)), dict(nbytes=need - 1)):
        assert call(**kw) == 5, kw
    assert call(n=0, sq=None, kp=None) == 0
    for bad in ((None, 2, 50, 1, 2), (b(T(n_rows=-1)), 2, 50, 1, 2), (b(T()), -1, 50, 1, 2), (b(T()), 2, -1, 1, 2),
                (b(T()), 2, 50, 0, 2), (b(T()), 2, 50, 1, 0)):
        assert lib.gdn_pages_evict_workspace_bytes(*bad) == 0


def test_python_layer_refuses():
    """CPU tensors raise before the library is called."""
    import torch
    import chunked_recurrence_gb300 as crg
    q, cache = torch.zeros(2, 4, 64), torch.zeros(8, 16, 2, 64)
    table, lens = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        crg.gdn_paged_attn_shared(q, cache, cache, table, lens, torch.tensor([0, 2]), torch.tensor([0]))
    with pytest.raises(ValueError, match="CUDA"):
        crg.gdn_pages_evict(table, lens, torch.zeros(8, dtype=torch.int32), lens, lens, torch.zeros(1, 2, 2, 64), [cache], 16, 4)
