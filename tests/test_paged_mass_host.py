"""gdn_paged_mass on the CPU: the line of work that its kernels share, compiled for the host, and the refusals."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BP = 64


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("mass") / "paged_mass_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-static-libubsan", "-I", os.path.join(ROOT, "chunked_recurrence_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "host_emulation", "paged_mass_host.cpp")], check=True)
    return ctypes.CDLL(so)


def _i32(a):
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def pieces(host, lens, cu, G, Hkv, RQ, window, everything, room, units, n_tok=None, most=1 << 20):
    la, lp = _i32(lens)
    ca, cp = _i32(cu) if cu is not None else (None, None)
    n_tok = n_tok if n_tok is not None else len(lens) if cu is None else int(cu[-1])
    cap = 100000
    out, bad = (ctypes.c_int32 * (11 * cap))(), ctypes.c_int32()
    n = host.host_mass_pieces(lp, cp, len(lens), n_tok, most, G, Hkv, RQ, window, int(everything), room, units, cap, out,
                              ctypes.byref(bad))
    assert n >= 0
    a = np.frombuffer(out, dtype=np.int32, count=11 * n).reshape(n, 11)
    return [dict(zip("s h tile q0 n nq i0 i1 share lo hi".split(), r)) for r in a.tolist()], bad.value


@pytest.mark.parametrize("window", [0, 1, 100, 5000])
@pytest.mark.parametrize("everything", [False, True])
@pytest.mark.parametrize("G,RQ,units", [(1, 32, 1), (4, 128, 152), (7, 126, 13), (300, 32, 152)])
def test_pieces_cover_the_work_once(host, G, RQ, units, everything, window):
    """Every tile with a position to write has its query tiles once, in order, in shares that follow each other; and
    those hold every token that sees one of its positions."""
    rng = random.Random(G + RQ + units + window)
    for _ in range(8):
        n = rng.randint(1, 6)
        new = [rng.choice([0, 1, 1, rng.randint(1, 300)]) for _ in range(n)]
        lens = [max(0, k + rng.choice([0, 1, rng.randint(0, 1500), -rng.randint(0, 3)])) for k in new]
        cu = np.concatenate([[0], np.cumsum(new)])
        hkv = rng.randint(1, 3)
        got, bad = pieces(host, lens, cu, G, hkv, RQ, window, everything, 1 << 20, units)
        assert bad == 0
        assert [g["share"] for g in got] == sorted(g["share"] for g in got)
        at = {}
        for g in got:
            key = (g["s"], g["h"], g["tile"])
            assert g["q0"] == at.get(key, 0) and g["n"] >= (1 if g["nq"] else 0)
            at[key] = g["q0"] + g["n"]
            s, first = g["s"], lens[g["s"]] - new[g["s"]]
            spots = range(max(g["lo"], g["tile"] * BP), min(g["hi"], g["tile"] * BP + BP))
            assert len(spots) > 0
            seen = [i for i in range(new[s]) if any(j <= first + i and (not window or j > first + i - window) for j in
                                                    (max(spots[0], 0), *spots))]
            if seen:
                assert g["i0"] <= seen[0] and seen[-1] < g["i1"]
            assert g["nq"] == -(-(g["i1"] - g["i0"]) * G // RQ)
            if g["nq"] == g["q0"] + g["n"]:
                at[key] = -1
        for s in range(n):
            first = lens[s] - new[s]
            want = [j for j in range(lens[s]) if everything or any(j <= first + i and (not window or j > first + i - window)
                                                                  for i in range(new[s]))]
            for h in range(hkv):
                tiles = {k[2] for k in at if k[:2] == (s, h)}
                assert tiles >= {j // BP for j in want}
                assert all(at[(s, h, t)] == -1 for t in tiles)


def test_lying_lengths_are_clamped(host):
    """Offsets that fall or leave the tokens, lengths past the table or the masses: flagged, and nothing past the tokens,
    the table or a row of masses is addressed."""
    for lens, cu, room in (([50, 5000], [0, 3, 6], 100), ([-4, 10], [0, 3, 6], 100), ([10, 10], [0, 9, 6], 100),
                           ([10, 10], [0, 3, 900], 100), ([10, 10], [-5, 3, 6], 100), ([60, 10], [0, 3, 6], 59),
                           ([60, 10], [0, 3, 6], 0)):
        for everything in (False, True):
            got, bad = pieces(host, lens, cu, 4, 2, 128, 0, everything, room, 152, n_tok=6, most=64)
            assert bad > 0
            for g in got:
                assert 0 <= g["i0"] <= g["i1"] <= 6 and 0 <= g["lo"] < g["hi"] <= min(64, room)


# ------------------------------------------------------------------ refusals

P = ctypes.c_void_p
FAKE, WS = P(0x10000), P(0x20000)  # never dereferenced


def test_refusals():
    from chunked_recurrence_gb300 import build as b
    b.build()
    import chunked_recurrence_gb300 as crg
    lib = crg.load()

    def shape(**kw):
        return crg.GdnCacheShape(**{**dict(n_seqs=2, n_tok=6, Hq=4, Hkv=2, D=128, dtype=1, page_size=16, n_pages=10,
                                           max_pages=5), **kw})

    def call(sh=None, q=FAKE, kc=FAKE, tb=FAKE, ln=FAKE, cu=FAKE, lse=FAKE, new=3, window=0, acc=1, flags=0, mass=FAKE, rs=0,
             hs=0, room=80, ws=WS, nbytes=1 << 40):
        sh = sh or shape()
        return lib.gdn_paged_mass(q, kc, tb, ln, cu, lse, ctypes.byref(sh), new, 0.1, window, acc, flags, mass, rs, hs, room,
                                  ws, nbytes, None)
    need = lib.gdn_paged_mass_workspace_bytes
    for bad, want in ((dict(n_seqs=-1), 1), (dict(n_tok=-1), 1), (dict(Hq=3), 1), (dict(Hkv=0), 1), (dict(D=0), 1),
                      (dict(dtype=2), 1), (dict(page_size=0), 1), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1),
                      (dict(table_stride=4), 1), (dict(head_stride=64, slot_stride=256, page_stride=4096), 1),
                      (dict(q_stride=511), 1), (dict(D=257), 2), (dict(Hq=1 << 17, Hkv=1 << 17), 2)):
        assert call(shape(**bad)) == want, bad
        assert need(ctypes.byref(shape(**bad))) == 0
    assert call(cu=None) == 1
    for kw in (dict(q=None), dict(kc=None), dict(tb=None), dict(ln=None), dict(lse=None), dict(mass=None), dict(new=-1),
               dict(window=-1), dict(acc=2), dict(flags=1), dict(room=-1), dict(rs=160, hs=79), dict(rs=79, hs=80)):
        assert call(**kw) == 1, kw
    nbytes = need(ctypes.byref(shape()))
    for kw in (dict(ws=None), dict(ws=P(0x20004)), dict(nbytes=nbytes - 1)):
        assert call(**kw) == 5, kw
    none = dict(q=None, kc=None, tb=None, ln=None, lse=None, mass=None)
    assert call(shape(n_tok=0), **none) == 0 == call(shape(n_tok=0, n_seqs=0), acc=0, **none)
    import torch
    q, cache, i32 = torch.zeros(2, 4, 64), torch.zeros(8, 16, 2, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        crg.gdn_paged_mass(q, cache, i32[:, None], i32, torch.zeros(2, 4), torch.zeros(2, 2, 10))
