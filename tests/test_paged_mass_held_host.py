"""gdn_paged_mass for few query rows, on the CPU: the queries that a warp keeps from tile to tile are those that the tiles'
positions are seen by, with the kernel's own shares."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WARPS = 152 * 12  # shares at D 64 and 128
FURTHER = [(64, 4, 6, 1, 0), (128, 4, 9, 2, 0), (128, 4, 9, 2, 500), (128, 1, 40, 9, 0), (256, 2, 7, 1, 300), (256, 2, 7, 3, 0)]


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("held") / "paged_mass_held_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-static-libubsan", "-I", os.path.join(ROOT, "chunked_recurrence_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "host_emulation", "paged_mass_held_host.cpp")], check=True)
    return ctypes.CDLL(so)


def walk(host, lens, new, G, Hkv, tokens, window, everything, units=WARPS):
    """(pieces, kept, lost, followed): see the C++ file."""
    arrays = [np.ascontiguousarray(x, dtype=np.int32) for x in (lens, np.concatenate([[0], np.cumsum(new)]))]
    out = (ctypes.c_int64 * 4)()
    host.host_mass_held(*[x.ctypes.data_as(ctypes.c_void_p) for x in arrays], len(lens), int(arrays[1][-1]), 1 << 20, G, Hkv,
                        tokens * G, window, int(everything), units, out)
    return list(out)


@pytest.mark.parametrize("everything", [False, True])
@pytest.mark.parametrize("seqs,lens,new,G,Hkv,window", [
    (64, lambda s: 4000 + 62 * s, 4, 4, 8, 1024),   # drafted tokens in a sliding-window layer
    (64, lambda s: 5000 + 37 * s, 4, 4, 8, 4096),
    (32, lambda s: 6000 + s, 8, 4, 8, 4096),
    (40, lambda s: 1500 + 64 * s, 2, 1, 16, 500),
    (9, lambda s: 70000 + 11 * s, 32, 1, 2, 30000),
    (64, lambda s: 4000 + 62 * s, 4, 4, 8, 0),
])
def test_kept_rows_are_all_that_see_a_tile(host, seqs, lens, new, G, Hkv, window, everything):
    pieces, kept, lost, _ = walk(host, [lens(s) for s in range(seqs)], [new] * seqs, G, Hkv, new, window, everything)
    assert pieces > WARPS and kept > 0  # warps with several tiles
    assert lost == 0


def test_any_shares(host):
    rng = np.random.default_rng(5)
    for _ in range(60):
        n = int(rng.integers(1, 7))
        new = rng.integers(0, 9, n)
        lens = new + rng.integers(0, 900, n) - rng.integers(0, 3, n) * (rng.random(n) < 0.2)
        for tokens in (1, 3, 8):  # the call's bound, kept or not
            out = walk(host, np.maximum(lens, 0), new, int(rng.integers(1, 5)), int(rng.integers(1, 4)), tokens,
                       int(rng.choice([0, 1, 60, 130, 500])), bool(rng.random() < 0.5), int(rng.choice([1, 2, 7, 40])))
            assert out[2] == 0


def test_more_rows_than_the_call_said(host):
    """The sizes of test_paged_mass_few_gpu's test of that name: warps take a tile's further query rows with another tile
    still to come."""
    for d, group, new, said, window in FURTHER:
        lens = [900 + 62 * s for s in range(32)]
        pieces, _, lost, followed = walk(host, lens, [new] * 32, group, 8, said, window, True, 152 * (6 if d == 256 else 12))
        assert followed > 1000 and lost == 0
