"""gdn_pages_evict's selection on the CPU: a block's threads one after another, the warps between two barriers in several
orders, against a stable sort."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIRST, LAST, MIXED = 0, 1, 7  # which warp goes first


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("choose") / "pages_choose_host.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fno-strict-aliasing", "-I",
                    os.path.join(ROOT, "chunked_recurrence_gb300", "csrc"), "-o", so,
                    os.path.join(ROOT, "tests", "host_emulation", "pages_choose_host.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def call(w, need, order):
        w = np.ascontiguousarray(w, dtype=np.float32)
        index, weight = np.full(2 * len(w) + 1, -9, np.int32), np.full(2 * len(w) + 1, -9, np.float32)
        p = lambda a: a.ctypes.data_as(ctypes.c_void_p)  # noqa: E731
        assert lib.host_choose(p(w), len(w), need, order, p(index), p(weight)) == 1, "threads parted at a barrier"
        assert (index[need:] == -9).all() and (weight[need:] == -9).all()
        return index[:need], weight[:need]
    return call


def wanted(w, need):
    order = np.lexsort((np.arange(len(w)), np.where(np.isnan(w), 0, -w), np.isnan(w)))
    return np.sort(order[:need]).astype(np.int32)


def weights(kind, n):
    rng = np.random.default_rng(n)
    if kind == "weights":
        return np.exp(2 * rng.standard_normal(n)).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 3, n).astype(np.float32)
    if kind == "one digit":  # more than the list of candidates holds begin alike
        return (1 + rng.random(n) / 16).astype(np.float32)
    return np.resize(np.array([0.0, -0.0, -1.0, np.inf, -np.inf, np.nan, 1e-40, 3.0], np.float32), n)


# one, four and eight rounds of 4096 in registers, and more
@pytest.mark.parametrize("n", [2, 33, 1500, 4096, 4097, 9001, 16384, 16385, 30000, 32768, 32769, 40000])
@pytest.mark.parametrize("kind", ["weights", "ties", "one digit", "odd values"])
def test_against_a_sort(choose, n, kind):
    w = weights(kind, n)
    some = ((max(1, n // 8), FIRST), (n - 1, MIXED))
    for need, order in some if n > 10000 else (*some, (1, FIRST), (n // 2, LAST)):
        index, weight = choose(w, need, order)
        assert np.array_equal(index, wanted(w, need)), (need, order)
        assert np.array_equal(weight, w[index], equal_nan=True)


@pytest.mark.parametrize("order", [FIRST, LAST, MIXED, 8, 9])
def test_any_order_of_the_warps(choose, order):
    """What a warp reads behind a barrier is not written over by one that is ahead of it."""
    for n in (700, 5000):
        for kind in ("weights", "ties"):
            w = weights(kind, n)
            assert np.array_equal(choose(w, n // 3, order)[0], wanted(w, n // 3))
