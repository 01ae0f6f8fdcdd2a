"""GPU parity of the attention weight that cached positions gather against a plain 64-bit implementation.

Tolerance: a weight e^(x - lse), x = scale <q, k>, is off by a factor of at most 1 + 2 (dx + 2^-20) with
dx = (D + 8) 2^-24 scale sum_d |q_d k_d| + 2^-23 (|x| + |lse|): the rounding of a sum of D products, of the exponent's
argument (two terms, in base 2) and of the base-2 exponential; n terms added in fp32 n 2^-24 of their sum, what was there
before as one more.
"""
import math
import threading

import numpy as np
import pytest
import torch

from tests.test_paged_gpu import DEV, Cache, cu_of, f64, gen, randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def crg():
    import chunked_recurrence_gb300 as m
    m.load()
    return m


def reference(q, lse, cache, new, window, scale, before, accumulate):
    """(mass, tolerance) [n_seqs, Hkv, length] in 64 bits."""
    q, lse, ref = f64(q), f64(lse), f64(before).copy()
    tol = np.zeros_like(ref)
    hq, d = q.shape[1:]
    hkv = cache.k.shape[2]
    t = 0
    with np.errstate(all="ignore"):
        for s, n in enumerate(new):
            k, m = cache.rows(s, cache.k), cache.lens_list[s]
            if not accumulate:
                ref[s, :, :m] = 0
            p, j = np.arange(m - n, m)[:, None], np.arange(m)[None]
            seen = (j <= p) & ((j > p - window) if window else True)
            for h in range(hq if m else 0):
                x = scale * (q[t: t + n, h] @ k[:, h * hkv // hq].T)
                size = abs(scale) * (np.abs(q[t: t + n, h]) @ np.abs(k[:, h * hkv // hq]).T)
                z = lse[t: t + n, h][:, None]
                w = np.where(seen & ~np.isneginf(z), np.exp(x - z), 0.0)
                dx = (d + 8) * 2.0 ** -24 * size + 2.0 ** -23 * (np.abs(x) + np.abs(np.where(np.isneginf(z), 0, z)))
                ref[s, h * hkv // hq, :m] += w.sum(0)
                tol[s, h * hkv // hq, :m] += np.where(w > 0, w * 2 * (dx + 2.0 ** -20), 0.0).sum(0)
            tol[s, :, :m] += (n * hq // hkv + 2) * 2.0 ** -24 * np.abs(ref[s, :, :m])
            t += n
    return ref, tol


def run(crg, seed, dtype, new, lens, hq, hkv, d, page, window=0, accumulate=True, order="token", gap=0, simt=False,
        max_new=None, one=False, scale=None, extra=3, lse=None):
    cache = Cache(seed, dtype, lens, hkv, d, page, order, gap)
    q = randn(gen(seed + 1), (sum(new), hq, d), dtype)
    cu = None if one else cu_of(new)
    scale = d ** -0.5 if scale is None else scale
    if lse is None:
        _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu, window=window, want_lse=True,
                                    scale=scale)
    big = torch.rand((len(lens), hkv + 1, max(lens + [1]) + extra), generator=gen(seed + 2), device=DEV)
    mass = big[:, :hkv]
    before = big.clone()
    ws = crg.Workspace(1 << 26, DEV)
    got = crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu, max_new=max_new, scale=scale, window=window,
                             accumulate=accumulate, simt=simt, workspace=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0 and got is mass
    ref, tol = reference(q, lse, cache, new, window, scale, before[:, :hkv], accumulate)
    off = np.abs(f64(mass) - ref)
    assert np.all(off <= tol), (off - tol).max()
    assert torch.equal(big[:, hkv], before[:, hkv])
    for s, m in enumerate(lens):
        assert torch.equal(mass[s, :, m:], before[s, :hkv, m:])
    return cache, q, lse, mass


PLAIN = [  # dtype, new, lens, hq, hkv, d, page, window
    ("f32", [1, 1, 1], [1, 17, 300], 4, 2, 64, 16, 0),
    ("f32", [5, 0, 37], [5, 9, 90], 6, 2, 64, 16, 0),
    ("f32", [33], [200], 3, 1, 128, 1, 50),
    ("bf16", [9, 3], [40, 3], 4, 4, 96, 5, 0),
    ("bf16", [70], [133], 8, 1, 200, 12, 1),
    ("f32", [4, 2], [2, 1], 2, 1, 7, 3, 0),          # rows that see nothing
    ("f32", [130, 1], [700, 65], 2, 1, 250, 48, 129),
    ("bf16", [3], [77], 130, 1, 64, 16, 0),          # more heads a group than a tile has rows
    ("f32", [300], [300], 4, 2, 128, 16, 0),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", PLAIN, ids=str)
def test_other_types_and_shapes(crg, case, accumulate):
    run(crg, 81, *case, accumulate=accumulate)


TC = [  # new, lens, hq, hkv, d, page, window
    ([1], [1], 1, 1, 128, 16, 0),
    ([1, 1, 1], [1, 127, 129], 4, 2, 128, 16, 0),
    ([1, 1, 1, 1], [0, 128, 1000, 3], 8, 1, 128, 64, 0),
    ([1, 1], [513, 77], 3, 3, 64, 8, 0),
    ([1, 1, 1], [300, 257, 64], 14, 2, 256, 32, 0),
    ([13, 1, 0, 40], [13, 500, 9, 333], 4, 2, 128, 48, 0),
    ([20, 3], [7, 3], 8, 2, 128, 16, 0),
    ([130], [130], 1, 1, 64, 128, 0),
    ([257, 5, 1], [400, 5, 1000], 2, 1, 64, 16, 0),
    ([65, 1, 129], [700, 513, 129], 8, 2, 128, 24, 0),
    ([200, 1], [200, 900], 4, 2, 256, 64, 0),
    ([70], [1500], 5, 1, 256, 16, 0),
    ([2, 1], [5000, 4001], 8, 1, 128, 256, 0),
    ([1], [20000], 8, 1, 64, 64, 0),
    ([700], [1300], 16, 2, 128, 32, 0),              # tiles cut between blocks
    ([900], [1000], 6, 1, 64, 16, 0),
    ([3], [400], 128, 1, 128, 16, 0),
    # windows
    ([1, 1, 1], [1000, 100, 129], 4, 2, 128, 16, 100),
    ([150, 9], [800, 9], 4, 2, 128, 16, 1),
    ([300, 33], [1000, 400], 2, 1, 64, 32, 129),
    ([90, 1], [900, 700], 4, 1, 256, 16, 260),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", TC, ids=str)
def test_tensor_cores(crg, case, accumulate):
    run(crg, 82, "bf16", *case, accumulate=accumulate)


@pytest.mark.parametrize("case", TC[::3], ids=str)
def test_without_tcgen05(crg, case):
    run(crg, 83, "bf16", *case, simt=True)


@pytest.mark.parametrize("order,gap", [("token", 3), ("head", 0), ("head", 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_layouts(crg, d, order, gap):
    run(crg, 84, "bf16", [40, 1], [150, 400], 4, 2, d, 16, order=order, gap=gap)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("max_new", [0, 1, 200])
def test_max_new_is_a_hint(crg, d, max_new):
    run(crg, 85, "bf16", [1, 90, 17], [300, 200, 17], 8, 2, d, 16, max_new=max_new)


def test_one_token_each_and_many_sequences(crg):
    run(crg, 86, "bf16", [1] * 37, [1 + 61 * i % 900 for i in range(37)], 8, 2, 128, 16, one=True)
    new = [i % 3 for i in range(400)]
    for dtype in ("bf16", "f32"):
        run(crg, 87, dtype, new, [n + (7 * i) % 40 for i, n in enumerate(new)], 2, 1, 64, 8, accumulate=False)


def test_scales(crg):
    """Scores over hundreds of e-folds, a negative scale, none at all."""
    for scale in (3.0, 0.01, -0.2, 0.0):
        run(crg, 88, "f32", [50, 1], [300, 200], 4, 2, 128, 16, scale=scale)
    for scale in (3.0, 0.01):
        run(crg, 88, "bf16", [50, 1], [300, 200], 4, 2, 128, 16, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_no_weight(crg, dtype):
    """Heads whose lse is -inf add nothing, wherever their tokens are."""
    cache = Cache(89, dtype, [100], 2, 128, 16)
    q = randn(gen(90), (40, 4, 128), dtype)
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([40]), want_lse=True)
    lse[::3, 1] = -math.inf
    mass = torch.zeros((1, 2, 100), device=DEV)
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu_of([40]))
    ref, tol = reference(q, lse, cache, [40], 0, 128 ** -0.5, torch.zeros_like(mass), True)
    assert np.all(np.abs(f64(mass) - ref) <= tol)


def test_weights_sum_to_the_tokens(crg):
    """The masses of a prompt add up to its tokens times the heads of a group."""
    cache = Cache(91, "bf16", [1000], 2, 128, 16)
    q = randn(gen(92), (1000, 8, 128), "bf16")
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([1000]), want_lse=True)
    mass = torch.full((1, 2, 1000), math.nan, device=DEV)
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu_of([1000]), accumulate=False)
    assert torch.all((mass.double().sum(-1) / 4000 - 1).abs() < 2.0 ** -16)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 96), ("bf16", 128), ("f32", 256)])
@pytest.mark.parametrize("new", [1, 40])
def test_infinities_and_nan(crg, dtype, d, new):
    """A key's reach its own position alone, a query's the positions that see it."""
    for what, value in (("k", math.inf), ("k", -math.inf), ("k", math.nan), ("q", math.inf), ("q", math.nan)):
        cache = Cache(93, dtype, [150, 70], 1, d, 16)
        q = randn(gen(94), (new + 1, 2, d), dtype)
        cu = cu_of([new, 1])
        _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu, want_lse=True)
        lse = torch.nan_to_num(lse, nan=2.0, posinf=2.0, neginf=2.0)
        if what == "k":
            cache.k[int(cache.table[0, 2]), 5, 0, 1] = value  # position 37
        else:
            q[0, 0, 1] = value                                # the first new token, at 150 - new
        mass = torch.zeros((2, 1, 150), device=DEV)
        crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu)
        ref, tol = reference(q, lse, cache, [new, 1], 0, d ** -0.5, torch.zeros_like(mass), True)
        got = f64(mass)
        fine = np.isfinite(ref)
        assert np.all(np.abs(got - ref)[fine] <= tol[fine]), what
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isposinf(got), np.isposinf(ref)), what


@pytest.mark.parametrize("simt", [False, True])
def test_bad_pages_and_lengths_are_reported(crg, simt):
    cache = Cache(95, "bf16", [100, 60, 80], 2, 128, 16)
    q = randn(gen(96), (9, 4, 128), "bf16")
    new = [4, 2, 3]
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of(new), want_lse=True)
    ref, tol = reference(q, lse, cache, new, 0, 128 ** -0.5, torch.zeros((3, 2, 101)), True)
    for what in ("page", "negative", "length", "room"):
        ws = crg.Workspace(1 << 26, DEV)
        table, lens = cache.table.clone(), cache.lens.clone()
        big = torch.zeros((3, 2, 101), device=DEV)
        mass = big
        if what == "length":
            lens[1] = 100000
        elif what == "room":
            mass = big[:, :, :59]
        else:
            table[1, 2] = 10 ** 9 if what == "page" else -5
        crg.gdn_paged_mass(q, cache.k, table, lens, lse, mass, cu_of(new), workspace=ws, simt=simt)
        assert ws.status() == crg.GDN_ERR_BOUNDS, what
        n = mass.shape[2]
        for s in (0, 2):
            assert np.all(np.abs(f64(mass)[s] - ref[s, :, :n]) <= tol[s, :, :n]), what
        assert (big[:, :, n:] == 0).all()


def test_statuses_of_calls_without_a_workspace(crg):
    cache = Cache(97, "bf16", [100, 60], 2, 128, 16)
    q, lse = randn(gen(98), (2, 4, 128), "bf16"), torch.zeros((2, 4), device=DEV)
    crg.gdn_paged_status_reset()
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, torch.zeros((2, 2, 100), device=DEV))
    assert crg.gdn_paged_status() == crg.GDN_OK
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, torch.zeros((2, 2, 99), device=DEV))
    assert crg.gdn_paged_status() == crg.GDN_ERR_BOUNDS
    crg.gdn_paged_status_reset()


def test_python_refusals(crg):
    cache = Cache(99, "bf16", [100, 60], 2, 128, 16)
    q, lse, mass = randn(gen(100), (2, 4, 128), "bf16"), torch.zeros((2, 4), device=DEV), torch.zeros((2, 2, 100), device=DEV)
    call = lambda x=q, z=lse, m=mass: crg.gdn_paged_mass(x, cache.k, cache.table, cache.lens, z, m)  # noqa: E731
    for kw, err in ((dict(z=lse.bfloat16()), ValueError), (dict(z=lse[:, :2]), ValueError), (dict(z=lse.t().contiguous().t()), ValueError),
                    (dict(m=mass.double()), TypeError), (dict(m=mass[0]), TypeError), (dict(m=mass[:1]), ValueError),
                    (dict(m=mass[:, :1]), ValueError), (dict(m=mass[:1].expand(2, -1, -1)), ValueError),
                    (dict(m=torch.zeros((2, 2, 200), device=DEV)[..., ::2]), TypeError), (dict(m=mass.cpu()), ValueError),
                    (dict(x=q.float()), TypeError)):
        with pytest.raises(err):
            call(**kw)


def test_empty_calls(crg):
    cache = Cache(101, "bf16", [10, 5], 1, 64, 16)
    q, lse = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV), torch.empty((0, 2), device=DEV)
    mass = torch.ones((2, 1, 12), device=DEV)
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu_of([0, 0]))
    assert (mass == 1).all()
    crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu_of([0, 0]), accumulate=False)
    assert mass[0, 0].tolist() == [0.0] * 10 + [1.0] * 2 and mass[1, 0].tolist() == [0.0] * 5 + [1.0] * 7
    crg.gdn_paged_mass(q, cache.k, cache.table[:0], cache.lens[:0], lse, mass[:0])


def test_offsets_past_32_bits(crg):
    """Pages, and rows of masses, more than 2^31 elements apart."""
    stride = (1 << 31) + 128
    buf = torch.empty(2 * stride + 8 * 128 + 64, dtype=torch.bfloat16, device=DEV)
    k = buf.as_strided((3, 8, 1, 128), (stride, 128, 128, 1), 0)
    cache = Cache(102, "bf16", [20], 1, 128, 8, spare=0)
    k.copy_(cache.k)
    q = randn(gen(103), (3, 2, 128), "bf16")
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of([3]), want_lse=True)
    for simt in (False, True):
        mass = torch.zeros((1, 1, 20), device=DEV)
        crg.gdn_paged_mass(q, k, cache.table, cache.lens, lse, mass, cu_of([3]), simt=simt)
        ref, tol = reference(q, lse, cache, [3], 0, 128 ** -0.5, torch.zeros_like(mass), True)
        assert np.all(np.abs(f64(mass) - ref) <= tol)
    del buf, k
    far = torch.empty((1 << 31) + 64, device=DEV)
    two = Cache(104, "bf16", [20, 33], 1, 128, 8)
    mass = far.as_strided((2, 1, 33), ((1 << 31) + 8, 33, 1), 0)
    mass.zero_()
    q = randn(gen(105), (2, 2, 128), "bf16")
    _, lse = crg.gdn_paged_attn(q, two.k, two.v, two.table, two.lens, want_lse=True)
    crg.gdn_paged_mass(q, two.k, two.table, two.lens, lse, mass)
    ref, tol = reference(q, lse, two, [1, 1], 0, 128 ** -0.5, torch.zeros_like(mass), True)
    assert np.all(np.abs(f64(mass) - ref) <= tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_stream_graph_and_the_same_bits(crg, dtype):
    """On another stream, and captured: a replay follows the lengths and contents of the moment; calls repeat bit by bit."""
    cache = Cache(106, dtype, [900, 700], 1, 128, 16)
    q = randn(gen(107), (150, 8, 128), dtype)
    new = [120, 30]
    cu = cu_of(new)
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu, want_lse=True)
    mass = torch.zeros((2, 1, 900), device=DEV)
    call = lambda **kw: crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, cu, accumulate=False, **kw)  # noqa: E731

    def check():
        torch.cuda.synchronize()
        ref, tol = reference(q, lse, cache, new, 0, 128 ** -0.5, mass, False)
        assert np.all(np.abs(f64(mass) - ref)[0, :, : cache.lens_list[0]] <= tol[0, :, : cache.lens_list[0]])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    check()
    first = mass.clone()
    for _ in range(20):
        call()
        assert torch.equal(mass, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    cache.lens -= 37
    cache.lens_list = [863, 663]
    q.mul_(0.5)
    graph.replay()
    check()


def test_two_threads(crg):
    """Calls of two threads on the default stream, each with scratch of its own."""
    state = []
    for i, (new, lens, d) in enumerate((([300], [2000], 128), ([40, 1], [300, 900], 64))):
        cache = Cache(110 + i, "bf16", lens, 1, d, 16)
        q = randn(gen(120 + i), (sum(new), 8, d), "bf16")
        _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu_of(new), want_lse=True)
        state.append((q, cache.k, cache.table, cache.lens, lse, torch.zeros((len(lens), 1, max(lens)), device=DEV), cu_of(new)))
    call = lambda i: crg.gdn_paged_mass(*state[i], accumulate=False)  # noqa: E731
    want = [call(i).clone() for i in range(2)]
    torch.cuda.synchronize()
    wrong, failed = torch.zeros(2, device=DEV), []

    def job(i):
        try:
            for _ in range(100):
                wrong[i] += (call(i) != want[i]).any()
        except BaseException as e:  # noqa: B036
            failed.append(e)
    threads = [threading.Thread(target=job, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and wrong.tolist() == [0, 0]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_window_never_reads_released_pages(crg, dtype, accumulate):
    """Pages wholly before every query's window may be given back (-1 in the table)."""
    cache = Cache(130, dtype, [1000, 600], 2, 128, 16)
    q = randn(gen(131), (31, 4, 128), dtype)
    new, cu = [30, 1], cu_of([30, 1])
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, cu, window=200, want_lse=True)
    table = cache.table.clone()
    for s, (n, m) in enumerate(((30, 1000), (1, 600))):
        table[s, : max(0, m - n - 200 + 1) // 16] = -1
    ws = crg.Workspace(1 << 26, DEV)
    mass = torch.rand((2, 2, 1000), generator=gen(132), device=DEV)
    before = mass.clone()
    crg.gdn_paged_mass(q, cache.k, table, cache.lens, lse, mass, cu, window=200, accumulate=accumulate, workspace=ws)
    assert ws.status() == 0
    ref, tol = reference(q, lse, cache, new, 200, 128 ** -0.5, before, accumulate)
    assert np.all(np.abs(f64(mass) - ref) <= tol)


@pytest.mark.parametrize("max_new", [1, 300])
def test_wait_that_runs_out_is_reported(crg, max_new):
    """The test mode gives up at the first wait: the status says so and the context stays usable."""
    cache = Cache(133, "bf16", [300, 200], 2, 128, 16)
    q, mass = randn(gen(134), (2, 8, 128), "bf16"), torch.zeros((2, 2, 300), device=DEV)
    _, lse = crg.gdn_paged_attn(q, cache.k, cache.v, cache.table, cache.lens, want_lse=True)
    ws = crg.Workspace(1 << 26, DEV)
    call = lambda **kw: crg.gdn_paged_mass(q, cache.k, cache.table, cache.lens, lse, mass, max_new=max_new,  # noqa: E731
                                           accumulate=False, workspace=ws, **kw)
    call(_test_no_wait=True)
    assert ws.status() == crg.GDN_ERR_TIMEOUT
    ws.reset()
    call()
    assert ws.status() == 0
    ref, tol = reference(q, lse, cache, [1, 1], 0, 128 ** -0.5, torch.zeros_like(mass), False)
    assert np.all(np.abs(f64(mass) - ref) <= tol)


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("d,hq,hkv,new", [(64, 12, 1, 1), (64, 16, 2, 2), (64, 15, 1, 2), (128, 16, 1, 1), (128, 6, 2, 5),
                                          (128, 32, 1, 1), (256, 5, 1, 1), (256, 16, 2, 2), (256, 1, 1, 13)])
def test_few_rows(crg, d, hq, hkv, new, accumulate, window):
    """One, two and four tiles of eight query rows, odd numbers of them; sequences that end in a tile or at its edge."""
    lens = [new, 64, 65, 200, 1000, 0, 127 + new]
    run(crg, 140, "bf16", [min(new, m) for m in lens], lens, hq, hkv, d, 16, window, accumulate, max_new=new)


@pytest.mark.parametrize("dtype,most", [("bf16", 40), ("bf16", 2), ("f32", 9)])
def test_more_sequences_than_threads_of_a_block(crg, dtype, most):
    n = 1500
    new = [i % (most + 1) for i in range(n)]
    lens = [x + 37 * i % 211 for i, x in enumerate(new)]
    run(crg, 99, dtype, new, lens, 4, 2, 64, 16)
