"""GPU parity of attention where groups of sequences share a prefix, against plain 64-bit attention of each sequence
over all its positions (test_paged_gpu's reference and tolerance: the operator is the same, only what is read is less; a row's
sums join in two parts more, each an fp32 rounding within the n 2^-23 of the tolerance)."""
import math
import threading

import numpy as np
import pytest
import torch

from tests.test_paged_gpu import DEV, HALF, Cache, assert_attn, attn_ref, cu_of, f64, gen, randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def crg():
    import chunked_recurrence_gb300 as m
    m.load()
    return m


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Shared(Cache):
    """A cache whose sequences [groups[g], groups[g + 1]) begin with the same prefix[g] tokens.  Only the first of a group
    has them in its pages where `bare`: the others' full pages of the prefix are not there (-1)."""

    def __init__(self, seed, dtype, groups, prefix, lens, hkv, d, page, bare=False, **kw):
        super().__init__(seed, dtype, lens, hkv, d, page, **kw)
        self.groups, self.prefix = i32(*groups), i32(*prefix)
        whole = self.table.clone()
        for g, p in enumerate(prefix):
            for s in range(groups[g] + 1, groups[g + 1]):
                for i in range(-(-min(p, lens[s]) // page)):
                    n = min(page, p - i * page, lens[s] - i * page)
                    a, b = int(whole[groups[g], i]), int(whole[s, i])
                    for c in (self.k, self.v):
                        c[b, :n] = c[a, :n]
        self.whole = whole
        if bare:
            for g, p in enumerate(prefix):
                self.table[groups[g] + 1: groups[g + 1], : p // page] = -1

    def rows(self, s, t):
        m = self.lens_list[s]
        pages = self.whole[s, : -(-m // self.page)].long()
        return f64(t[pages].reshape(-1, *t.shape[2:])[:m]) if m else np.zeros((0, *t.shape[2:]))


def run(crg, seed, dtype, groups, prefix, new, lens, hq, hkv, d, page, bare=True, simt=False, most=None, one=False,
        scale=None, tensor=None, **kw):
    cache = Shared(seed, dtype, groups, prefix, lens, hkv, d, page, bare, **kw)
    q = randn(gen(seed + 1), (sum(new), hq, d), dtype)
    ws = crg.Workspace(1 << 29, DEV)
    o, lse = crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups, cache.prefix,
                                       None if one else cu_of(new), max_group_new=most, want_lse=True, simt=simt,
                                       workspace=ws, scale=scale)
    torch.cuda.synchronize()
    assert ws.status() == 0
    assert_attn(o, lse, q, cache, new, 0, scale, tensor=dtype == "bf16" and not simt if tensor is None else tensor)
    return cache, q, o, lse


PLAIN = [  # dtype, groups, prefix, new, lens, hq, hkv, d, page
    ("f32", [0, 3], [200], [1, 1, 1], [201, 217, 300], 4, 2, 64, 16),
    ("f32", [0, 2, 3], [70, 0], [5, 2, 37], [75, 90, 90], 6, 2, 64, 16),
    ("f32", [0, 0, 2, 2, 3], [0, 33, 0, 40], [9, 1, 3], [44, 33, 43], 3, 1, 128, 1),   # groups of none
    ("bf16", [0, 2], [38], [9, 3], [50, 41], 4, 4, 96, 5),
    ("f32", [0, 2], [20], [4, 2], [22, 21], 2, 1, 7, 3),          # new tokens that lie in the prefix
    ("f32", [0, 2, 4], [5, 1], [3, 1, 2, 2], [5, 5, 2, 1], 2, 1, 250, 48),  # nothing behind it, and rows that see nothing
    ("f32", [0, 4], [900], [20, 1, 0, 40], [950, 901, 950, 960], 4, 2, 256, 48),
    ("bf16", [0, 30], [77], [1] * 30, [78 + i for i in range(30)], 130, 1, 64, 16),
]


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("case", PLAIN, ids=str)
def test_other_types_and_shapes(crg, case, simt):
    run(crg, 51, *case, simt=simt, tensor=case[0] == "bf16" and case[7] in (64, 128, 256) and not simt)


TC = [  # groups, prefix, new, lens, hq, hkv, d, page
    ([0, 1], [1], [1], [1], 1, 1, 128, 16),                             # nothing of its own
    ([0, 1], [0], [1], [1], 1, 1, 128, 16),                             # nothing shared
    ([0, 3], [500], [1, 1, 1], [501, 627, 700], 4, 2, 128, 16),
    ([0, 4], [129], [1, 1, 1, 1], [130, 1000, 257, 200], 8, 1, 128, 64),
    ([0, 2, 5], [400, 77], [1, 1, 1, 1, 1], [513, 402, 77, 78, 205], 3, 3, 64, 8),
    ([0, 40], [1000], [1] * 40, [1001 + 13 * i for i in range(40)], 14, 2, 256, 32),
    ([0, 70], [300], [1] * 70, [301 + 3 * i for i in range(70)], 8, 2, 64, 16),
    ([0, 2, 2, 3, 5], [128, 0, 9, 333], [13, 1, 9, 40, 0], [500, 129, 9, 600, 333], 4, 2, 128, 48),
    ([0, 2], [40], [20, 3], [45, 41], 8, 2, 128, 16),                   # new tokens that lie in the prefix
    ([0, 2], [300], [300, 200], [310, 450], 2, 1, 64, 16),              # most of them
    ([0, 2], [130], [130, 5], [130, 140], 8, 2, 256, 64),               # all of them
    ([0, 3], [600], [257, 5, 1], [900, 605, 1000], 4, 1, 128, 24),
    ([0, 3], [900], [200, 1, 33], [1100, 901, 940], 8, 2, 256, 64),
    ([0, 16], [6000], [3] * 16, [6003 + i for i in range(16)], 8, 1, 128, 256),
    ([0, 2], [20000], [1, 1], [20001, 20500], 8, 1, 64, 64),
    ([0, 1, 2, 3], [50, 600, 3], [1, 1, 1], [51, 601, 4], 128, 1, 128, 16),
]


@pytest.mark.parametrize("case", TC, ids=str)
def test_tensor_cores(crg, case):
    run(crg, 52, "bf16", *case)


@pytest.mark.parametrize("order,gap", [("token", 3), ("head", 0), ("head", 8)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_cache_layouts(crg, d, order, gap):
    run(crg, 53, "bf16", [0, 3], [90], [40, 1, 2], [150, 400, 92], 4, 2, d, 16, order=order, gap=gap)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [0, 1, 40, 5000])
def test_max_group_new_is_a_hint(crg, d, most):
    run(crg, 54, "bf16", [0, 3, 4], [250, 10], [1, 60, 17, 90], [300, 400, 267, 200], 8, 2, d, 16, most=most)


def test_one_token_each(crg):
    run(crg, 55, "bf16", [0, 20, 21, 37], [500, 0, 64], [1] * 37, [501 + 61 * i % 900 for i in range(37)], 8, 2, 128, 16,
        one=True)


def test_many_sequences_and_groups(crg):
    """More of both than a block has threads."""
    groups = sorted({0, 410} | set(range(0, 410, 3)) | set(range(0, 410, 7)))
    groups = [0, 0] + groups[1:]
    prefix = [0] + [5 + g % 11 for g in groups[1:-1]]
    new = [i % 3 for i in range(410)]
    of = np.searchsorted(groups, np.arange(410), side="right") - 1
    lens = [prefix[g] + n + (7 * i) % 40 for i, (g, n) in enumerate(zip(of, new))]
    run(crg, 56, "bf16", groups, prefix, new, lens, 2, 1, 64, 8)


def test_scores_far_apart(crg):
    """The maximum in the prefix, or behind it, by hundreds of e-folds."""
    for scale in (3.0, 0.01):
        run(crg, 57, "bf16", [0, 2], [400], [50, 1], [700, 700], 4, 2, 128, 16, scale=scale)
    for where in (slice(0, 40), slice(40, None)):
        cache = Shared(58, "bf16", [0, 2], [640], [1200, 1000], 1, 128, 16)
        q = torch.ones((90, 1, 128), dtype=torch.bfloat16, device=DEV)
        for s in range(2):
            pages = cache.table[s][where]
            cache.k[pages[pages >= 0].long()] += 1.0
        o, lse = crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups, cache.prefix,
                                           cu_of([60, 30]), want_lse=True, scale=3.0)
        assert_attn(o, lse, q, cache, [60, 30], scale=3.0)


def test_strided_q_and_given_outputs(crg):
    cache = Shared(59, "bf16", [0, 2], [50], [100, 60], 2, 128, 16)
    x = randn(gen(60), (24, 8 * 128 + 64), "bf16")
    q = x.as_strided((24, 8, 128), (x.stride(0), 128, 1), 64)
    o = torch.empty((24, 8, 128), dtype=torch.bfloat16, device=DEV)
    r, _ = crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups, cache.prefix,
                                     cu_of([20, 4]), o=o)
    assert r.data_ptr() == o.data_ptr()
    assert_attn(o, None, q, cache, [20, 4])


@pytest.mark.parametrize("simt", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_groups_and_pages_are_reported(crg, dtype, simt):
    """Groups that miss sequences, prefixes longer than a sequence, pages outside the cache: GDN_ERR_BOUNDS, and the groups
    that are none of it as they should be."""
    lens, new = [100, 60, 80, 90, 70], [4, 2, 3, 1, 1]
    cache = Shared(61, dtype, [0, 2, 4, 5], [40, 50, 0], lens, 2, 128, 16)
    q = randn(gen(62), (11, 4, 128), dtype)
    ro, _, a, ds = attn_ref(q, cache, new, 0, 128 ** -0.5)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for what in ("page", "missing", "prefix", "negative", "last"):
        ws = crg.Workspace(1 << 28, DEV)
        table, groups, prefix = cache.table.clone(), cache.groups.clone(), cache.prefix.clone()
        right = slice(0, 6)
        if what == "page":
            table[2, 1] = 10 ** 9
        elif what == "missing":
            table[2, 0] = -1
        elif what == "prefix":
            prefix[1] = 81
        elif what == "negative":
            prefix[1] = -3
        else:
            groups[3], right = 4, slice(0, 10)
        o, _ = crg.gdn_paged_attn_shared(q, cache.k, cache.v, table, cache.lens, groups, prefix, cu_of(new),
                                         workspace=ws, simt=simt)
        assert ws.status() == crg.GDN_ERR_BOUNDS, what
        off = np.abs(f64(o)[right] - ro[right])
        assert np.all(off <= u * np.abs(ro[right]) + (u + 4 * ds[right][..., None] + 2.0 ** -16) * a[right]), what


def test_statuses_of_calls_without_a_workspace(crg):
    cache = Shared(63, "bf16", [0, 2], [40], [100, 60], 2, 128, 16)
    q = randn(gen(64), (2, 4, 128), "bf16")
    crg.gdn_paged_status_reset()
    call = lambda p: crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups, p)  # noqa: E731
    call(cache.prefix)
    assert crg.gdn_paged_status() == crg.GDN_OK
    call(i32(61))
    assert crg.gdn_paged_status() == crg.GDN_ERR_BOUNDS
    crg.gdn_paged_status_reset()


def test_python_refusals(crg):
    cache = Shared(65, "bf16", [0, 2], [40], [100, 60], 2, 128, 16)
    q = randn(gen(66), (2, 4, 128), "bf16")
    call = lambda g=cache.groups, p=cache.prefix, x=q, **kw: crg.gdn_paged_attn_shared(  # noqa: E731
        x, cache.k, cache.v, cache.table, cache.lens, g, p, **kw)
    with pytest.raises(TypeError, match="group_offsets"):
        call(g=cache.groups.long())
    with pytest.raises(TypeError, match="prefix_lens"):
        call(p=cache.prefix.float())
    with pytest.raises(ValueError, match="one entry more"):
        call(p=i32(40, 40))
    with pytest.raises(ValueError, match="CUDA"):
        call(g=cache.groups.cpu())
    with pytest.raises(ValueError, match="overlap"):
        call(x=q[:1].expand(2, -1, -1))
    with pytest.raises(ValueError, match="lse"):
        call(lse=torch.empty((2, 4), dtype=torch.bfloat16, device=DEV))


def test_empty_calls(crg):
    cache = Shared(67, "bf16", [0, 1], [4], [10], 1, 64, 16)
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    o, lse = crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups, cache.prefix, cu_of([0]),
                                       want_lse=True)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    o, _ = crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table[:0], cache.lens[:0], i32(0), i32())
    assert o.shape == (0, 2, 64)


def test_offsets_past_32_bits(crg):
    """Pages more than 2^31 elements apart."""
    stride = (1 << 31) + 128
    buf = torch.empty(2 * stride + 16 * 128 + 64, dtype=torch.bfloat16, device=DEV)
    view = lambda o: buf.as_strided((3, 8, 1, 128), (stride, 128, 128, 1), o)  # noqa: E731
    k, v = view(0), view(8 * 128)
    cache = Shared(68, "bf16", [0, 1], [9], [20], 1, 128, 8, spare=0)
    k.copy_(cache.k)
    v.copy_(cache.v)
    q = randn(gen(69), (3, 2, 128), "bf16")
    for simt in (False, True):
        o, lse = crg.gdn_paged_attn_shared(q, k, v, cache.table, cache.lens, cache.groups, cache.prefix, cu_of([3]),
                                           want_lse=True, simt=simt)
        assert_attn(o, lse, q, cache, [3], tensor=not simt)


def test_stream_and_graph(crg):
    """On another stream, and captured: a replay follows the lengths, groups and contents of the moment."""
    cache = Shared(70, "bf16", [0, 2], [150], [300, 200], 2, 128, 16)
    q = randn(gen(71), (2, 8, 128), "bf16")
    call = lambda **kw: crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups,  # noqa: E731
                                                  cache.prefix, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, _ = call()
    side.synchronize()
    assert_attn(o, None, q, cache, [1, 1])
    side.wait_stream(torch.cuda.current_stream())
    o, _ = call(stream=side)
    side.synchronize()
    assert_attn(o, None, q, cache, [1, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o=o)
    cache.lens -= 37
    cache.lens_list = [263, 163]
    cache.prefix.fill_(100)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert_attn(o, None, q, cache, [1, 1])


def test_wait_that_runs_out_is_reported(crg):
    """The test mode gives up at the first wait: the status says so and the context stays usable."""
    cache = Shared(72, "bf16", [0, 2], [150], [300, 200], 2, 128, 16)
    q = randn(gen(73), (2, 8, 128), "bf16")
    ws = crg.Workspace(1 << 28, DEV)
    call = lambda **kw: crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups,  # noqa: E731
                                                  cache.prefix, workspace=ws, **kw)
    call(_test_no_wait=True)
    assert ws.status() == crg.GDN_ERR_TIMEOUT
    ws.reset()
    o, _ = call()
    assert ws.status() == 0
    assert_attn(o, None, q, cache, [1, 1])


def test_two_threads(crg):
    """Calls of two threads on the default stream, each with scratch of its own."""
    caches = [Shared(74, "bf16", [0, 3], [3000], [3100, 3200, 3050], 2, 128, 16),
              Shared(75, "bf16", [0, 40], [500], [501 + i for i in range(40)], 1, 64, 16)]
    qs = [randn(gen(76), (3, 8, 128), "bf16"), randn(gen(77), (40, 8, 64), "bf16")]
    call = lambda i: crg.gdn_paged_attn_shared(qs[i], caches[i].k, caches[i].v, caches[i].table, caches[i].lens,  # noqa: E731
                                               caches[i].groups, caches[i].prefix, want_lse=True)
    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    wrong, failed = torch.zeros(2, device=DEV), []

    def job(i):
        try:
            for _ in range(100):
                for a, b in zip(call(i), want[i]):
                    wrong[i] += (a != b).any()
        except BaseException as e:  # noqa: B036
            failed.append(e)
    threads = [threading.Thread(target=job, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and wrong.tolist() == [0, 0]


INF = math.inf


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 96)])
@pytest.mark.parametrize("what,where,value", [("k", 30, INF), ("k", 30, -INF), ("k", 110, math.nan), ("v", 30, INF),
                                              ("v", 110, math.nan)])
def test_infinities_reach_the_rows_that_see_them(crg, dtype, d, what, where, value):
    """On the paths that multiply in fp32: a position of the prefix (30) or of the second sequence's own (110)."""
    cache = Shared(78, dtype, [0, 2, 3], [50, 0], [120, 130, 80], 2, d, 16)
    pages = cache.table if where >= 50 else cache.whole
    for s in ((1,) if where >= 50 else (0, 1)):
        getattr(cache, what)[int(cache.whole[s, where // 16]), where % 16, 0, 1] = value
    assert pages is not None
    q = randn(gen(79), (4, 4, d), dtype)
    new = [1, 2, 1]
    o, lse = crg.gdn_paged_attn_shared(q, cache.k, cache.v, cache.table, cache.lens, cache.groups, cache.prefix, cu_of(new),
                                       want_lse=True)
    with np.errstate(all="ignore"):
        ro, rl, a, ds = attn_ref(q, cache, new, 0, d ** -0.5)
    hit = np.zeros((4, 4), dtype=bool)
    hit[0 if where < 50 else 1: 3, :2] = True  # query heads 0 and 1 read kv head 0
    got, ref = f64(o), ro
    u = HALF[o.dtype]
    fine = ~hit
    assert np.all(np.abs(got[fine] - ref[fine]) <= u * np.abs(ref[fine]) + (4 * ds[fine][:, None] + 2.0 ** -15) * a[fine])
    assert np.all(np.isfinite(f64(lse)[fine]))
    if what == "v":  # that column alone
        assert np.all(~np.isfinite(got[hit][:, 1]))
        ok = np.delete(np.arange(d), 1)
        assert np.all(np.isfinite(got[hit][:, ok]))
    elif value == value and value > 0:
        sign = f64(q)[..., 1]  # +inf scores make NaN (inf - inf), -inf ones weigh nothing
        for t, h in zip(*np.nonzero(hit)):
            assert np.isnan(got[t, h]).all() if sign[t, h] > 0 else np.isfinite(got[t, h]).all()
    elif value != value:
        assert np.isnan(got[hit]).all()
