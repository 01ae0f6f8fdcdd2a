"""GPU tests of eviction by accumulated weight against a plain model of tables, rows and weights: everything is whole
numbers or moved as it is, so everything has to be equal."""
import math

import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"


@pytest.fixture(scope="module")
def crg():
    import chunked_recurrence_gb300 as m
    m.load()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """The tables, weights and caches in plain numpy."""

    def __init__(self, table, lens, refs, mass, pools, page):
        self.table, self.lens, self.refs, self.mass = (t.cpu().numpy().copy() for t in (table, lens, refs, mass))
        self.pools = [p.float().cpu().numpy().copy() for p in pools]
        self.page = page

    def evict(self, seqs, keep, recent, max_keep):
        """kept, or None where it cannot be carried out."""
        page, (layers, _, heads, _) = self.page, self.mass.shape
        kept = np.full((layers, len(seqs), heads, max_keep), -1, dtype=np.int32)
        free = [i for i, r in enumerate(self.refs) if r == 0]
        fresh = []
        for s, m in zip(seqs, keep):
            need = -(-m // page) if m < self.lens[s] else 0
            if need > len(free):
                return None
            fresh.append([free.pop(0) for _ in range(need)])
        per = len(self.pools) // layers
        before = [p.copy() for p in self.pools]
        old = self.table.copy()
        for i, (s, m) in enumerate(zip(seqs, keep)):
            n = int(self.lens[s])
            if m >= n:
                kept[:, i, :, :n] = np.arange(n)
                continue
            late = min(recent, m)
            for lay in range(layers):
                for h in range(heads):
                    w = self.mass[lay, s, h, : n - late].copy()
                    rank = sorted(range(n - late), key=lambda j: (w[j] != w[j], 0.0 if w[j] != w[j] else -w[j], j))
                    stay = sorted(rank[: m - late]) + list(range(n - late, n))
                    kept[lay, i, h, :m] = stay
                    for j, src in enumerate(stay):
                        for p in range(lay * per, (lay + 1) * per):
                            self.pools[p][fresh[i][j // page], j % page, h] = before[p][old[s, src // page], src % page, h]
                    self.mass[lay, s, h, :n] = np.concatenate([self.mass[lay, s, h, stay], np.zeros(n - m, np.float32)])
            for k in range(-(-n // page)):
                self.refs[old[s, k]] -= 1
                self.table[s, k] = fresh[i][k] if k < len(fresh[i]) else -1
            self.refs[fresh[i]] = 1
            self.lens[s] = m
        return kept


def make(seed, lens, layers, heads, d, page, dtype=torch.bfloat16, order="token", spare=0, share=0, per=2, length=None):
    """Tables whose pages lie anywhere; the last `share` sequences begin with the first one's full pages."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    need = [-(-m // page) for m in lens]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g, device=DEV).tolist()
    table = np.full((len(lens), max(need + [1]) + 1), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    for s, n in enumerate(need):
        common = min(n, lens[0] // page) if s >= len(lens) - share and s > 0 else 0
        table[s, :common] = table[0, :common]
        table[s, common:n] = [perm.pop() for _ in range(n - common)]
        refs[table[s, :n]] += 1
    pools = []
    for _ in range(layers * per):
        shape = (n_pages, heads, page, d) if order == "head" else (n_pages, page, heads, d)
        t = torch.randn(shape, generator=g, device=DEV).to(dtype)
        pools.append(t.transpose(1, 2) if order == "head" else t)
    length = max(lens + [1]) if length is None else length
    mass = torch.randn((layers, len(lens), heads, length), generator=g, device=DEV).mul_(2).exp_()
    return i32(table), i32(lens), i32(refs), mass, pools


def run(crg, state, page, seqs, keep, recent, max_keep=None, want=None, ws=None):
    """The call beside the model; returns the status."""
    table, lens, refs, mass, pools = state
    model = Model(*state, page)
    max_keep = max(keep + [0]) if max_keep is None else max_keep
    ws = ws or crg.Workspace(1 << 26, DEV)
    kept = crg.gdn_pages_evict(table, lens, refs, i32(seqs), i32(keep), mass, pools, page, max_keep, recent, want_kept=True,
                               workspace=ws)
    ref = model.evict(seqs, keep, recent, max_keep) if want is None else None
    assert ws.status() == (crg.GDN_ERR_PAGES if ref is None and want is None else want or 0)
    ws.reset()
    for a, b in ((table, model.table), (lens, model.lens), (refs, model.refs)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert np.array_equal(mass.cpu().numpy(), model.mass, equal_nan=True)
    for p, b in zip(pools, model.pools):
        assert np.array_equal(p.float().cpu().numpy(), b)
    if ref is not None:
        assert np.array_equal(kept.cpu().numpy(), ref)
    return ref


CASES = [  # lens, layers, heads, d, page, dtype, keep, recent
    ([1], 1, 1, 64, 16, "bf16", [0], 0),                       # to nothing
    ([1, 0, 5], 1, 1, 64, 16, "bf16", [1, 0, 9], 3),           # nothing to evict
    ([33, 400, 17], 1, 2, 128, 16, "bf16", [32, 100, 3], 8),
    ([500, 77], 2, 4, 64, 8, "bf16", [100, 76], 1),
    ([300, 2000], 3, 2, 256, 32, "bf16", [299, 1023], 2000),   # recent ones alone
    ([2100, 40], 1, 3, 96, 48, "bf16", [1500, 40], 0),
    ([130, 129, 128], 1, 2, 7, 5, "f32", [128, 128, 128], 16),
    ([1024, 1025], 2, 1, 40, 1, "f32", [512, 1], 1),
    ([60], 1, 8, 250, 16, "bf16", [31], 5),
]
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.parametrize("order", ["token", "head"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_the_model(crg, case, order):
    lens, layers, heads, d, page, dtype, keep, recent = case
    fresh = sum(-(-m // page) for m in keep)
    state = make(len(lens) + d, lens, layers, heads, d, page, TYPES[dtype], order, spare=fresh + 3)
    assert run(crg, state, page, list(range(len(lens))), keep, recent) is not None


def test_again_and_again(crg):
    """A cache that stays near its bound: evicted, then grown, many times; two sequences of three, in another order."""
    page = 16
    state = make(3, [200, 90, 300], 2, 2, 64, page, spare=40)
    table, lens, refs, mass, pools = state
    ws = crg.Workspace(crg.gdn_pages_workspace_bytes(refs.shape[0], 3), DEV)
    for step in range(6):
        assert run(crg, state, page, [2, 0], [150, 120 + step], 20) is not None
        crg.gdn_pages_grow(table, lens, refs, i32([0, 2]), lens[[0, 2]] + 16 + step, page, workspace=ws)
        assert ws.status() == 0
        mass[:, 0, :, 120 + step: 136 + 2 * step] = 0.5
        mass[:, 2, :, 150: 166 + step] = 0.25


def test_pages_of_others_stay(crg):
    """Sequences that share an evicted one's pages keep them, evicted ones that share pages each get their own."""
    page = 16
    state = make(4, [200, 90, 210, 205], 1, 2, 64, page, spare=30, share=2)
    before = [state[4][0][state[0][2, :13].long()].clone()]
    assert run(crg, state, page, [0, 3], [64, 100], 10) is not None
    assert torch.equal(before[0], state[4][0][state[0][2, :13].long()])
    assert state[2][state[0][2, :12].long()].tolist() == [1] * 12


@pytest.mark.parametrize("n", [1500, 49152, 70000])  # weights kept in shared memory, all of it, and read each time
def test_ties_signs_and_odd_values(crg, n):
    """Equal weights go to the lowest position; zeros of either sign are equal; infinities in their order, NaN last."""
    page = 64
    state = make(5, [n], 1, 4, 8, page, torch.float32, spare=-(-n // page))
    mass = state[3]
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    mass[0, 0, 0] = 0.25                                                       # all equal
    mass[0, 0, 1] = torch.randint(0, 3, (n,), generator=g, device=DEV).float()
    mass[0, 0, 2] = torch.tensor([0.0, -0.0, -1.0, math.inf, -math.inf, math.nan], device=DEV).repeat(-(-n // 6))[:n]
    mass[0, 0, 3] = torch.randn(n, generator=g, device=DEV) * 1e-40            # subnormal
    assert run(crg, state, page, [0], [n * 9 // 10], 7) is not None


def test_more_rows_than_threads(crg):
    page, n = 4, 1100
    lens = [1 + (7 * i) % 23 for i in range(n)]
    keep = [(5 * i) % 17 for i in range(n)]
    state = make(7, lens, 1, 1, 4, page, torch.float32, spare=6000)
    order = np.random.default_rng(0).permutation(n).tolist()
    assert run(crg, state, page, order, [keep[i] for i in order], 2, max_keep=20) is not None


def test_weights_in_a_strided_buffer_and_odd_alignment(crg):
    """Masses as a view of a larger buffer, pools whose addresses are multiples of 4 and of 2 bytes."""
    page = 16
    for dtype, off in ((torch.float32, 1), (torch.bfloat16, 1)):
        table, lens, refs, mass, pools = make(8, [100, 77], 2, 2, 10, page, dtype, spare=20)
        big = torch.full((2, 3, 3, mass.shape[3] + 5), 7.0, device=DEV)
        view = big[:, :2, :2, 2: 2 + mass.shape[3]]
        view.copy_(mass)
        odd = []
        for p in pools:
            b = torch.empty(p.numel() + off, dtype=dtype, device=DEV)
            odd.append(b[off:].view(p.shape))
            odd[-1].copy_(p)
        assert run(crg, (table, lens, refs, view, odd), page, [0, 1], [40, 41], 3) is not None
        assert (big[:, 2] == 7).all() and (big[:, :, 2] == 7).all() and (big[..., :2] == 7).all() and (big[..., -3:] == 7).all()


def test_tables_alone(crg):
    """No pools: the tables and weights are cut."""
    page = 16
    table, lens, refs, mass, _ = make(9, [100, 77], 1, 2, 8, page, spare=9)
    assert run(crg, (table, lens, refs, mass, []), page, [1], [30], 3) is not None


def test_refused_lists_change_nothing(crg):
    page = 16
    state = make(10, [100, 60, 80], 2, 2, 16, page, spare=6)
    before = [t.clone() for t in state[:4]] + [p.clone() for p in state[4]]
    table, lens, refs, mass, pools = state
    ws = crg.Workspace(1 << 20, DEV)

    def call(seqs, keep, most=70, **kw):
        kept = torch.full((2, len(seqs), 2, most), 9, dtype=torch.int32, device=DEV)
        assert kept is not None
        crg.gdn_pages_evict(kw.get("table", table), kw.get("lens", lens), refs, i32(seqs), i32(keep), kw.get("mass", mass),
                            pools, page, most, 2, workspace=ws)
        st = ws.status()
        ws.reset()
        for a, b in zip(before, [*state[:4], *pools]):
            assert torch.equal(a, b), (seqs, keep)
        return st
    for seqs, keep in (([0, 0], [10, 10]), ([0, 3], [10, 10]), ([0, -1], [10, 10]), ([1, 0], [10, -1]), ([1, 0], [10, 71]),
                       ([0, 1, 2], [60, 40, 60])):  # the last: eleven pages of six
        assert call(seqs, keep) == crg.GDN_ERR_PAGES, (seqs, keep)
    for entry, want in ((-1, crg.GDN_ERR_PAGES), (10 ** 9, crg.GDN_ERR_BOUNDS), (-7, crg.GDN_ERR_BOUNDS)):
        bad = table.clone()
        bad[1, 3] = entry
        assert call([0, 1], [10, 10], table=bad) == want
    long = lens.clone()
    long[1] = 10 ** 6
    assert call([0, 1], [10, 10], lens=long) == crg.GDN_ERR_PAGES
    assert call([0, 1], [10, 10], mass=mass[..., :99]) == crg.GDN_ERR_BOUNDS
    crg.gdn_paged_status_reset()
    crg.gdn_pages_evict(table, lens, refs, i32([0, 0]), i32([1, 1]), mass, pools, page, 1)
    assert crg.gdn_paged_status() == crg.GDN_ERR_PAGES
    crg.gdn_paged_status_reset()


def test_python_refusals(crg):
    page = 16
    table, lens, refs, mass, pools = make(11, [100, 60], 2, 2, 16, page, spare=6)
    call = lambda m=mass, p=pools, s=i32([0]), k=i32([5]): crg.gdn_pages_evict(table, lens, refs, s, k, m, p, page, 5)  # noqa: E731
    for kw, err in ((dict(m=mass.double()), TypeError), (dict(m=mass[0]), TypeError), (dict(m=mass[:, :1]), ValueError),
                    (dict(m=mass[:, :, :, :1].expand(-1, -1, -1, 100)), TypeError),
                    (dict(m=mass[:1].expand(2, -1, -1, -1)), ValueError), (dict(p=pools[:3]), ValueError),
                    (dict(p=[x[:, :, :1] for x in pools]), ValueError), (dict(p=[x.transpose(1, 2) for x in pools]), ValueError),
                    (dict(s=i32([0]).long()), TypeError), (dict(k=i32([5, 6])), TypeError), (dict(m=mass.cpu()), ValueError)):
        with pytest.raises(err):
            call(**kw)


def test_stream_and_graph(crg):
    """On another stream; and captured, where a replay follows the lengths and weights of the moment."""
    page = 16
    state = make(12, [100, 60], 1, 2, 16, page, spare=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    model = Model(*state, page)
    table, lens, refs, mass, pools = state
    seqs, keep = i32([1, 0]), i32([50, 50])
    kept = crg.gdn_pages_evict(table, lens, refs, seqs, keep, mass, pools, page, 50, 4, want_kept=True, stream=side)
    side.synchronize()
    assert np.array_equal(kept.cpu().numpy(), model.evict([1, 0], [50, 50], 4, 50))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        crg.gdn_pages_evict(table, lens, refs, seqs, keep, mass, pools, page, 50, 4)
    keep.copy_(i32([33, 12]))
    mass.copy_(mass.flip(-1))
    model = Model(*state, page)
    graph.replay()
    torch.cuda.synchronize()
    model.evict([1, 0], [33, 12], 4, 50)
    for a, b in ((table, model.table), (lens, model.lens), (refs, model.refs), (mass, model.mass)):
        assert np.array_equal(a.cpu().numpy(), b)
    for p, b in zip(pools, model.pools):
        assert np.array_equal(p.float().cpu().numpy(), b)


def test_pages_past_32_bits(crg):
    """Pages more than 2^31 bytes apart."""
    stride = (1 << 31) + 256
    buf = torch.zeros(3 * stride + 4096, dtype=torch.uint8, device=DEV).view(torch.bfloat16)
    pool = buf.as_strided((4, 8, 1, 64), (stride // 2, 64, 64, 1), 0)
    pool.copy_(torch.randn((4, 8, 1, 64), device=DEV))
    table, lens, refs = i32([[3, 1, -1]]), i32([16]), i32([0, 1, 0, 1])
    mass = torch.rand((1, 1, 1, 16), device=DEV)
    assert run(crg, (table, lens, refs, mass, [pool]), 8, [0], [11], 2) is not None


@pytest.mark.parametrize("keep", [[10, 10], [60, 40]])
def test_pages_that_nobody_holds_are_refused(crg, keep):
    """They are free for the fresh ones: rows would be written over while they are read."""
    page = 16
    table, lens, refs, mass, pools = make(13, [100, 60], 2, 2, 16, page, spare=12)
    refs[int(table[1, 2])] = 0
    state = [table, lens, refs, mass, *pools]
    before = [t.clone() for t in state]
    ws = crg.Workspace(1 << 20, DEV)
    crg.gdn_pages_evict(table, lens, refs, i32([0, 1]), i32(keep), mass, pools, page, 70, 2, workspace=ws)
    assert ws.status() == crg.GDN_ERR_PAGES
    for a, b in zip(state, before):
        assert torch.equal(a, b)
