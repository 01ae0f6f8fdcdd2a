"""gdn_pages_evict on pages whose refs are fewer than the rows that give them back: refused, and nothing changes."""
import pytest
import torch

from tests.test_pages_evict_gpu import DEV, crg, i32, make, run  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
PAGE = 16


def refused(crg, state, seqs, keep):  # noqa: F811
    table, lens, refs, mass, pools = state
    before = [t.clone() for t in (table, lens, refs, mass, *pools)]
    ws = crg.Workspace(1 << 26, DEV)
    crg.gdn_pages_evict(table, lens, refs, i32(seqs), i32(keep), mass, pools, PAGE, max(keep), 2, workspace=ws)
    same = all(torch.equal(a, b) for a, b in zip(before, (table, lens, refs, mass, *pools)))
    return ws.status() == crg.GDN_ERR_PAGES and same


@pytest.mark.parametrize("at", [0, 4])
def test_two_rows_and_one_reference(crg, at):  # noqa: F811
    """A page in two rows, of either's place, with refs 1; with refs 2 all is well, and with one row listed."""
    def state(count):
        s = make(30, [100, 60, 80], 2, 2, 16, PAGE, spare=12)
        s[2][s[0][0, 3].long()] = count
        s[2][s[0][2, at].long()] = 0
        s[0][2, at] = s[0][0, 3]
        return s
    assert refused(crg, state(1), [0, 2], [40, 40])
    assert refused(crg, state(1), [2, 1, 0], [40, 10, 40])
    for count, seqs in ((2, [0, 2]), (1, [2]), (1, [0])):
        assert run(crg, state(count), PAGE, seqs, [40] * len(seqs), 2) is not None


def test_a_page_twice_in_a_row(crg):  # noqa: F811
    state = make(31, [100, 60], 1, 2, 16, PAGE, spare=8)
    state[0][0, 5] = state[0][0, 1]
    assert refused(crg, state, [0], [40])


def test_many_rows_and_a_large_cache(crg):  # noqa: F811
    """Counts of more rows than warps, of pages in every range of the cache."""
    n, n_pages = 90, 30000
    lens = torch.full((n,), 5 * PAGE, dtype=torch.int32, device=DEV)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3))[: n * 5].view(n, 5).int().to(DEV)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    perm[40:, 0] = perm[7, 0]  # 51 rows begin with one page
    refs.index_add_(0, perm.flatten().long(), torch.ones(n * 5, dtype=torch.int32, device=DEV))
    mass = torch.rand((1, n, 1, 5 * PAGE), device=DEV)
    pools = [torch.randn((n_pages, PAGE, 1, 4), device=DEV)]
    state = [perm.clone(), lens, refs, mass, pools]
    state[2][perm[7, 0].long()] = 50
    assert refused(crg, state, list(range(n)), [20] * n)
    for last in (0, n_pages - 1):  # a page at either end that two rows name
        s = [perm.clone(), lens.clone(), refs.clone(), mass, pools]
        s[2][perm[7, 0].long()] = 51
        s[0][3, 4] = s[0][5, 2] = last
        s[2][last] = 1
        assert refused(crg, s, list(range(n)), [20] * n)
    state[2][perm[7, 0].long()] = 51
    assert run(crg, state, PAGE, list(range(n)), [20] * n, 2) is not None


@pytest.mark.parametrize("n", [1, 3, 31, 33])
def test_any_number_of_rows(crg, n):  # noqa: F811
    """Long rows, shared by some; refs in order, then one too few for a page that all hold."""
    lens = [40 * PAGE + 5] * n
    state = make(32, lens, 1, 1, 4, PAGE, torch.float32, spare=n * 3, share=n - 1)
    before = [t.clone() for t in state[:4]], [p.clone() for p in state[4]]
    assert run(crg, state, PAGE, list(range(n)), [33] * n, 4) is not None
    if n > 1:
        state = [*before[0], before[1]]
        state[2][state[0][0, 39].long()] -= 1
        assert refused(crg, state, list(range(n)), [33] * n)
