"""A fork whose parents name pages that are not there changes nothing and says why."""
import pytest
import torch

import chunked_recurrence_gb300 as crg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

PAGE = 16


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(width, full, part):
    """Two parents of `full` pages and `part` more tokens, two empty rows, some free pages."""
    n = 2 * (full + 1) + 5
    table = torch.full((5, width), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(n, generator=torch.Generator().manual_seed(width)).to(torch.int32)
    held = full + (part > 0)
    for s in range(2):
        table[s, :held] = order[s * held: (s + 1) * held].cuda()
    lens = i32(full * PAGE + part, full * PAGE + part, 0, 0, 0)
    refs = torch.zeros(n, dtype=torch.int32, device="cuda")
    refs[table[:2, :held].flatten().long()] = 1
    pools = [torch.rand(n, 33, device="cuda") for _ in range(2)]
    return table, lens, refs, pools


# few entries (checked by the plan) and many (by a kernel of their own)
@pytest.mark.parametrize("width,full", [(9, 8), (3000, 1000), (3000, 2998)])
@pytest.mark.parametrize("part", [0, 5])
def test_pages_outside_the_cache(width, full, part):
    table, lens, refs, pools = _state(width, full, part)
    n = refs.numel()
    ws = crg.Workspace(crg.gdn_pages_workspace_bytes(n, 5), "cuda")
    bad = [(1, k, page, crg.GDN_ERR_BOUNDS) for k in (0, full // 2, full - 1) for page in (n, 2 ** 31 - 1, -2, -2 ** 31)]
    if part:
        bad += [(1, full, n, crg.GDN_ERR_BOUNDS), (0, full, -7, crg.GDN_ERR_BOUNDS), (1, full, -1, crg.GDN_ERR_PAGES)]
    for row, k, page, status in bad:
        t = table.clone()
        t[row, k] = page
        before = [x.clone() for x in (t, lens, refs, *pools)]
        for parents, children in ((i32(0, 1), i32(3, 2)), (i32(1, 0, 1), i32(2, 3, 4)), (i32(row), i32(4))):
            crg.gdn_pages_fork(t, lens, refs, parents, children, pools, PAGE, workspace=ws)
            assert ws.status() == status, (row, k, page)
            ws.reset()
            assert all(torch.equal(a, b) for a, b in zip(before, (t, lens, refs, *pools))), (row, k, page)
    # entries past a parent's end are nobody's, and a full page may have been given back
    t = table.clone()
    t[0, full + (part > 0):] = 2 ** 30
    freed = int(t[1, 0])
    t[1, 0] = -1
    r = refs.clone()
    r[freed] = 0
    crg.gdn_pages_fork(t, lens, r, i32(0, 1), i32(3, 2), pools, PAGE, workspace=ws)
    assert ws.status() == crg.GDN_OK
    assert lens.tolist() == [full * PAGE + part] * 2 + [full * PAGE + part] * 2 + [0]
    assert torch.equal(t[3, :full], t[0, :full]) and torch.equal(t[2, :full], t[1, :full])
    want = refs.clone()
    want[freed] = 0
    for row in (0, 1):
        held = t[row, :full].long()
        want[held[held >= 0]] += 1
    for row, parent in ((3, 0), (2, 1)):
        if part:
            new = int(t[row, full])
            assert want[new] == 0
            want[new] = 1
            assert all(torch.equal(p[new], p[int(t[parent, full])]) for p in pools)
    assert torch.equal(r, want)
