"""What a call without a workspace finds wrong on the GPU can be asked for, and what one with a workspace finds stays
in that."""
import pytest
import torch

import chunked_recurrence_gb300 as crg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def clean():
    crg.gdn_paged_status_reset()
    yield
    crg.gdn_paged_status_reset()


def _tables():
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    return table, i32(0, 0, 0), torch.zeros(6, dtype=torch.int32, device="cuda")


def test_refused_growth():
    tables = _tables()
    crg.gdn_pages_grow(*tables, i32(0, 1), i32(40, 20), 16)
    assert crg.gdn_paged_status() == crg.GDN_OK
    before = [t.clone() for t in tables]
    crg.gdn_pages_grow(*tables, i32(0, 1), i32(64, 64), 16)
    assert crg.gdn_paged_status() == crg.GDN_ERR_PAGES
    assert all(torch.equal(a, b) for a, b in zip(before, tables))
    crg.gdn_pages_grow(*tables, i32(0), i32(41), 16)  # the first error stays until it is cleared
    assert crg.gdn_paged_status() == crg.GDN_ERR_PAGES
    crg.gdn_paged_status_reset()
    assert crg.gdn_paged_status() == crg.GDN_OK


def test_refused_fork_and_free():
    tables = _tables()
    pool = torch.zeros(6, 8, device="cuda")
    crg.gdn_pages_grow(*tables, i32(0, 1), i32(60, 20), 16)
    crg.gdn_pages_fork(*tables, i32(0), i32(2), [pool], 16)
    assert crg.gdn_paged_status() == crg.GDN_ERR_PAGES and tables[1].tolist() == [60, 20, 0]
    crg.gdn_paged_status_reset()
    crg.gdn_pages_free(*tables, i32(9), 16)
    assert crg.gdn_paged_status() == crg.GDN_ERR_PAGES
    crg.gdn_paged_status_reset()
    tables[0][1, 0] = 77
    crg.gdn_pages_compact(*tables, [pool], 16)
    assert crg.gdn_paged_status() == crg.GDN_ERR_BOUNDS
    crg.gdn_paged_status_reset()
    crg.gdn_pages_copy([pool], i32(1, 9), i32(2, 3))
    assert crg.gdn_paged_status() == crg.GDN_ERR_BOUNDS


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("simt", [False, True])
def test_bad_pages(dtype, simt):
    cache = torch.zeros(4, 16, 2, 64, device="cuda", dtype=dtype)
    q, k = torch.zeros(2, 4, 64, device="cuda", dtype=dtype), torch.zeros(2, 2, 64, device="cuda", dtype=dtype)
    table, lens = i32([0, 1], [2, 99]), i32(20, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call in (lambda **kw: crg.gdn_kv_append(k, k, cache, cache.clone(), table, lens, **kw),
                 lambda **kw: crg.gdn_paged_attn(q, cache, cache, table, lens, simt=simt, **kw)):
        ws = crg.Workspace(1 << 26, "cuda")
        call(workspace=ws)
        assert ws.status() == crg.GDN_ERR_BOUNDS and crg.gdn_paged_status() == crg.GDN_OK
        call(stream=side)
        assert crg.gdn_paged_status(stream=side) == crg.GDN_ERR_BOUNDS
        crg.gdn_paged_status_reset(stream=side)
        assert crg.gdn_paged_status("cuda:0", side) == crg.GDN_OK


def test_wait_that_runs_out():
    cache = torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    crg.gdn_paged_attn(q, cache, cache, i32([0, 1], [2, 3]), i32(20, 20), _test_no_wait=True)
    assert crg.gdn_paged_status() == crg.GDN_ERR_TIMEOUT
    torch.cuda.synchronize()
