"""A thread whose first CUDA call is one of the library's: the context becomes current in it before tensor maps are made."""
import threading

import pytest
import torch

import chunked_recurrence_gb300 as crg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _in_a_thread(call):
    """call() in a new thread, its outputs and scratch from blocks that the allocator holds already."""
    want = call()
    torch.cuda.synchronize()
    got = []

    def run():
        try:
            got.append(call())
        except Exception as e:  # noqa: BLE001
            got.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if isinstance(got[0], Exception):
        raise got[0]
    assert all(torch.equal(a, b) for a, b in zip(got[0], want))


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention(dtype, new):
    cache = torch.randn(20, 16, 1, 128, device="cuda").to(dtype)
    q = torch.randn(new, 4, 128, device="cuda").to(dtype)
    table = torch.arange(20, device="cuda", dtype=torch.int32)[None]
    lens, cu = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in ([310], [0, new]))
    _in_a_thread(lambda: crg.gdn_paged_attn(q, cache, cache, table, lens, cu, want_lse=True))


@pytest.mark.parametrize("kw", [dict(), dict(fused=True), dict(simt=True)], ids=str)
def test_chunk_fwd(kw):
    q, k = (torch.randn(300, 2, 128, device="cuda").bfloat16() for _ in range(2))
    v = torch.randn(300, 4, 128, device="cuda").bfloat16()
    g, beta = -torch.rand(300, 4, device="cuda") / 20, torch.rand(300, 4, device="cuda")
    _in_a_thread(lambda: crg.gdn_chunk_fwd(q, k, v, g, beta, **kw))


def test_segment_summary():
    k = torch.randn(300, 2, 128, device="cuda").bfloat16()
    v = torch.randn(300, 4, 128, device="cuda").bfloat16()
    g, beta = -torch.rand(300, 4, device="cuda") / 20, torch.rand(300, 4, device="cuda")
    bounds = torch.tensor([0, 100, 300], device="cuda", dtype=torch.int32)
    _in_a_thread(lambda: crg.gdn_segment_summary(k, v, g, beta, bounds))
