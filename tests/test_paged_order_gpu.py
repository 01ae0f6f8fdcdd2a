"""The paged operators start up under the kernel before them on the stream: what that one, a copy, a memset or another
stream leaves must be there when they read it, called directly and in a captured graph."""
import pytest
import torch

import chunked_recurrence_gb300 as crg

pytestmark = pytest.mark.gpu


def _before(kind, src, dst, side):
    """dst = src by way of a kernel, a copy, a copy and a memset elsewhere, or another stream."""
    if kind == "kernel":
        torch.add(src, 0, out=dst)
    elif kind == "copy":
        dst.copy_(src)
    elif kind == "memset":
        dst.copy_(src)
        torch.zeros(1 << 20, dtype=torch.uint8, device="cuda").zero_()
    else:
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(4):
                dst.copy_(src)
        torch.ones(1000, device="cuda").mul_(2)
        main.wait_stream(side)


def _check(kind, srcs, dsts, run, want):
    side = torch.cuda.Stream()

    def step():
        for s, d in zip(srcs, dsts):
            _before(kind, s, d, side)
        return run()

    for _ in range(3):
        for d in dsts:
            d.zero_()
        got = step()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for d in (*dsts, *got):
            d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


KINDS = ("kernel", "copy", "memset", "stream")


@pytest.mark.parametrize("kind", KINDS)
def test_rope_order(kind):
    torch.manual_seed(0)
    n = 20000
    freqs = crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(64))
    x, pos = torch.randn(n, 4, 64, device="cuda"), torch.arange(n, device="cuda")
    buf = torch.empty_like(x)
    want = crg.gdn_rope(x, None, pos, freqs)[:1]
    torch.cuda.synchronize()
    _check(kind, [x], [buf], lambda: crg.gdn_rope(buf, None, pos, freqs)[:1], want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype,d,new", [(torch.bfloat16, 128, 1), (torch.bfloat16, 64, 150), (torch.bfloat16, 256, 150),
                                         (torch.float32, 64, 30)])
def test_attn_order(kind, dtype, d, new):
    torch.manual_seed(0)
    n_seqs, page, hkv, hq, length = 5, 16, 2, 4, 700
    pages = -(-length // page)
    kv = [torch.randn(n_seqs * pages, page, hkv, d, device="cuda").to(dtype) for _ in range(2)]
    q = torch.randn(n_seqs * new, hq, d, device="cuda").to(dtype)
    table = torch.randperm(n_seqs * pages, device="cuda").to(torch.int32).view(n_seqs, pages)
    lens = torch.full((n_seqs,), length, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, n_seqs * new + 1, new, dtype=torch.int32, device="cuda")
    # one split into shares: with the same lengths every call sums in the same order
    want = crg.gdn_paged_attn(q, *kv, table, lens, cu, max_new=new)[:1]
    torch.cuda.synchronize()
    srcs = [q, *kv, lens]
    dsts = [torch.empty_like(t) for t in srcs]
    _check(kind, srcs, dsts, lambda: crg.gdn_paged_attn(*dsts[:3], table, dsts[3], cu, max_new=new)[:1], want)


@pytest.mark.parametrize("kind", KINDS)
def test_pages_order(kind):
    torch.manual_seed(0)
    n, page = 64, 4
    table = torch.arange(8 * 8, dtype=torch.int32, device="cuda").view(8, 8)
    table = torch.where(torch.arange(8, device="cuda")[:, None] < 4, table, -1).to(torch.int32).contiguous()
    lens = torch.tensor([30, 32, 29, 31, 0, 0, 0, 0], dtype=torch.int32, device="cuda")
    refs = (torch.arange(n, device="cuda") < 32).to(torch.int32)
    pool = torch.randn(n, page, 2, 16, device="cuda")
    parents = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    children = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    srcs = [table, lens, refs, pool]

    def run(dsts):
        crg.gdn_pages_fork(dsts[0], dsts[1], dsts[2], parents, children, [dsts[3]], page)
        crg.gdn_pages_free(dsts[0], dsts[1], dsts[2], parents[:1], page)
        crg.gdn_pages_compact(dsts[0], dsts[1], dsts[2], [dsts[3]], page)
        return [d.clone() for d in dsts]

    want = run([t.clone() for t in srcs])
    torch.cuda.synchronize()
    live = int((want[2] > 0).sum())
    want = want[:3] + [want[3][:live]]
    dsts = [torch.empty_like(t) for t in srcs]

    def step():
        got = run(dsts)
        return got[:3] + [got[3][:live]]

    _check(kind, srcs, dsts, step, want)
