"""Calls without a workspace whose kernels mix: two threads on one stream, and graphs among other calls."""
import threading

import pytest
import torch

import chunked_recurrence_gb300 as crg

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _attn(seed, n_seqs, new, length, hq, hkv, d, dtype=torch.bfloat16, page=16):
    """A call of attention whose sequences are cut over many blocks, and its output."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = -(-length // page)
    k, v = (torch.randn((n_seqs * n, page, hkv, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn((n_seqs * new, hq, d), generator=g, device="cuda").to(dtype)
    table = torch.randperm(n_seqs * n, generator=g, device="cuda").to(torch.int32).view(n_seqs, n)
    lens = torch.full((n_seqs,), length, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, n_seqs * new + 1, new, dtype=torch.int32, device="cuda")
    return lambda **kw: crg.gdn_paged_attn(q, k, v, table, lens, cu, max_new=new, want_lse=True, **kw)


def _threads(*jobs):
    failed = []

    def run(job):
        try:
            job()
        except BaseException as e:  # noqa: B036
            failed.append(e)
    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_attention_of_two_threads(dtype):
    """Small and large calls from two threads on the default stream: each gets its own outputs."""
    calls = [_attn(1, 3, 1, 5000, 8, 1, 128, dtype), _attn(2, 2, 40, 3000, 16, 2, 128, dtype)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = torch.zeros(2, device="cuda")

    def job(i):
        def run():
            for _ in range(150):
                for a, b in zip(calls[i](), want[i]):
                    wrong[i] += (a != b).any()
        return run
    _threads(job(0), job(1))
    assert wrong.tolist() == [0, 0]


def test_pages_of_two_threads():
    """Forks and compactions of two caches from two threads on the default stream."""
    def cache(n, rows, page=4):
        table = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda")
        table[: rows // 2] = torch.randperm(n, device="cuda")[: rows // 2 * 8].to(torch.int32).view(-1, 8)
        lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
        lens[: rows // 2] = torch.arange(rows // 2, device="cuda") % 7 + 25
        refs = torch.zeros(n, dtype=torch.int32, device="cuda")
        refs[table[: rows // 2].flatten().long()] = 1
        pool = torch.arange(n, device="cuda", dtype=torch.float32)[:, None].repeat(1, 64)
        return table, lens, refs, pool

    def work(state, rows):
        table, lens, refs, pool = (t.clone() for t in state)
        parents = torch.arange(rows // 2, dtype=torch.int32, device="cuda")
        crg.gdn_pages_fork(table, lens, refs, parents, parents + rows // 2, [pool], 4)
        crg.gdn_pages_free(table, lens, refs, parents[::2].contiguous(), 4)
        crg.gdn_pages_compact(table, lens, refs, [pool], 4)
        live = pool[table.clamp(min=0).long()] * (table >= 0)[..., None]
        return table, lens, refs, live

    torch.manual_seed(0)
    sizes = [(64, 8), (1000, 60)]
    states = [cache(*s) for s in sizes]
    want = [work(st, s[1]) for st, s in zip(states, sizes)]
    torch.cuda.synchronize()
    wrong = torch.zeros(2, device="cuda")

    def job(i):
        def run():
            for _ in range(100):
                for a, b in zip(work(states[i], sizes[i][1]), want[i]):
                    wrong[i] += (a != b).any()
        return run
    _threads(job(0), job(1))
    assert wrong.tolist() == [0, 0]


def test_replay_after_a_larger_call():
    """Eager and captured on one stream, then a larger call there: a replay leaves what others hold alone."""
    side = torch.cuda.Stream()
    small, large = _attn(3, 2, 1, 9000, 8, 1, 128), _attn(4, 1, 300, 2000, 32, 8, 128)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        want = small()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = small()
        large()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        others = [torch.full((5 << 20,), 7.0, device="cuda") for _ in range(8)]
        for t in got:
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in others)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_at_once():
    """Captured one after another, replayed side by side on two streams."""
    calls = [_attn(5, 2, 1, 9000, 8, 1, 128), _attn(6, 3, 5, 7000, 16, 2, 128)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, got = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append([c() for _ in range(20)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, w))


FIRST_CALL_IS_CAPTURED = """
import torch
import chunked_recurrence_gb300 as crg
cache = torch.randn(8, 16, 1, 128, device="cuda").bfloat16()
q = torch.randn(2, 4, 128, device="cuda").bfloat16()
table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
lens = torch.tensor([50, 64], device="cuda", dtype=torch.int32)
refs = torch.ones(8, device="cuda", dtype=torch.int32)
rows, to = torch.zeros(1, device="cuda", dtype=torch.int32), torch.full((1,), 60, device="cuda", dtype=torch.int32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, _ = crg.gdn_paged_attn(q, cache, cache, table, lens)
    crg.gdn_kv_append(q[:, :1].contiguous(), q[:, :1].contiguous(), cache.clone(), cache.clone(), table, lens)
    crg.gdn_pages_grow(table, lens, refs, rows, to, 16)
g.replay()
torch.cuda.synchronize()
assert crg.gdn_paged_status() == crg.GDN_OK
assert lens.tolist() == [60, 64]
lens[0] = 50
w, _ = crg.gdn_paged_attn(q, cache, cache, table, lens)
assert torch.equal(o, w)
lens.fill_(1000)
g.replay()
torch.cuda.synchronize()
assert crg.gdn_paged_status() == crg.GDN_ERR_BOUNDS
print("done")
"""


def test_first_call_of_a_process_is_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IS_CAPTURED], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-3000:]


OUT_OF_MEMORY = """
import torch
import chunked_recurrence_gb300 as crg
cache = torch.zeros(64, 16, 8, 128, device="cuda").bfloat16()
q = torch.zeros(1, 64, 128, device="cuda").bfloat16()
table, lens = torch.zeros(1, 64, device="cuda", dtype=torch.int32), torch.ones(1, device="cuda", dtype=torch.int32)
free = 24 << 20
torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + free) / torch.cuda.mem_get_info()[1])
hold = [torch.empty(8 << 20, device="cuda", dtype=torch.uint8) for _ in range(2)]
for call in (lambda: crg.gdn_paged_attn(q, cache, cache, table, lens),
             lambda: paged._like(torch.zeros(1, device="cuda").expand(1 << 27), 1, True)):
    from chunked_recurrence_gb300 import paged
    try:
        call()
    except torch.OutOfMemoryError:
        print("out of memory")
del hold
crg.gdn_paged_attn(q, cache, cache, table, lens)
torch.cuda.synchronize()
print("done")
"""


def test_memory_that_runs_out_is_torchs_error():
    """Outputs and scratch that the allocator refuses (a limit of this process's own) raise what torch's do."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", OUT_OF_MEMORY], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split("\n")[:3] == ["out of memory"] * 2 + ["done"], r.stdout + r.stderr[-3000:]
