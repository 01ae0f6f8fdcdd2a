"""The recurrent calls' workspaces, where the caller gives none: not shared by calls that may run at once."""
import threading

import pytest
import torch

import chunked_recurrence_gb300 as crg


@pytest.fixture
def on_cpu(monkeypatch):
    import ctypes
    state = {"capturing": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(crg, "_stream", lambda t, stream=None: ctypes.c_void_p(stream or 0))
    monkeypatch.setattr(crg, "_ws_cache", {})
    from contextlib import nullcontext
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device: s)
    return state


def test_threads_streams_and_graphs_have_their_own(on_cpu):
    t, got = torch.zeros(1), {}

    def take(name, stream=None):
        got[name] = crg._workspace_for(1000, t, stream)
    take("main")
    take("again")
    assert got["main"] is got["again"] and got["main"].nbytes == 1000
    take("stream", 7)
    other = threading.Thread(target=take, args=("thread",))
    other.start()
    other.join()
    on_cpu["capturing"] = True
    take("graph")
    kinds = [got[n] for n in ("main", "stream", "thread", "graph")]
    assert len({id(w) for w in kinds}) == len({w.buf.data_ptr() for w in kinds}) == 4


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_two_threads_and_two_streams():
    """The same shape, so the same size of workspace, with other values, side by side."""
    def inputs(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        return [r(2000, 2, 128).bfloat16(), r(2000, 2, 128).bfloat16(), r(2000, 4, 128).bfloat16(),
                -torch.rand((2000, 4), generator=g, device="cuda") / 20, torch.rand((2000, 4), generator=g, device="cuda")]
    args = [inputs(1), inputs(2)]
    want = [crg.gdn_chunk_fwd(*a) for a in args]
    torch.cuda.synchronize()
    for streams in ([None, None], [torch.cuda.Stream(), torch.cuda.Stream()]):
        wrong, failed = torch.zeros(2, device="cuda"), []
        torch.cuda.synchronize()

        def run(i):
            try:
                with torch.cuda.stream(streams[i]):
                    for _ in range(60):
                        for a, b in zip(crg.gdn_chunk_fwd(*args[i]), want[i]):
                            wrong[i] += (a != b).any()
            except Exception as e:  # noqa: BLE001
                failed.append(e)
        threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert not failed and wrong.tolist() == [0, 0]
