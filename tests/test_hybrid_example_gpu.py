"""The hybrid example: cached single tokens, forks and compaction against whole prompts."""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("hybrid_beam", os.path.join(ROOT, "examples", "hybrid_beam.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["hybrid_beam"] = m
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return ((a - b).norm() / b.norm()).item()


def test_tokens_one_at_a_time_are_the_prompt(ex):
    """fp32: logits of tokens fed one at a time after a prompt, in forked and moved rows, equal those of the whole
    text as one prompt (both through fp32 sums of the same terms in other orders)."""
    model = ex.Hybrid(ex.Config(dtype=torch.float32))
    text = torch.arange(60, device="cuda") * 7 % 500
    whole = model.forward(text, [0], [60])
    model.free([0])
    model.forward(torch.cat([text[:41], text[:20]]), [5, 2], [41, 20])
    model.fork([5, 5], [1, 7])
    model.free([2, 5])
    model.compact()
    for t in range(41, 60):
        got = model.forward(text[t].repeat(2), [1, 7])
        assert rel(got[0], whole[t]) <= 1e-4 and rel(got[1], whole[t]) <= 1e-4, t
    assert model.check()
    model.free([1, 7])
    assert model.refs.sum().item() == 0 and model.lens.sum().item() == 0


def test_several_prompts_at_once(ex):
    """Packed prompts of other lengths do not see each other."""
    model = ex.Hybrid(ex.Config(dtype=torch.float32))
    a, b = torch.arange(33, device="cuda") % 500, torch.arange(50, device="cuda") * 3 % 500
    both = model.forward(torch.cat([a, b]), [3, 0], [33, 50])
    model.free([3, 0])
    assert rel(both[:33], model.forward(a, [1], [33])) <= 1e-5
    assert rel(both[33:], model.forward(b, [2], [50])) <= 1e-5
    assert model.check()


def test_beam_search_runs_in_bf16(ex):
    model = ex.Hybrid(ex.Config())
    prompt = torch.arange(37, device="cuda") * 11 % 500
    texts, scores = ex.beams(model, prompt, 4, 20)
    assert [len(t) for t in texts] == [20] * 4 and torch.isfinite(scores).all()
    assert scores.tolist() == sorted(scores.tolist(), reverse=True)
    assert model.refs.sum().item() == 0
