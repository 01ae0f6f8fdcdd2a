"""The hybrid example with beams over a shared prompt, and with a prompt cut to the positions that were looked at most."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("hybrid_beam_evict", os.path.join(ROOT, "examples", "hybrid_beam.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["hybrid_beam_evict"] = m
    spec.loader.exec_module(m)
    return m


def rel(a, b):
    return ((a - b).norm() / b.norm()).item()


def test_shared_tokens_are_the_plain_ones(ex):
    """fp32: forked rows' tokens with the prompt read once, against each row by itself (sums of the same terms in other
    orders)."""
    model = ex.Hybrid(ex.Config(dtype=torch.float32))
    text = torch.arange(50, device="cuda") * 7 % 500
    model.forward(text, [3], [50])
    model.fork([3] * 3, [0, 1, 6])
    for t in range(4):
        tokens = torch.tensor([5 + t, 90, 400 - t, 17], device="cuda")
        state = [x.clone() for lay in model.layers for n, x in lay.items() if n in ("state", "last")]
        at = model.at.clone()
        a = model.forward(tokens, [3, 0, 1, 6], shared=50)
        for x, y in zip([x for lay in model.layers for n, x in lay.items() if n in ("state", "last")], state):
            x.copy_(y)
        model.at.copy_(at)
        model.lens[[3, 0, 1, 6]] -= 1  # the same tokens once more, over themselves
        b = model.forward(tokens, [3, 0, 1, 6])
        assert rel(a, b) <= 1e-4
    assert model.check()


def test_all_kept_is_nothing_evicted(ex):
    prompt = torch.arange(61, device="cuda") * 11 % 500
    plain = ex.beams(ex.Hybrid(ex.Config(dtype=torch.float32)), prompt, 3, 6)
    kept = ex.beams(ex.Hybrid(ex.Config(dtype=torch.float32, keep=100)), prompt, 3, 6)
    assert plain[0] == kept[0] and torch.equal(plain[1], kept[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams_over_a_cut_prompt(ex, dtype):
    """It runs, the pages come back, and the prompt's weights add up to its tokens times the heads of a group."""
    model = ex.Hybrid(ex.Config(dtype=dtype, keep=24))
    prompt = torch.arange(150, device="cuda") * 13 % 500
    model.forward(prompt, [0], [150])
    total = model.mass[:, 0, :, :150].double().sum(-1) / (150 * model.cfg.heads // model.cfg.kv_heads)
    assert ((total - 1).abs() < 2.0 ** -8).all()
    model.evict([0])
    assert model.lens[0].item() == 24 and (model.refs > 0).sum().item() == 2 and model.at[0].item() == 150
    assert (model.mass[:, 0, :, 24:] == 0).all()
    model.free([0])
    texts, scores = ex.beams(model, prompt, 4, 12)
    assert [len(t) for t in texts] == [12] * 4 and torch.isfinite(scores).all()
    assert model.refs.sum().item() == 0 and model.check()
