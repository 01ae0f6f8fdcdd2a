"""The hybrid example's beams: a short prompt by the plain call, one that pays (or is said to) read once for all of them."""
import pytest
import torch

from tests.test_hybrid_evict_gpu import ex  # noqa: F401

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("keep", [0, 24])
def test_which_call_the_beams_take(ex, keep, monkeypatch):  # noqa: F811
    calls = {"shared": 0}
    call = ex.crg.gdn_paged_attn_shared

    def counted(*args, **kw):
        calls["shared"] += 1
        return call(*args, **kw)
    monkeypatch.setattr(ex.crg, "gdn_paged_attn_shared", counted)
    prompt = torch.arange(61, device="cuda") * 11 % 500
    ex.beams(ex.Hybrid(ex.Config(dtype=torch.float32, keep=keep)), prompt, 3, 6)
    assert calls["shared"] == 0
    least = 3 * (keep or 61) * 2 * 2 * 128 * 4  # beams, positions, k and v, kv heads, width, bytes
    ex.beams(ex.Hybrid(ex.Config(dtype=torch.float32, keep=keep, pays=least + 1)), prompt, 3, 6)
    assert calls["shared"] == 0
    texts, scores = ex.beams(ex.Hybrid(ex.Config(dtype=torch.float32, keep=keep, pays=least)), prompt, 3, 6)
    assert calls["shared"] == 5
    assert [len(t) for t in texts] == [6] * 3 and torch.isfinite(scores).all()
