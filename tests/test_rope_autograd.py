"""gdn_rope under autograd: its gradient is its own transposed rotation, and nothing ends without a word."""
import pytest
import torch

import chunked_recurrence_gb300 as crg
from chunked_recurrence_gb300 import GDN_FLAG_ROPE_BACKWARD, paged


@pytest.fixture
def calls(monkeypatch):
    """The binding on CPU tensors; the library's calls are recorded and leave ones."""
    seen = []

    def entry(name):
        def call(q, k, positions, freqs, *rest):
            for t in rest[-3:-1]:
                if t is not None:
                    t.fill_(1)
            seen.append((q is not None, k is not None, rest[-4]))
            return 0
        return call
    for name, to in (("_entry", entry), ("_need_cuda", lambda *t: None), ("_handle", lambda t, stream: 0), ("_plans", {})):
        monkeypatch.setattr(paged, name, to)
    return seen


def _inputs(grad_q=True, grad_k=True):
    return (torch.randn(5, 4, 64, requires_grad=grad_q), torch.randn(5, 2, 64, requires_grad=grad_k), torch.arange(5),
            crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(64), "cpu"))


def test_outputs_carry_gradients(calls):
    q, k, *rest = _inputs()
    qo, ko = crg.gdn_rope(q, k, *rest)
    assert qo.requires_grad and ko.requires_grad
    (qo.sum() + ko.sum()).backward()  # broadcast gradients
    assert calls == [(True, True, 0), (True, True, GDN_FLAG_ROPE_BACKWARD)]
    assert q.grad.eq(1).all() and k.grad.eq(1).all()


def test_only_what_is_asked_for(calls):
    q, k, *rest = _inputs(grad_k=False)
    qo, ko = crg.gdn_rope(q, k, *rest, backward=True)
    qo.sum().backward()
    assert calls == [(True, True, GDN_FLAG_ROPE_BACKWARD), (True, False, 0)] and k.grad is None
    q, k, *rest = _inputs()
    crg.gdn_rope(q, k, *rest)[1].sum().backward()
    assert calls[-1] == (False, True, GDN_FLAG_ROPE_BACKWARD) and q.grad is None
    assert crg.gdn_rope(None, k, *rest)[1].requires_grad
    with torch.no_grad():
        assert not crg.gdn_rope(q, k, *rest)[0].requires_grad
    assert not crg.gdn_rope(q.detach(), k.detach(), *rest)[0].requires_grad


def test_given_outputs_are_refused(calls):
    q, k, *rest = _inputs()
    with pytest.raises(ValueError, match="gradients"):
        crg.gdn_rope(q, k, *rest, q_out=torch.empty(5, 4, 64))
    assert calls == []
    with torch.no_grad():
        crg.gdn_rope(q, k, *rest, q_out=torch.empty(5, 4, 64))
    assert len(calls) == 1


def _plain(x, pos, inv, rd, inter, scale):
    a = pos.double()[:, None, None] * inv.to(x.device)
    c, s = scale * a.cos(), scale * a.sin()
    r = x[..., :rd]
    x1, x2 = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., : rd // 2], r[..., rd // 2:])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    y = torch.stack((y1, y2), -1).flatten(-2) if inter else torch.cat((y1, y2), -1)
    return torch.cat((y, x[..., rd:]), -1)


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("own_stream", [False, True])
def test_gradients(inter, own_stream):
    """fp32 gradients of a shared leaf against autograd of the formula in 64 bits: two products of 2^-23 each way and
    their sum for cos and sin of 2^-23, at most 2^-20 of |dy1| + |dy2|."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    n, d, rd = 37, 64, 48
    x = torch.randn(n, 6, d, generator=g, device="cuda")
    weight = torch.randn(n, 6, d, generator=g, device="cuda").transpose(0, 1).contiguous().transpose(0, 1)
    pos = torch.randint(0, 5000, (n,), generator=g, device="cuda")
    inv = crg.gdn_rope_inv_freq(rd)
    freqs = crg.gdn_rope_freqs(inv)
    leaf, exact = x.clone().requires_grad_(), x.double().requires_grad_()
    torch.cuda.synchronize()
    kw = dict(stream=torch.cuda.Stream()) if own_stream else {}
    q, k = crg.gdn_rope(leaf[:, :4], leaf[:, 3:], pos, freqs, inter, 1.25, **kw)  # the fourth head is in both
    if own_stream:
        torch.cuda.current_stream().wait_stream(kw["stream"])
    loss = (q * weight[:, :4]).sum() + (k * weight[:, 3:]).sum()
    loss.backward()
    torch.cuda.synchronize()
    y = _plain(exact, pos, inv, rd, inter, 1.25)
    ((y[:, :4] * weight[:, :4].double()).sum() + (y[:, 3:] * weight[:, 3:].double()).sum()).backward()
    size = 1.25 * 2 * 2 * weight.abs().amax().double()  # both uses of a head, both elements of a pair
    assert (leaf.grad.double() - exact.grad).abs().max() <= 2.0 ** -20 * size
    assert leaf.grad.abs().amax() > 1


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")
def test_gradient_of_the_gradient():
    """The step is linear, so the gradient of its gradient is the step itself, by the same kernel."""
    x = torch.randn(9, 2, 64, device="cuda", requires_grad=True)
    dy = torch.randn(9, 2, 64, device="cuda", requires_grad=True)
    u = torch.randn(9, 2, 64, device="cuda")
    pos, freqs = torch.arange(9, device="cuda"), crg.gdn_rope_freqs(crg.gdn_rope_inv_freq(64))
    y, _ = crg.gdn_rope(x, None, pos, freqs)
    dx, = torch.autograd.grad(y, x, dy, create_graph=True)
    back, = torch.autograd.grad(dx, dy, u)
    want, _ = crg.gdn_rope(u, None, pos, freqs)
    assert torch.equal(back, want)
