"""The autograd functions have no second derivatives and say so: a gradient taken with
create_graph=True, used in another loss, raises where its term would be lost in silence.
On the CPU, with the library's calls replaced by torch's."""
import pytest
import torch


def one(name, ck, monkeypatch):
    """(function of x, x) with the calls behind it replaced."""
    like = torch.ones_like
    if name == "linear_attention":
        monkeypatch.setattr(ck, "linear_fwd", lambda q, *a, **kw: (q * q, None))
        monkeypatch.setattr(ck, "linear_bwd", lambda q, k, v, g, do, **kw: (
            2 * q * do, like(k), like(v), like(g), None))
        k, v, g = torch.ones(1, 1, 3, 4), torch.ones(1, 1, 3, 4), torch.zeros(1, 1, 3)
        return lambda x: ck.linear_attention(x, k, v, g)[0], torch.randn(1, 1, 3, 4)
    if name == "layer_norm":
        monkeypatch.setattr(ck, "layernorm_fwd", lambda x, *a, **kw: (x * x, x[..., 0], x[..., 0]))
        monkeypatch.setattr(ck, "layernorm_bwd", lambda dy, x, *a, **kw: (2 * x * dy, None, None))
        return ck.layer_norm, torch.randn(3, 4)
    if name == "recurrence":
        monkeypatch.setattr(ck, "fwd", lambda q, *a, **kw: (q * q, None))
        monkeypatch.setattr(ck, "bwd", lambda q, k, v, al, be, do, **kw: (
            2 * q * do, like(k), like(v), like(al), like(be), None))
        z = torch.ones(1, 1, 3, 4)
        return lambda x: ck.recurrence(x, z, z, z, z[..., 0])[0], torch.randn(1, 1, 3, 4)
    monkeypatch.setattr(ck, "prep", lambda k, a, b, q_raw, *x, **kw: (
        q_raw * q_raw, k.clone(), a.clone(), b.clone()))
    monkeypatch.setattr(ck, "prep_bwd", lambda k, a, b, dk, da, db, q_raw, d_q, *x, **kw: (
        2 * q_raw * d_q, dk, da, db))
    z = torch.ones(3, 4)
    return lambda x: ck.prepare(x, z, z, z[..., 0])[0], torch.randn(3, 4)


@pytest.mark.parametrize("name", ["linear_attention", "layer_norm", "recurrence", "prepare"])
def test_a_gradient_penalty_is_refused(name, monkeypatch):
    import gated_delta_rule_ckda_gb300 as ck
    f, x = one(name, ck, monkeypatch)
    x.requires_grad_()
    y = f(x)
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    torch.testing.assert_close(g, 2 * x)
    with pytest.raises(RuntimeError, match="no second derivative"):
        (f(x).sum() + g.square().sum()).backward()
    # by way of the gradient that comes in as well, and not where no second one is asked for
    (g,) = torch.autograd.grad(f(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        g.sum().backward()
    x.grad = None
    f(x).sum().backward()
    torch.testing.assert_close(x.grad, 2 * x.detach())
    assert not x.grad.requires_grad
