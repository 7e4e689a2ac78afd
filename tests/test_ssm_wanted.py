"""An initial state's gradient is formed only where it is wanted (with the library's calls
replaced: which of them the autograd functions ask for it)."""
import pytest
import torch


def run(name, ck, monkeypatch, h0):
    asked = []
    like = torch.ones_like

    def back(n):
        def f(dy, x, *a, **kw):
            asked.append(kw["store_dh0"])
            given = [x, *a[:n - 1]]
            return (*(None if t is None else like(t) for t in given), like(h0) if kw["store_dh0"] else None)
        return f
    x = torch.randn(1, 3, 4, requires_grad=True)
    if name == "short_conv":
        monkeypatch.setattr(ck, "conv_fwd", lambda x, *a, **kw: (x * x, x[:, :1].clone()))
        monkeypatch.setattr(ck, "conv_bwd", back(3))
        y, _ = ck.short_conv(x, torch.ones(4, 4), None, h0)
    else:
        monkeypatch.setattr(ck, "scan_fwd", lambda x, *a, **kw: (x * x, x[:, :1].clone()))
        monkeypatch.setattr(ck, "scan_bwd", back(8))
        y, _ = ck.selective_scan(x, torch.ones(1, 3, 4), torch.ones(4, 2), torch.ones(1, 3, 2), torch.ones(1, 3, 2), h0=h0)
    y.sum().backward()
    assert x.grad is not None
    return asked


@pytest.mark.parametrize("name", ["short_conv", "selective_scan"])
def test_initial_state(name, monkeypatch):
    import gated_delta_rule_ckda_gb300 as ck
    h0 = torch.randn(1, 3, 4)
    assert run(name, ck, monkeypatch, h0) == [False]
    h0.requires_grad_()
    assert run(name, ck, monkeypatch, h0) == [True]
    assert torch.equal(h0.grad, torch.ones_like(h0))
