"""The example layer of linear attention: it trains, and serving token by token
agrees with one call over the whole sequences."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "linear_attention.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("linear_attention_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 96), (20, 36)])
def test_train_and_serve(example, dk, dv):
    losses, got, want = example.main(["--steps", "25", "--dk", str(dk), "--dv", str(dv)])
    assert torch.isfinite(losses).all()
    assert losses[-3:].mean() < losses[:3].mean()
    # Both sides round at most eight values in a row to bf16 (norm, projection,
    # weights of the tokens, state's parts, o, norm, output projection, sum), each
    # by at most 2^-8 of it; the sides may round apart in each.
    assert (got.double() - want.double()).norm() <= 8 * 2 ** -8 * want.double().norm()
    assert got.shape == (4, 20, 256)


def test_layer_gradients_by_differences(example):
    """The whole layer in fp32 along a random direction, against a central
    difference in steps of h.  The loss has errors of a few 2^-24 of its terms'
    size, so the difference has at most that over h; a unit direction moves each row by
    a small part of itself, so the third derivative's term is below h^2 of that size."""
    gen = torch.Generator().manual_seed(3)
    B, H, T, d = 1, 2, 70, 16
    mk = lambda *s: torch.randn(*s, generator=gen).cuda()
    q, k, v = mk(B, 1, T, d), mk(B, 1, T, d), mk(B, H, T, d)
    g = -mk(B, H, T).abs() * 0.2
    w, b, r = 1 + 0.1 * mk(d), 0.1 * mk(d), mk(B, H, T, d)
    x = [z.requires_grad_() for z in (q, k, v, g, w, b)]
    ck = example.ck

    def loss(q, k, v, g, w, b):
        qn = ck.layer_norm(q)
        o, _ = ck.linear_attention(qn, ck.layer_norm(k), v, g, scale=0.25)
        return (ck.layer_norm(o, w, b).double() * r.double()).sum()

    grads = torch.autograd.grad(loss(*x), x)
    h = 1e-2
    scale = r.double().norm().item()  # the loss is a sum of N terms of random sign
    for i, gr in enumerate(grads):
        u = mk(*x[i].shape)
        u /= u.norm()
        with torch.no_grad():
            up = [z if j != i else z + h * u for j, z in enumerate(x)]
            dn = [z if j != i else z - h * u for j, z in enumerate(x)]
            diff = ((loss(*up) - loss(*dn)) / (2 * h)).item()
        got = (gr.double() * u.double()).sum().item()
        assert abs(got - diff) <= scale * (16 * 2 ** -24 / h + h * h), (i, got, diff)
