"""The 64-bit linear-attention and layer-norm references: the recurrence
against the sum over all pairs, the gradients against differences and autograd."""
import pytest
import torch

import linear_ref as ref


def make(B, H, Hk, T, dk, dv, seed, h0=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    return dict(q=r(B, Hk, T, dk), k=r(B, Hk, T, dk), v=r(B, H, T, dv),
                g=-torch.rand(B, H, T, generator=g, dtype=torch.float64),
                h0=r(B, H, dk, dv) if h0 else None)


def test_recurrence_is_the_sum_over_pairs():
    x = make(2, 4, 2, 9, 5, 3, 0)
    o, hT = ref.linear(**x, scale=0.7)
    L = x["g"].cumsum(-1)
    for b in range(2):
        for h in range(4):
            q, k, v = x["q"][b, h // 2], x["k"][b, h // 2], x["v"][b, h]
            for t in range(9):
                want = torch.exp(L[b, h, t]) * (q[t] @ x["h0"][b, h])
                for j in range(t + 1):
                    want = want + torch.exp(L[b, h, t] - L[b, h, j]) * (q[t] @ k[j]) * v[j]
                assert torch.allclose(o[b, h, t], 0.7 * want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("per_head", [False, True])
def test_gradients_against_differences(per_head):
    x = make(2, 4, 2, 6, 3, 4, 1)
    if per_head:
        x["g"] = x["g"][0, :, 0].clone()
    gen = torch.Generator().manual_seed(2)
    do = torch.randn(2, 4, 6, 4, generator=gen, dtype=torch.float64)
    dhT = torch.randn(2, 4, 3, 4, generator=gen, dtype=torch.float64)

    def loss():
        o, hT = ref.linear(**x, scale=0.5)
        return float((o * do).sum() + (hT * dhT).sum())

    grads = dict(zip("q k v g h0".split(), ref.linear(**x, scale=0.5, do=do, dhT=dhT)[2:]))
    for name, t in x.items():
        flat, g = t.view(-1), grads[name].reshape(-1)
        assert g.shape == flat.shape
        for i in range(0, flat.numel(), 5):
            keep, step = float(flat[i]), 1e-5
            flat[i] = keep + step
            up = loss()
            flat[i] = keep - step
            down = loss()
            flat[i] = keep
            assert abs((up - down) / (2 * step) - float(g[i])) <= 1e-7 * (1 + abs(float(g[i])))


def test_packed_is_each_sequence_alone():
    x = make(1, 2, 1, 11, 3, 3, 3, h0=False)
    cu = [0, 4, 4, 11]
    o, hT = ref.linear(**x, cu=cu)
    for n in range(3):
        part = {m: (t[:, :, cu[n]:cu[n + 1]] if t is not None else None) for m, t in x.items()}
        po, ph = ref.linear(**part)
        assert torch.equal(o[:, :, cu[n]:cu[n + 1]], po) and torch.equal(hT[n:n + 1], ph)


def test_reset_forgets():
    x = make(1, 1, 1, 8, 4, 4, 4)
    x["g"][0, 0, 5] = -float("inf")
    o, _ = ref.linear(**x)
    tail = {m: t[:, :, 5:] for m, t in x.items() if m != "h0"}
    assert torch.allclose(o[:, :, 5:], ref.linear(**tail)[0], rtol=1e-13, atol=1e-13)


def test_layer_norm_gradients_are_autograd():
    gen = torch.Generator().manual_seed(5)
    x, w, b, dy = (torch.randn(*s, generator=gen, dtype=torch.float64).requires_grad_()
                   for s in ((7, 12), (12,), (12,), (7, 12)))
    y = torch.nn.functional.layer_norm(x, (12,), w, b, 1e-5)
    want = torch.autograd.grad((y * dy.detach()).sum(), (x, w, b))
    yr, mean, rstd = ref.layer_norm(x, w, b, 1e-5)
    assert torch.allclose(yr, y.detach(), rtol=1e-12, atol=1e-12)
    got = ref.layer_norm_bwd(dy, x, mean, rstd, w)
    for a, r in zip(got, want):
        assert torch.allclose(a, r, rtol=1e-10, atol=1e-10)
