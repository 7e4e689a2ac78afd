"""The 64-bit references of short convolution, selective scan and RMS norm against torch's
autograd of the formulas and against differences, on the CPU."""
import pytest
import torch

import ssm_ref as ref


def r(gen, *s):
    return torch.randn(*s, generator=gen, dtype=torch.float64)


EPS = 1e-6


def numeric(loss, t, count=6, eps=EPS):
    """Differences of loss() in some entries of t, which loss() reads."""
    flat = t.view(-1)
    got = {}
    for i in range(0, flat.numel(), max(1, flat.numel() // count)):
        was = flat[i].item()
        flat[i] = was + eps
        up = loss()
        flat[i] = was - eps
        got[i] = float(up - loss()) / (2 * eps)
        flat[i] = was
    return got


def near(grad, diffs, terms):
    """A difference is off by the third derivative (1e-7 of what is near one) and by the two
    losses' roundings: 64 of 2^-53 of the sum of their terms' sizes, over 2 EPS."""
    for i, v in diffs.items():
        tol = 1e-7 * (1 + abs(v)) + 64 * 2 ** -53 * terms / EPS
        assert abs(float(grad.reshape(-1)[i]) - v) <= tol, (i, float(grad.reshape(-1)[i]), v, tol)


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 3, 9, 9]])
@pytest.mark.parametrize("W,silu", [(2, True), (3, False), (4, True)])
def test_conv_gradients_against_differences(cu, W, silu):
    gen = torch.Generator().manual_seed(W)
    B, n = (2, 2) if cu is None else (1, 5)
    x, w, b = r(gen, B, 9, 3), r(gen, 3, W), r(gen, 3)
    h0, dy, dhT = r(gen, n, W - 1, 3), r(gen, B, 9, 3), r(gen, n, W - 1, 3)

    def loss():
        y, hT = ref.conv(x, w, b, h0, cu, silu)
        return (y * dy).sum() + (hT * dhT).sum()
    y, hT, g, _ = ref.conv(x, w, b, h0, cu, silu, dy, dhT)
    terms = float((y * dy).abs().sum() + (hT * dhT).abs().sum())
    for t, name in ((x, "dx"), (w, "dw"), (b, "db"), (h0, "dh0")):
        near(g[name], numeric(loss, t, 12), terms)


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 3, 9, 9]])
@pytest.mark.parametrize("G,softplus,gate", [(1, True, True), (2, False, True), (2, True, False)])
def test_scan_gradients_against_differences(cu, G, softplus, gate):
    gen = torch.Generator().manual_seed(G)
    B, n, D, N = (2, 2, 4, 3) if cu is None else (1, 5, 4, 3)
    x, dt, A = r(gen, B, 9, D), r(gen, B, 9, D), -torch.exp(r(gen, D, N))
    Bm, C, skip, bias = r(gen, B, 9, G, N), r(gen, B, 9, G, N), r(gen, D), r(gen, D)
    z = r(gen, B, 9, D) if gate else None
    h0, dy, dhT = r(gen, n, D, N), r(gen, B, 9, D), r(gen, n, D, N)

    def loss():
        y, hT = ref.scan(x, dt, A, Bm, C, skip, z, bias, h0, cu, softplus)
        return (y * dy).sum() + (hT * dhT).sum()
    y, hT, g, _ = ref.scan(x, dt, A, Bm, C, skip, z, bias, h0, cu, softplus, dy, dhT)
    terms = float((y * dy).abs().sum() + (hT * dhT).abs().sum())
    for t, name in ((x, "dx"), (dt, "ddt"), (A, "dA"), (Bm, "dB"), (C, "dC"), (skip, "dD"), (z, "dz"),
                    (bias, "ddt_bias"), (h0, "dh0")):
        if t is not None:
            near(g[name], numeric(loss, t, 12), terms)


def test_rms_gradients_against_autograd():
    gen = torch.Generator().manual_seed(1)
    h, w, dy, dh = r(gen, 5, 7).requires_grad_(), r(gen, 7).requires_grad_(), r(gen, 5, 7), r(gen, 5, 7)
    rstd = (h.square().mean(-1) + 1e-5).rsqrt()
    ((h * rstd[:, None] * w * dy).sum() + (h * dh).sum()).backward()
    y, rs = ref.rms(h, w, 1e-5)
    dx, dw, _ = ref.rms_bwd(dy, h, rs, w, dh)
    torch.testing.assert_close(y, (h * rstd[:, None] * w).detach())
    torch.testing.assert_close(dx, h.grad)
    torch.testing.assert_close(dw, w.grad)
