"""States of linear attention in bf16 against 64 bits, with bounds that a lost part would break,
and lengths of many segments.  The 64-bit values are made on the GPU, chunk by chunk."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def exact(q, k, v, g, h0, scale, do, dhT, C=64):
    """o, hT, dq, dk, dv, dg, dh0 of one sequence in float64, heads side by side: [H, T, d]."""
    q, k, v, g, h0, do, dhT = (t.double() for t in (q, k, v, g, h0, do, dhT))
    T = q.shape[1]
    late = torch.ones(C, C, dtype=torch.bool, device=q.device).tril()
    S, states, o = h0, [], torch.empty_like(v)

    def decays(c):
        L = g[:, c].cumsum(-1)
        D = (L[:, :, None] - L[:, None, :]).masked_fill(~late[:L.shape[1], :L.shape[1]], -torch.inf)
        return L, D.exp(), L.exp()[..., None], (L[:, -1:] - L).exp()[..., None], L[:, -1].exp()
    cuts = [slice(t, min(t + C, T)) for t in range(0, T, C)]
    for c in cuts:
        _, D, into, out, all_ = decays(c)
        states.append(S)
        o[:, c] = scale * (((q[:, c] @ k[:, c].mT) * D) @ v[:, c] + into * (q[:, c] @ S))
        S = all_[:, None, None] * S + (out * k[:, c]).mT @ v[:, c]
    hT, G, end = S, dhT, (S * dhT).sum((-1, -2))
    dq, dk, dv = (torch.empty_like(t) for t in (q, k, v))
    for c, S in zip(reversed(cuts), reversed(states)):
        _, D, into, out, all_ = decays(c)
        A, dA = scale * (q[:, c] @ k[:, c].mT) * D, scale * (do[:, c] @ v[:, c].mT) * D
        dq[:, c] = dA @ k[:, c] + scale * into * (do[:, c] @ S.mT)
        dk[:, c] = dA.mT @ q[:, c] + out * (v[:, c] @ G.mT)
        dv[:, c] = A.mT @ do[:, c] + out * (k[:, c] @ G)
        G = all_[:, None, None] * G + scale * (into * q[:, c]).mT @ do[:, c]
    x = (q * dq).sum(-1) - (k * dk).sum(-1)
    dg = x.flip(-1).cumsum(-1).flip(-1) + end[:, None]
    return o, hT, dq, dk, dv, dg, G


def state_bound(T):
    """The decayed keys (queries) enter in two bf16 parts: their factor in two, and what the
    second rounds, each 2^-17 at most and spread below it (rms 2^-17 / sqrt 3, two of them in
    quadrature), and half again for what tokens share; a walk in fp32 over the chunks and the
    eight steps of a product of 128 tokens.  A part two bits shorter would be 4 times as far."""
    return 1.5 * (2 / 3) ** 0.5 * 2.0 ** -17 + 4 * (T / 128 + 8) ** 0.5 * 2.0 ** -24


@pytest.mark.parametrize("T,H,d", [(128, 4, 128), (300, 4, 64), (1000, 3, 128), (8192, 2, 128),
                                   (32768, 1, 64), (20001, 2, 128)])
def test_against_64_bits(T, H, d):
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    q, k, v, do = (r(1, H, T, d).to(BF) for _ in range(4))
    g = -0.02 * torch.nn.functional.softplus(r(1, H, T))
    h0, dhT = r(1, H, d, d), r(1, H, d, d)
    scale = d ** -0.5
    o, hT = ck.linear_fwd(q, k, v, g, h0, scale=scale)
    grads = ck.linear_bwd(q, k, v, g, do, h0=h0, dhT=dhT, scale=scale)
    want = [t.cpu() for t in exact(*(t[0] for t in (q, k, v, g)), h0[0], scale, do[0], dhT[0])]
    got = [o[0], hT[0], *(t[0] for t in grads)]
    for n, a, b in zip(("o", "hT", "dq", "dk", "dv", "dg", "dh0"), got, want):
        tol = state_bound(T) if n in ("hT", "dh0") else \
            ref.decay_tol(BF, T) if n == "dg" else ref.token_tol(BF, T)
        print(n, "rms %.2e max %.2e" % ref.far(a, b), "tolerance %.2e" % tol)
        ref.check(a, b, tol, n)
