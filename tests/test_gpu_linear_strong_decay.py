"""The decay's gradient where little is left of the state: dg_t = e^{g_t} <H_{t-1}, dL/dH_t> is
small beside products that no decay touches, such as the last token's own with dhT, and has to be
exact all the same."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [-2.0, -4.0, -8.0])
@pytest.mark.parametrize("T", [13, 64, 100])
@pytest.mark.parametrize("dt,dk,dv", [(torch.float32, 64, 128), (torch.float32, 40, 36),
                                      (torch.bfloat16, 50, 70), (torch.bfloat16, 64, 128)])
def test_strong_decays(dt, dk, dv, T, g):
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen)
    q, k = (r(1, 2, T, dk).to(dt) for _ in range(2))
    v, do = (r(1, 2, T, dv).to(dt) for _ in range(2))
    h0, dhT = r(1, 2, dk, dv), r(1, 2, dk, dv)
    gs = g * (0.8 + 0.4 * torch.rand(1, 2, T, generator=gen))
    cuda = lambda *x: [t.cuda() for t in x]
    got = ck.linear_bwd(*cuda(q, k, v, gs, do), h0=h0.cuda(), dhT=dhT.cuda(), scale=dk ** -0.5)
    want = ref.linear(q, k, v, gs, h0, scale=dk ** -0.5, do=do, dhT=dhT)
    # on CUDA cores everything is fp32; on the tensor cores the states pass in two bf16 parts
    chunks = dt == torch.bfloat16 and dk % 8 == 0 and dv % 8 == 0
    ref.check(got[3], want[5], ref.decay_tol(dt if chunks else torch.float32, T), "dg")
    for n, a, b in zip(("dq", "dk", "dv"), got, want[2:]):
        ref.check(a, b, ref.token_tol(dt, T), n)
