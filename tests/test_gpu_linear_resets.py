"""The decay's gradient next to many resets.  A block of 32 tokens begins with strong decays and
goes on with mild ones; dg of the mild tokens is a sum over pairs behind the last reset, with
nothing of a state in it, and has to be as exact as sums in fp32 are."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("strong", [-float("inf"), -100.0])
@pytest.mark.parametrize("resets", [1, 4, 8, 16])
@pytest.mark.parametrize("dt,d", [(torch.bfloat16, 64), (torch.bfloat16, 128), (torch.float32, 40)])
def test_mild_decays_behind_resets(dt, d, resets, strong):
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator().manual_seed(100 * d + resets)
    r = lambda *s: torch.randn(*s, generator=gen)
    T = 320
    q, k, v, do = (r(1, 2, T, d).to(dt) for _ in range(4))
    g = -0.05 * torch.nn.functional.softplus(r(1, 2, T))
    mild = torch.arange(T) % 32 >= resets
    g[:, :, ~mild] = strong
    got = ck.linear_bwd(*(x.cuda() for x in (q, k, v, g, do)), scale=d ** -0.5)
    want = ref.linear(q, k, v, g, scale=d ** -0.5, do=do)
    # a walk over the block's tokens and the columns of the two products, as for fp32 inputs: the
    # bf16 parts of a state, which other bounds allow for, have no share in these tokens
    ref.check(got[3][:, :, mild], want[5][:, :, mild], ref.decay_tol(torch.float32, 32), "dg")
    for name, a, b in zip(("dq", "dk", "dv"), got, want[2:]):
        ref.check(a, b, ref.token_tol(dt, T), name)
