"""The product of thousands of decays in a row that stays whole.  A mean error of single
decays adds up over a state's memory (2^-o tokens, where delta |A| log2(e) is near 2^o), and
only there: rows that are cut take one exponential over each piece."""
import pytest
import torch

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def steps(rows, T, D, o):
    gen = torch.Generator(device="cuda").manual_seed(-o)
    r = torch.rand(rows, T, D, generator=gen, device="cuda")
    A = -(1 + 0.01 * torch.rand(D, 4, generator=gen, device="cuda"))
    return r.exp2_().mul_(2.0 ** o / LOG2E), A


def drift(got, delta, A, o):
    """Mean relative error of a product of T decays, over the tokens of a memory."""
    total = delta.double().sum(1)   # [rows, D]
    want = torch.exp(total[..., None] * A.double())
    return float((got.double() / want - 1).mean()) / delta.shape[1] * 2.0 ** -o


def tolerance(o):
    """The exponential's mean error by octaves is -2.7e-8 to -1.4e-8 for arguments of 2^-8 to
    2^-1 and -9e-9 to -5e-9 below 2^-9.  One addend takes out the middle of the second, which
    leaves 2e-9 a token of those, and of the first 2e-8 over 128 tokens or 1e-8 over 256: less
    than 3e-6.  (Without the addend, or with one that suits the first alone, 2^-12 is off by
    2.4e-5 and 4.7e-5.)"""
    return 3e-6 + 2.0 ** -o * 2e-9


@pytest.mark.parametrize("o", [-14, -13, -12, -11, -10, -9, -8, -7])
def test_forward(ck, o):
    rows, T, D = 32, min(2048, 2 ** (5 - o)), 1024   # (a state decays by 2^-50 at most)
    assert ck.lib().ckda_scan_fwd_workspace_bytes(rows, T, D, 4, 1) == 0
    delta, A = steps(rows, T, D, o)
    none, B = torch.zeros_like(delta), torch.zeros(rows, T, 4, device="cuda")
    _, hT = ck.scan_fwd(none, delta, A, B, B, h0=torch.ones(rows, D, 4, device="cuda"), softplus=False)
    off = drift(hT, delta, A, o)
    assert abs(off) <= tolerance(o), f"{off:.2e} over 2^{-o} tokens (tolerance {tolerance(o):.2e})"


@pytest.mark.parametrize("o", [-12, -8])
def test_backward(ck, o):
    """dh0 from hT's gradient alone is the same product; 58 rows of 1024 channels are whole in
    the backward pass."""
    rows, T, D = 58, 2048, 1024
    delta, A = steps(rows, T, D, o)
    none, B, one = torch.zeros_like(delta), torch.zeros(rows, T, 4, device="cuda"), torch.ones(rows, D, 4, device="cuda")
    dh0 = ck.scan_bwd(none, none, delta, A, B, B, dhT=one, softplus=False)[8]
    off = drift(dh0, delta, A, o)
    assert abs(off) <= tolerance(o), f"{off:.2e} over 2^{-o} tokens (tolerance {tolerance(o):.2e})"
