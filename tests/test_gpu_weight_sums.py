"""Gradients of weights: sums over the blocks' parts carry what their additions round off.
One token's term is so large that a part of all other tokens of a block is below half a
step of it, and would be lost one block after another; together they are many steps."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def near(got, want, step):
    """Two roundings to a step, of what the blocks' sums leave and of the whole, and what the
    large term's own block loses beside it: half a step each, and one for the last."""
    assert ((got.double() - want).abs() <= 2 * step).all(), float((got.double() - want).abs().max() / step)


def test_conv(ck):
    """163,840 tokens in blocks of 512: 2^35 and ones, in steps of 4096."""
    T, D = 64 * 8 * 320, 128
    x = torch.ones(1, T, D, device="cuda")
    dy = torch.ones_like(x)
    dy[0, 5] = 2.0 ** 35
    dy[0, 6:64] = 0    # (the large term's own run)
    w, b = torch.zeros(D, 2, device="cuda"), torch.zeros(D, device="cuda")
    _, dw, db, _ = ck.conv_bwd(dy, x, w, b, silu=False)
    want = 2.0 ** 35 + T - 59
    near(db, torch.full_like(db, want).double(), 4096)
    near(dw[:, 1], torch.full_like(db, want).double(), 4096)
    near(dw[:, 0], torch.full_like(db, want).double(), 4096)


@pytest.mark.parametrize("D", [4096, 512, 301])
def test_norm(ck, D):
    """16,384 rows: 2^34 and ones, in steps of 2048."""
    rows = 16384
    h, rstd = torch.ones(rows, D, device="cuda"), torch.ones(rows, device="cuda")
    dy = torch.ones_like(h)
    dy[0] = 2.0 ** 34
    _, dw = ck.rmsnorm_bwd(dy, h, rstd, torch.ones(D, device="cuda"))
    near(dw, torch.full_like(dw, 2.0 ** 34 + rows - 1).double(), 2048)


@pytest.mark.parametrize("T,D", [(32000, 32), (32000, 31)])
def test_scan(ck, T, D):
    """1000 pieces of 32 tokens: 2^30 and ones, in steps of 128."""
    x, A = torch.ones(1, T, D, device="cuda"), -torch.ones(D, 4, device="cuda")
    B = torch.zeros(1, T, 4, device="cuda")
    dy = torch.ones_like(x)
    dy[0, 3] = 2.0 ** 30
    g = ck.scan_bwd(dy, x, -x, A, B, B, D=torch.ones(D, device="cuda"))
    near(g[5], torch.full_like(g[5], 2.0 ** 30 + T - 1).double(), 128)


def test_terms_that_are_not_finite(ck):
    """An infinite term makes an infinite sum, as in the plain form, and no NaN."""
    rows, D = 3000, 96
    h, rstd = torch.ones(rows, D, device="cuda"), torch.ones(rows, device="cuda")
    dy = torch.ones_like(h)
    dy[7, 5], dy[9, 6] = float("inf"), float("-inf")
    dy[11, 8] = float("nan")
    dy[13, 9] = dy[2700, 9] = 3e38
    dw = ck.rmsnorm_bwd(dy, h, rstd, torch.ones(D, device="cuda"))[1]
    assert dw[5] == float("inf") and dw[6] == float("-inf") and torch.isnan(dw[8])
    assert dw[9] == float("inf")   # (past fp32)
    keep = [i for i in range(D) if i not in (5, 6, 8, 9)]
    assert (dw[keep] == rows).all()
    T = 3000
    x, A, B = torch.ones(1, T, 32, device="cuda"), -torch.ones(32, 4, device="cuda"), torch.zeros(1, T, 4, device="cuda")
    dy = torch.ones_like(x)
    dy[0, 70, 5] = float("inf")
    dD = ck.scan_bwd(dy, x, -x, A, B, B, D=torch.ones(32, device="cuda"))[5]
    assert dD[5] == float("inf") and (dD[[i for i in range(32) if i != 5]] == T).all()
