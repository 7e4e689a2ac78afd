"""Which rows of the selective scan are cut into pieces, by the workspaces that the calls ask
for: a larger batch is never the one that stays whole while a smaller one of about its time is
cut (a cut forward row computes every decay twice)."""
import pytest


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_ckda_gb300 import build
    build.build()
    import gated_delta_rule_ckda_gb300 as ck
    return ck.lib()


def whole_bwd(L, B, T, D, N):
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    one = (up(B * ((T + 3) // 4) * D * N * 4) + up((D + 31) // 32 * B * T * 2 * N * 4) + up(B * D * N * 4)
           + up(B * 2 * D * 4))
    return L.ckda_scan_bwd_workspace_bytes(B, T, D, N, 1) == one


@pytest.mark.parametrize("N", [4, 16, 64])
@pytest.mark.parametrize("D,rows", [(4096, (3, 4)), (2048, (7, 8)), (4095, (3, 4)), (512, (28, 29))])
def test_forward(L, D, rows, N):
    """Whole where 1824 warps hold fewer than four pieces of the batch."""
    size = lambda B: L.ckda_scan_fwd_workspace_bytes(B, 2048, D, N, 1)  # noqa: E731
    assert all(size(B) > 0 for B in range(1, rows[0] + 1))
    assert not any(size(B) for B in range(rows[1], 40))


@pytest.mark.parametrize("N,rows", [(4, (7, 8)), (16, (7, 8)), (32, (7, 8)), (33, (2, 3)), (64, (2, 3))])
def test_backward(L, N, rows):
    """Whole where 3648 warps hold fewer than four pieces, of more than 32 states fewer than
    twelve."""
    assert not any(whole_bwd(L, B, 1024, 4096, N) for B in range(1, rows[0] + 1))
    assert all(whole_bwd(L, B, 1024, 4096, N) for B in range(rows[1], 20))


def test_short_rows_stay_whole(L):
    assert L.ckda_scan_fwd_workspace_bytes(1, 128, 64, 16, 1) == 0
    assert L.ckda_scan_fwd_workspace_bytes(1, 129, 64, 16, 1) > 0
    assert whole_bwd(L, 1, 32, 64, 16) and not whole_bwd(L, 1, 33, 64, 16)
    assert whole_bwd(L, 1, 64, 64, 64) and not whole_bwd(L, 1, 65, 64, 64)
