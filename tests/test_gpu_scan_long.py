"""Selective scan where a row of more tokens than one piece's sums take at once stays whole:
the decays of a row one behind the other, and dA's sums over more than 512 tokens.  Whole
rows need a batch that fills the card, so a few rows and channels are repeated: outputs
repeat, dB and dC (sums over channels) and dA, dD, ddt_bias (over rows) are multiples."""
import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def whole_rows(ck, rows, T, D, N):
    """That neither pass cuts the rows, by their workspaces: the backward's of one piece."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    blocks = (D + 31) // 32
    one = (up(rows * ((T + 3) // 4) * D * N * 4) + up(blocks * rows * T * 2 * N * 4) + up(rows * D * N * 4)
           + up(rows * 2 * D * 4))
    L = ck.lib()
    return L.ckda_scan_fwd_workspace_bytes(rows, T, D, N, 1) == 0 and L.ckda_scan_bwd_workspace_bytes(rows, T, D, N, 1) == one


ROWS, CHANS = 29, 32   # times two rows and 32 (or 31) channels of their own


@pytest.mark.parametrize("T,N,dt,chans", [
    (512, 16, F32, 32), (513, 16, F32, 32), (520, 16, BF, 32), (1030, 16, F32, 32), (1030, 16, BF, 32), (1030, 20, F32, 32),
    (1030, 5, F32, 31), (1030, 15, BF, 31), (600, 40, BF, 32)])
def test_whole_rows(ck, T, N, dt, chans):
    """Both sides of the 512 tokens behind which dA's sums go to memory, and twice that; states
    of one slice and of more; whole vectors and single elements."""
    gen = torch.Generator().manual_seed(T + N)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n, times = 2, 33 if chans == 31 else CHANS
    D, rows = chans * times, n * ROWS
    assert whole_rows(ck, rows, T, D, N)
    small = dict(x=r(n, T, chans).to(dt), dt=r(n, T, chans).to(dt), z=r(n, T, chans).to(dt), dy=r(n, T, chans).to(dt),
                 B=r(n, T, N).to(dt), C=r(n, T, N).to(dt), A=-torch.exp(0.8 * r(chans, N)), D=r(chans), bias=r(chans) - 3,
                 h0=r(n, chans, N), dhT=r(n, chans, N))
    y, hT, want, size = ref.scan(*(small[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0")), None, True,
                                 small["dy"], small["dhT"])
    c = {}
    for k, v in small.items():
        v = v.cuda()
        axis = {"x": 2, "dt": 2, "z": 2, "dy": 2, "A": 0, "D": 0, "bias": 0, "h0": 1, "dhT": 1}.get(k)
        if axis is not None:
            v = torch.cat([v] * times, axis)
        c[k] = v if k in ("A", "D", "bias") else torch.cat([v] * ROWS, 0)
    more = dict(D=c["D"], z=c["z"], dt_bias=c["bias"], h0=c["h0"])
    got_y, got_h = ck.scan_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], **more)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
    grads = dict(zip(names, ck.scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], dhT=c["dhT"], **more)))

    def rows_of(t):   # the rows that are no repetition; the repetitions have their bits
        assert all(torch.equal(t[i * n:i * n + n], t[:n]) for i in range(ROWS))
        return t[:n]

    def check(t, axis, tol, k, want, size=0.0):
        # every repetition of 32 channels has the first one's bits; 31 lie otherwise in a warp
        parts = t.split(chans, axis)
        if chans == 32:
            assert all(torch.equal(p, parts[0]) for p in parts)
        for p in (parts[0], parts[-1]):
            ref.check(p, want, tol, k, size=size)
    check(rows_of(got_y), 2, ref.scan_tol(dt, T), "y", y)
    check(rows_of(got_h), 1, ref.scan_tol(F32, T), "hT", hT)
    for k in ("dx", "ddt", "dz"):
        check(rows_of(grads[k]), 2, ref.scan_tol(dt, T, True), k, want[k], size[k])
    check(rows_of(grads["dh0"]), 1, ref.scan_tol(F32, T, True), "dh0", want["dh0"], size["dh0"])
    # sums of `times` (ROWS) equal parts: each part's errors, and those of adding them up
    for k in ("dB", "dC"):
        ref.check(rows_of(grads[k]).double() / times, want[k], ref.sum_tol(dt, T, D), k, size=size[k])
    for k in ("dA", "dD", "ddt_bias"):
        check(grads[k].double() / ROWS, 0, ref.sum_tol(F32, T, rows * T), k, want[k], size[k])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("cuts", [[0, 300, 600, 900], [0, 1, 17, 640, 900]])
def test_parts_of_a_row(ck, dt, cuts):
    """Less workspace: a row's parts forward, each from the state of the one before, then their
    gradients from the last part to the first, dh0 handed on as dhT."""
    gen = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n, T, D, N = 2, 900, 40, 16
    s = dict(x=r(n, T, D).to(dt), dt=r(n, T, D).to(dt), B=r(n, T, N).to(dt), C=r(n, T, N).to(dt), z=r(n, T, D).to(dt),
             dy=r(n, T, D).to(dt))
    A, skip, bias, h0, dhT = -torch.exp(0.8 * r(D, N)), r(D), r(D) - 3, r(n, D, N), r(n, D, N)
    y, hT, want, size = ref.scan(s["x"], s["dt"], A, s["B"], s["C"], skip, s["z"], bias, h0, None, True, s["dy"], dhT)
    c = {k: v.cuda() for k, v in s.items()}
    A, skip, bias = A.cuda(), skip.cuda(), bias.cuda()
    # (a batch's rows of a part are not evenly apart: copied)
    parts = [{k: v[:, a:b].contiguous() for k, v in c.items()} for a, b in zip(cuts, cuts[1:])]
    state, states, ys = h0.cuda(), [], []
    for p in parts:
        states.append(state)
        out, state = ck.scan_fwd(p["x"], p["dt"], A, p["B"], p["C"], skip, p["z"], bias, state)
        ys.append(out)
    ref.check(torch.cat(ys, 1), y, ref.scan_tol(dt, T), "y")
    ref.check(state, hT, ref.scan_tol(F32, T), "hT")
    passed, by_token, sums = dhT.cuda(), [], 0
    for p, h in zip(reversed(parts), reversed(states)):
        dx, ddt, dA, dB, dC, dD, dz, dbias, passed = ck.scan_bwd(p["dy"], p["x"], p["dt"], A, p["B"], p["C"], skip, p["z"], bias, h,
                                                                 passed)
        by_token.insert(0, (dx, ddt, dz, dB, dC))
        sums = [a + b for a, b in zip(sums, (dA, dD, dbias))] if sums else [dA, dD, dbias]
    for i, k in enumerate(("dx", "ddt", "dz", "dB", "dC")):
        tol = ref.scan_tol(dt, T, True) if i < 3 else ref.sum_tol(dt, T, D)
        ref.check(torch.cat([p[i] for p in by_token], 1), want[k], tol, k, size=size[k])
    for g, k in zip(sums, ("dA", "dD", "ddt_bias")):
        ref.check(g, want[k], ref.sum_tol(F32, T, n * T), k, size=size[k])
    ref.check(passed, want["dh0"], ref.scan_tol(F32, T, True), "dh0", size=size["dh0"])
