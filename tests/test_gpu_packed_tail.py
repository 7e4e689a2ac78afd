"""Packed sequences that end before the last row of their tensors (a batch padded to a fixed
length): rows behind the last sequence are not read, and new memory holds zeros there, in
outputs and in gradients.  All new memory of these tests holds NaN, and so do the inputs'
rows behind the last sequence: what nothing writes, or what reads them, shows."""
import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


@pytest.fixture(autouse=True)
def new_memory_is_nan():
    torch.use_deterministic_algorithms(True, warn_only=True)
    assert torch.utils.deterministic.fill_uninitialized_memory
    yield
    torch.use_deterministic_algorithms(False)


def offsets(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def behind(t, last):
    """A copy with NaN in the rows that no sequence has, and one that ends with the last."""
    padded = t.clone()
    padded[:, last:] = NAN
    return padded, t[:, :last].contiguous()


def zero_behind(t, last, name):
    assert t[:, last:].numel() == 0 or not (t[:, last:] != 0).any(), name   # (NaN != 0)
    assert torch.isfinite(t[:, :last].float()).all(), name


# sequences that end at once, inside and at the end of a run of tokens, and in the last row
ENDS = [[0, 0, 0], [0, 20, 61], [0, 64, 64, 128], [0, 5, 299], [0, 300]]


@pytest.mark.parametrize("cu", ENDS)
@pytest.mark.parametrize("dt,D,W", [(BF, 64, 4), (F32, 36, 3), (BF, 5, 2), (F32, 1, 4)])
def test_conv(ck, dt, D, W, cu):
    gen = torch.Generator().manual_seed(D)
    T, last, off = 300, cu[-1], offsets(cu)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, xs = behind(r(1, T, D).to(dt).cuda(), last)
    dy, dys = behind(r(1, T, D).to(dt).cuda(), last)
    w, b = r(D, W).cuda(), r(D).cuda()
    h0, dhT = (r(len(cu) - 1, W - 1, D).to(dt).cuda() for _ in range(2))
    y, hT = ck.conv_fwd(x, w, b, h0=h0, cu_seqlens=off)
    grads = ck.conv_bwd(dy, x, w, b, h0=h0, dhT=dhT, cu_seqlens=off)
    zero_behind(y, last, "y")
    zero_behind(grads[0], last, "dx")
    wy, wh, want, size = ref.conv(xs, w, b, h0, cu, True, dys, dhT)
    ref.check(y[:, :last], wy, ref.conv_tol(dt, W), "y")
    assert torch.equal(hT.cpu().double(), wh)
    ref.check(grads[0][:, :last], want["dx"], ref.conv_tol(dt, W), "dx", size=size["dx"])
    sums = ref.conv_tol(F32, W) + 2 * T ** 0.5 * ref.U[F32]
    for g, n in zip(grads[1:], ("dw", "db", "dh0")):
        ref.check(g, want[n], sums if n != "dh0" else ref.conv_tol(dt, W), n, size=size[n])


def test_conv_given_memory_is_left(ck):
    x, w = torch.randn(1, 90, 64, device="cuda").to(BF), torch.randn(64, 4, device="cuda")
    y = torch.full((1, 90, 64), 7.0, dtype=BF, device="cuda")
    got, _ = ck.conv_fwd(x, w, cu_seqlens=offsets([0, 20, 61]), y=y)
    assert got is y and (y[:, 61:] == 7).all()
    assert torch.equal(y[:, :61], ck.conv_fwd(x, w, cu_seqlens=offsets([0, 20, 61]))[0][:, :61])


def test_conv_under_a_projection(ck):
    """The weight before it has the gradient of the batch without padding."""
    T, last, D, off = 200, 150, 48, offsets([0, 60, 150])
    u, us = behind(torch.randn(1, T, D, device="cuda"), last)
    u[:, last:] = 1.0   # (rows of padding are finite where a user's loss masks them)
    cw, dy = torch.randn(D, 4, device="cuda"), torch.randn(1, T, D, device="cuda")

    def grad(u, dy):
        s = torch.ones(D, device="cuda", requires_grad=True)
        y, _ = ck.short_conv(u * s, cw, cu_seqlens=off)
        y.backward(dy)
        return s.grad
    dy[:, last:] = 0
    ref.check(grad(u, dy), ref.d(grad(us, dy[:, :last].contiguous())), 2 * last ** 0.5 * ref.U[F32],
              "weight")


@pytest.mark.parametrize("cu", ENDS)
@pytest.mark.parametrize("dt,D,N,G", [(BF, 32, 16, 1), (F32, 24, 12, 2), (BF, 5, 3, 1), (F32, 136, 4, 1), (BF, 16, 64, 1)])
@pytest.mark.parametrize("more", [0, 1000])
def test_scan(ck, dt, D, N, G, cu, more):
    """more: whole pieces of the row lie behind the last sequence."""
    gen = torch.Generator().manual_seed(D)
    T, last, off, n = 300 + more, cu[-1], offsets(cu), len(cu) - 1
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    rows = {k: behind(r(1, T, *s).to(dt).cuda(), last)
            for k, s in (("x", (D,)), ("dt", (D,)), ("B", (G, N)), ("C", (G, N)), ("z", (D,)), ("dy", (D,)))}
    A, skip, bias = -torch.exp(0.8 * r(D, N)).cuda(), r(D).cuda(), r(D).cuda() - 2
    h0, dhT = r(n, D, N).cuda(), r(n, D, N).cuda()

    def call(i):
        x, step, B, C, z, dy = (rows[k][i] for k in ("x", "dt", "B", "C", "z", "dy"))
        return x, step, A, B, C, skip, z, bias, h0, dy
    x, step, _, B, C, _, z, _, _, dy = call(0)
    y, hT = ck.scan_fwd(x, step, A, B, C, D=skip, z=z, dt_bias=bias, h0=h0, cu_seqlens=off)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")
    grads = dict(zip(names, ck.scan_bwd(dy, x, step, A, B, C, D=skip, z=z, dt_bias=bias, h0=h0, dhT=dhT, cu_seqlens=off)))
    zero_behind(y, last, "y")
    for k in ("dx", "ddt", "dB", "dC", "dz"):
        zero_behind(grads[k], last, k)
    x, step, _, B, C, _, z, _, _, dy = call(1)
    wy, wh, want, size = ref.scan(x, step, A, B, C, skip, z, bias, h0, cu, True, dy, dhT)
    ref.check(y[:, :last], wy, ref.scan_tol(dt, T), "y")
    ref.check(hT, wh, ref.scan_tol(F32, T), "hT")
    for k, g in grads.items():
        w = want[k]
        if k in ("dx", "ddt", "dz"):
            tol, g = ref.scan_tol(dt, T, True), g[:, :last]
        elif k in ("dB", "dC"):
            tol, g = ref.sum_tol(dt, T, D), g[:, :last]
        else:
            tol = ref.scan_tol(F32, T, True) if k == "dh0" else ref.sum_tol(F32, T, T)
        ref.check(g, w, tol, k, size=size[k])


def test_scan_given_memory_is_left(ck):
    x, A, B = torch.randn(1, 90, 32, device="cuda"), -torch.rand(32, 4, device="cuda"), torch.randn(1, 90, 4, device="cuda")
    y = torch.full((1, 90, 32), 7.0, device="cuda")
    off = offsets([0, 20, 61])
    got, _ = ck.scan_fwd(x, x, A, B, B, cu_seqlens=off, y=y)
    assert got is y and (y[:, 61:] == 7).all()
    assert torch.equal(y[:, :61], ck.scan_fwd(x, x, A, B, B, cu_seqlens=off)[0][:, :61])


def test_scan_between_projections(ck):
    """Weights before and behind the scan have finite gradients, the padding's masked."""
    T, last, D, off = 400, 290, 32, offsets([0, 100, 290])
    s = [torch.ones(D, device="cuda", requires_grad=True) for _ in range(2)]
    u, A, B = torch.randn(1, T, D, device="cuda"), -torch.rand(D, 16, device="cuda"), torch.randn(1, T, 16, device="cuda")
    mask = (torch.arange(T, device="cuda") < last)[None, :, None].float()

    def loss(T, mask):
        x = u[:, :T] * s[0]
        y, _ = ck.selective_scan(x, (x - 2), A, B[:, :T], B[:, :T], cu_seqlens=off)
        return (y * s[1] * mask).square().sum()
    padded = torch.autograd.grad(loss(T, mask), s)
    for a, b in zip(padded, torch.autograd.grad(loss(last, 1.0), s)):
        ref.check(a, ref.d(b), 2 * ref.sum_tol(F32, last, last), "weight")


def test_conv_captured(ck):
    x, w = torch.randn(1, 300, 64, device="cuda").to(BF), torch.randn(64, 4, device="cuda")
    captured(lambda off: (ck.conv_fwd(x, w, cu_seqlens=off)[0], ck.conv_bwd(x, x, w, cu_seqlens=off)[0]))


def test_scan_captured(ck):
    x, A, B = torch.randn(1, 300, 64, device="cuda"), -torch.rand(64, 16, device="cuda"), torch.randn(1, 300, 16, device="cuda")

    def run(off):
        g = ck.scan_bwd(x, x, x, A, B, B, cu_seqlens=off)
        return (ck.scan_fwd(x, x, A, B, B, cu_seqlens=off)[0], g[0], g[1], g[3], g[4])
    captured(run)


def captured(call):
    off = offsets([0, 30, 200])
    run = lambda: call(off)  # noqa: E731
    run()
    torch.use_deterministic_algorithms(False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for cu in ([0, 30, 200], [0, 100, 130], [0, 7, 300]):   # the batch's end moves between replays
        off.copy_(offsets(cu))
        for t in got:
            t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, run()):
            zero_behind(a, cu[-1], str(cu))
            assert torch.equal(a, b)
