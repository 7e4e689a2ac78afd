"""RMS norm with the residual's addition, in the I/O type and in 8 bits, forward and
backward, against its 64-bit reference."""
import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-5


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def make(rows, width, dt, wdt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=r(rows, width).to(dt), res=(r(rows, width) * (0.3 + r(rows, 1).abs())).to(dt),
                w=(1 + 0.2 * r(width)).to(wdt), dy=r(rows, width).to(dt), dh=r(rows, width).to(dt))


def compare(ck, s, residual=True, weight=True):
    c = {k: v.cuda() for k, v in s.items()}
    (rows, width), dt = s["x"].shape, s["x"].dtype
    w = c["w"] if weight else None
    cw = s["w"] if weight else None
    y, h, rstd = ck.rmsnorm_fwd(c["x"], w, residual=c["res"] if residual else None, eps=EPS)
    assert torch.equal(h.cpu(), (s["x"].float() + s["res"].float()).to(dt) if residual else s["x"])
    wy, wr = ref.rms(h, cw, EPS)
    ref.check(y, wy, ref.rms_tol(dt, width), "y")
    ref.check(rstd, wr, ref.rms_tol(F32, width), "rstd")
    dh = c["dh"] if residual else None
    dx, dw = ck.rmsnorm_bwd(c["dy"], h, rstd, w, dh=dh)
    rx, rw, size = ref.rms_bwd(s["dy"], h, rstd, cw, dh)
    ref.check(dx, rx, ref.rms_tol(dt, width), "dx", size=size)
    wdt = s["w"].dtype if weight else F32
    assert dw.dtype == wdt
    sums = (ref.rounding(BF) if wdt == BF else 0.0) + (8 + 2 * rows ** 0.5) * ref.U[F32]
    ref.check(dw, rw, sums, "dw", size=float((ref.d(s["dy"]) * ref.d(h) * wr[:, None]).square().sum(0).mean().sqrt()))
    return h


def compare8(ck, s, group, residual=True):
    """The scale to fp32's roundings; each value within half a step of e4m3 (2^-4 of it, or
    2^-10 in units of the scale where the steps are even) of y / scale."""
    c = {k: v.cuda() for k, v in s.items()}
    rows, width = s["x"].shape
    y8, scale, h, rstd = ck.rmsnorm_fwd8(c["x"], c["w"], residual=c["res"] if residual else None, eps=EPS, group=group)
    assert y8.dtype == E4M3 and scale.shape == ((rows, width // group) if group else (rows,))
    y, hh, rs = ck.rmsnorm_fwd(c["x"], c["w"], residual=c["res"] if residual else None, eps=EPS)
    assert torch.equal(h, hh)
    wy, _ = ref.rms(h, s["w"], EPS)
    g = wy.view(rows, -1, group or width)
    want = g.abs().amax(-1).clamp(min=2.0 ** -100) / 448
    u = (12 + 2 * width ** 0.5) * ref.U[F32]   # of y; three more for the scale and the quotient
    assert ((ref.d(scale).view(want.shape) - want).abs() <= 4 * u * want).all()
    units = g / want[..., None]
    off = (ref.d(y8).view(g.shape) - units).abs()
    assert (off <= torch.clamp(units.abs() * 2.0 ** -4, min=2.0 ** -10) + 448 * 4 * u).all(), float(off.max())
    assert float(ref.d(y8).abs().max()) <= 448
    assert torch.allclose(rstd, rs, rtol=2 * u, atol=0)


# both sides of each variant's border: lanes a row, vectors a lane, a block a row, beyond
WIDTHS = [1, 2, 7, 8, 32, 63, 64, 65, 127, 128, 129, 256, 257, 264, 512, 520, 1000, 1024, 1031, 1040, 2047, 2048,
          2056, 4096, 5000, 8192, 8200]


@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(ck, dt, wdt, width):
    compare(ck, make(37, width, dt, wdt, width))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("width", [16384, 16392, 20000, 40001])
def test_wide_rows(ck, dt, width):
    compare(ck, make(5, width, dt, F32, 1))
    compare(ck, make(5, width, dt, F32, 1), residual=False)
    compare8(ck, make(5, width, dt, F32, 1), 0)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 33, 1217, 20000])
@pytest.mark.parametrize("width", [40, 128, 1024])
def test_rows(ck, rows, width):
    compare(ck, make(rows, width, BF, F32, rows))


@pytest.mark.parametrize("residual,weight", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("dt,width", [(BF, 300), (BF, 512), (F32, 96), (F32, 4000)])
def test_without_parts(ck, dt, width, residual, weight):
    compare(ck, make(50, width, dt, F32, 5), residual, weight)


@pytest.mark.parametrize("dt,width", [(BF, 768), (BF, 1536), (BF, 2560), (BF, 5120), (BF, 12288), (BF, 16384),
                                      (F32, 900), (F32, 5120), (F32, 8192)])
def test_more_rows_than_blocks(ck, dt, width):
    compare(ck, make(2500 if width < 5000 else 700, width, dt, F32, width))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("width", [128, 256, 640, 1024, 2048, 4096, 8192, 16384])
def test_eight_bits(ck, width, group, dt):
    compare8(ck, make(21, width, dt, F32, width + group), group)


@pytest.mark.parametrize("width,group", [(32, 32), (64, 32), (96, 32), (64, 64), (192, 64), (24576, 128), (24576, 64),
                                         (33, 0), (7, 0), (1, 0), (1031, 0), (5000, 0)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_eight_bits_odd(ck, width, group, dt):
    compare8(ck, make(9, width, dt, BF, width), group, residual=width % 2 == 0)


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("dt", [BF, F32])
def test_eight_bits_unaligned(ck, dt, group):
    s = make(13, 384, dt, F32, 2)
    c = {k: v.cuda() for k, v in s.items()}
    want = ck.rmsnorm_fwd8(c["x"], c["w"], eps=EPS, group=group)
    buf = torch.empty(13 * 384 + 1, dtype=dt, device="cuda")
    x = buf[1:].view(13, 384)
    x.copy_(c["x"])
    got = ck.rmsnorm_fwd8(x, c["w"], eps=EPS, group=group)
    # the row's sum in another order: a step of e4m3 at most, for few values
    assert torch.allclose(got[1], want[1], rtol=1e-5)
    a, b = got[0].float(), want[0].float()
    assert ((a - b).abs() <= torch.clamp(b.abs() * 0.126, min=2.0 ** -9)).all() and (a != b).float().mean() < 1e-2


def test_rows_of_zeros_and_tiny_values(ck):
    x = torch.zeros(4, 256, device="cuda")
    x[1] = 1e-30
    x[2, 7] = 3.0
    for group in (0, 32, 128):
        y8, scale, _, _ = ck.rmsnorm_fwd8(x, eps=1e-5, group=group)
        s = scale.view(4, -1).repeat_interleave(256 // max(1, scale.view(4, -1).shape[1]), 1)
        assert torch.isfinite(scale).all() and (scale > 0).all()
        assert not y8[0].float().any() and not y8[3].float().any()
        back = y8.float() * s
        want = ck.rmsnorm_fwd(x, eps=1e-5)[0]
        # of the largest value in the row or its group a half step, 2^-4
        assert torch.allclose(back[2, 7], want[2, 7], rtol=2 ** -4) and torch.allclose(back[1], want[1], rtol=2 ** -4)


def test_values_that_are_not_finite_stay_in_their_row(ck):
    s = make(40, 128, BF, F32, 9)
    c = {k: v.cuda() for k, v in s.items()}
    run = lambda: (ck.rmsnorm_fwd(c["x"], c["w"], residual=c["res"])[0],  # noqa: E731
                   ck.rmsnorm_fwd8(c["x"], c["w"], residual=c["res"], group=32)[0].float())
    clean = run()
    c["x"][3, 5], c["x"][8, 0] = float("inf"), float("nan")
    dirty = run()
    keep = [i for i in range(40) if i not in (3, 8)]
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep]) and torch.isnan(b[[3, 8]].float()).any(-1).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_misaligned_in_place_and_leading_axes(ck, dt):
    s = make(24, 96, dt, F32, 11)
    c = {k: v.cuda() for k, v in s.items()}
    lead = lambda t: t.view(2, 3, 4, 96)  # noqa: E731
    want = ck.rmsnorm_fwd(lead(c["x"]), c["w"], residual=lead(c["res"]), eps=EPS)
    assert want[2].shape == (2, 3, 4)
    buf = torch.empty(24 * 96 + 1, dtype=dt, device="cuda")
    m = buf[1:].view(2, 3, 4, 96)
    m.copy_(lead(c["x"]))
    got = ck.rmsnorm_fwd(m, c["w"], residual=lead(c["res"]), eps=EPS)
    ref.check(got[0], ref.d(want[0]), 2 * ref.rms_tol(dt, 96), "misaligned")
    assert torch.equal(got[1], want[1])
    # the sum in place of the residual, the output in place of x
    x, res = lead(c["x"]).clone(), lead(c["res"]).clone()
    y, h, _ = ck.rmsnorm_fwd(x, c["w"], residual=res, eps=EPS, y=x, h=res)
    assert y is x and h is res and torch.equal(y, want[0]) and torch.equal(h, want[1])
    x, res = lead(c["x"]).clone(), lead(c["res"]).clone()
    y, h, _ = ck.rmsnorm_fwd(x, c["w"], residual=res, eps=EPS, h=x)
    assert h is x and torch.equal(y, want[0]) and torch.equal(h, want[1])
    grad = ck.rmsnorm_bwd(lead(c["dy"]), want[1], want[2], c["w"], dh=lead(c["dh"]))
    for name in ("dy", "dh"):
        t = {k: lead(c[k]).clone() for k in ("dy", "dh")}
        dx, dw = ck.rmsnorm_bwd(t["dy"], want[1], want[2], c["w"], dh=t["dh"], dx=t[name])
        assert dx is t[name] and torch.equal(dx, grad[0]) and torch.equal(dw, grad[1])


@pytest.mark.parametrize("width", [20000, 40001])
def test_wide_rows_in_place(ck, width):
    s = make(4, width, BF, F32, 3)
    c = {k: v.cuda() for k, v in s.items()}
    want = ck.rmsnorm_fwd(c["x"], c["w"], residual=c["res"])
    x, res = c["x"].clone(), c["res"].clone()
    y, h, _ = ck.rmsnorm_fwd(x, c["w"], residual=res, y=x, h=res)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,width", [(3001, 127), (1501, 301), (701, 1031), (333, 4853)])
def test_odd_rows_in_place(ck, dt, rows, width):
    """Rows that share 16-byte vectors with their neighbours, in place, and what lies behind
    the last one."""
    s = make(rows, width, dt, F32, 5)
    c = {k: v.cuda() for k, v in s.items()}
    n = rows * width

    def framed(t):
        buf = torch.full((n + 64,), 7.0, dtype=dt, device="cuda")
        buf[:n] = t.flatten()
        return buf, buf[:n].view(rows, width)

    want = ck.rmsnorm_fwd(c["x"], c["w"], residual=c["res"])
    (bx, x), (br, res) = framed(c["x"]), framed(c["res"])
    y, h, rstd = ck.rmsnorm_fwd(x, c["w"], residual=res, y=x, h=res)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1]) and torch.equal(rstd, want[2])
    assert (bx[n:] == 7).all() and (br[n:] == 7).all()
    grad = ck.rmsnorm_bwd(c["dy"], want[1], want[2], c["w"], dh=c["dh"])
    for name in ("dy", "dh", "h"):
        t = {"dy": c["dy"], "dh": c["dh"], "h": want[1]}
        buf, t[name] = framed(t[name])
        dx, dw = ck.rmsnorm_bwd(t["dy"], t["h"], want[2], c["w"], dh=t["dh"], dx=t[name])
        assert torch.equal(dx, grad[0]) and torch.equal(dw, grad[1]) and (buf[n:] == 7).all()


def test_no_rows(ck):
    x = torch.empty(0, 64, device="cuda")
    y, h, rstd = ck.rmsnorm_fwd(x)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    assert ck.rmsnorm_fwd8(x, group=32)[1].shape == (0, 2)
    _, dw = ck.rmsnorm_bwd(x, x, rstd, torch.ones(64, device="cuda"))
    assert not dw.any()


def test_autograd_and_graph(ck):
    s = make(300, 256, BF, F32, 13)
    c = {k: v.cuda() for k, v in s.items()}
    leaves = [c[k].clone().requires_grad_() for k in ("x", "w", "res")]
    y, h = ck.rms_norm(*leaves, eps=EPS)
    torch.autograd.backward([y, h], [c["dy"], c["dh"]])
    m = ck.rmsnorm_fwd(c["x"], c["w"], residual=c["res"], eps=EPS)
    dx, dw = ck.rmsnorm_bwd(c["dy"], m[1], m[2], c["w"], dh=c["dh"])
    assert torch.equal(y, m[0]) and torch.equal(h, m[1])
    for t, g in zip(leaves, (dx, dw, dx)):
        assert torch.equal(t.grad, g)
    assert leaves[0].grad.data_ptr() != leaves[2].grad.data_ptr()
    del y, h
    # without a residual, and through the sum alone
    x = c["x"].clone().requires_grad_()
    ck.rms_norm(x, c["w"]).backward(c["dy"])
    z = ck.rmsnorm_fwd(c["x"], c["w"])
    assert torch.equal(x.grad, ck.rmsnorm_bwd(c["dy"], z[1], z[2], c["w"])[0])
    x = c["x"].clone().requires_grad_()
    ck.rms_norm(x, c["w"], c["res"])[1].backward(c["dh"])
    assert torch.equal(x.grad, c["dh"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*ck.rmsnorm_fwd8(c["x"], c["w"], residual=c["res"], group=64),
               *ck.rmsnorm_bwd(c["dy"], m[1], m[2], c["w"], dh=c["dh"]))
    c["dy"].copy_(torch.randn_like(c["dy"]))
    c["x"].copy_(torch.randn_like(c["x"]))
    graph.replay()
    torch.cuda.synchronize()
    again = (*ck.rmsnorm_fwd8(c["x"], c["w"], residual=c["res"], group=64),
             *ck.rmsnorm_bwd(c["dy"], m[1], m[2], c["w"], dh=c["dh"]))
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, again))


def test_differences(ck):
    """The gradient of a sum against differences of the forward, in fp32: a step of 2^-7
    leaves 2^-14 of curvature and 2^-24 / 2^-7 of rounding, on terms near one."""
    s = make(3, 40, F32, F32, 21)
    c = {k: v.cuda() for k, v in s.items()}
    y, h, rstd = ck.rmsnorm_fwd(c["x"], c["w"], eps=EPS)
    dx, _ = ck.rmsnorm_bwd(c["dy"], h, rstd, c["w"])
    loss = lambda x: (ck.rmsnorm_fwd(x, c["w"], eps=EPS)[0].double() * c["dy"].double()).sum(1)  # noqa: E731
    for i in (0, 17, 39):
        e = torch.zeros_like(c["x"])
        e[:, i] = 2.0 ** -7
        diff = (loss(c["x"] + e) - loss(c["x"] - e)) / 2 ** -6
        assert ((diff - dx[:, i].double()).abs() <= 40 ** 0.5 * (2 ** -14 + 4 * 2 ** -17)).all()
