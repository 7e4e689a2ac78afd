"""RMS norm of fp32 rows between the widest that a block holds in vectors (8192 columns) and
the widest that it holds at all (16,384), on both sides of each, more of them than blocks."""
import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
F32 = torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def make(rows, width):
    gen = torch.Generator(device="cuda").manual_seed(width)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return dict(x=r(rows, width), res=r(rows, width), w=1 + 0.2 * r(width), dy=r(rows, width), dh=r(rows, width))


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("width", [8192, 8196, 12288, 16380, 16384, 16388])
def test_rows(ck, width, residual):
    s = make(400, width)
    res = s["res"] if residual else None
    y, h, rstd = ck.rmsnorm_fwd(s["x"], s["w"], residual=res, eps=EPS)
    assert torch.equal(h, s["x"] + s["res"] if residual else s["x"])
    wy, wr = ref.rms(h, s["w"], EPS)
    ref.check(y, wy, ref.rms_tol(F32, width), "y")
    ref.check(rstd, wr, ref.rms_tol(F32, width), "rstd")
    dh = s["dh"] if residual else None
    dx, dw = ck.rmsnorm_bwd(s["dy"], h, rstd, s["w"], dh=dh)
    rx, rw, size = ref.rms_bwd(s["dy"], h, rstd, s["w"], dh)
    ref.check(dx, rx, ref.rms_tol(F32, width), "dx", size=size)
    ref.check(dw, rw, (8 + 2 * 400 ** 0.5) * ref.U[F32], "dw",
              size=float((ref.d(s["dy"]) * ref.d(h) * wr[:, None]).square().sum(0).mean().sqrt()))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("width", [8192, 8320, 16256, 16384, 16512])
def test_eight_bits(ck, width, group):
    """Values within half a step of e4m3, or of its even steps, of y over its scale."""
    s = make(170, width)
    y8, scale, h, _ = ck.rmsnorm_fwd8(s["x"], s["w"], residual=s["res"], eps=EPS, group=group)
    assert torch.equal(h, s["x"] + s["res"])
    want = ref.rms(h, s["w"], EPS)[0].view(170, -1, group or width)
    top = want.abs().amax(-1) / 448
    u = (12 + 2 * width ** 0.5) * ref.U[F32]   # of y; three more for the scale and the quotient
    assert ((ref.d(scale).view(top.shape) - top).abs() <= 4 * u * top).all()
    units = want / top[..., None]
    off = (ref.d(y8).view(units.shape) - units).abs()
    assert (off <= torch.clamp(units.abs() * 2.0 ** -4, min=2.0 ** -10) + 448 * 4 * u).all()


@pytest.mark.parametrize("width", [8196, 16384])
def test_in_place(ck, width):
    s = make(333, width)
    want = ck.rmsnorm_fwd(s["x"], s["w"], residual=s["res"])
    x, res = s["x"].clone(), s["res"].clone()
    y, h, _ = ck.rmsnorm_fwd(x, s["w"], residual=res, y=x, h=res)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    grad = ck.rmsnorm_bwd(s["dy"], want[1], want[2], s["w"], dh=s["dh"])
    for name in ("dy", "dh", "h"):
        t = {"dy": s["dy"].clone(), "dh": s["dh"].clone(), "h": want[1].clone()}
        dx, dw = ck.rmsnorm_bwd(t["dy"], t["h"], want[2], s["w"], dh=t["dh"], dx=t[name])
        assert torch.equal(dx, grad[0]) and torch.equal(dw, grad[1])
