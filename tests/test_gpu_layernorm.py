"""Layer norm, forward and backward, against its 64-bit reference."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def tol(dt, width, cond=1.0):
    """One rounding (rms u / sqrt 3, a quarter on top) after fp32 sums of `width`
    terms; `cond` is how much larger the fp32 terms are than what is left of them."""
    out = 1.25 / 3 ** 0.5 * ref.U[dt] if dt == BF else 0.0
    return out + 1.25 / 3 ** 0.5 * ref.U[F32] * 4 * width ** 0.5 * cond


def weight_tol(wdt, rows):
    return 1.25 / 3 ** 0.5 * ref.U[wdt] * (1 if wdt == BF else 1) + 4 * (rows + 16) ** 0.5 * ref.U[F32]


def make(rows, width, dt, wdt, seed, offset=0.5):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    return ((r(rows, width) + offset * r(rows, 1)).to(dt), (1 + 0.2 * r(width)).to(wdt),
            (0.3 * r(width)).to(wdt), r(rows, width).to(dt))


def compare(ck, x, w, b, dy):
    rows, width = x.numel() // x.shape[-1], x.shape[-1]
    c = lambda t: None if t is None else t.cuda()
    y, mean, rstd = ck.layernorm_fwd(c(x), c(w), c(b), eps=EPS)
    wy, wm, wr = ref.layer_norm(x, w, b, EPS)
    # x - mean loses the digits in which |x| exceeds the row's spread, and the
    # mean those in which |x| exceeds it
    cond = 1 + float((x.double().abs() * wr[:, None]).max())
    ref.check(y, wy, tol(x.dtype, width, cond), "y")
    ref.check(mean, wm, tol(F32, width, 1 + float(x.float().abs().max() / (wm.abs().max() + 1e-30))), "mean")
    ref.check(rstd, wr, tol(F32, width, cond), "rstd")
    dx, dw, db = ck.layernorm_bwd(c(dy), c(x), mean, rstd, c(w))
    rx, rw, rb = ref.layer_norm_bwd(dy, x, mean, rstd, w)
    # dx is a difference of terms of the size of rstd dy weight (for a width of
    # two or so next to nothing is left of them): errors go by the terms' size
    t = wr[:, None] * dy.double() * (1 if w is None else w.double())
    ref.check(dx, rx, tol(x.dtype, width, cond), "dx", size=float(t.square().mean().sqrt()))
    wdt = F32 if w is None else w.dtype
    assert dw.dtype == wdt and db.dtype == wdt
    ref.check(dw, rw, weight_tol(wdt, rows), "dw")
    ref.check(db, rb, weight_tol(wdt, rows), "db")


# both sides of each variant's border: 8, 16, 32 lanes a row, two and four
# vectors a lane, a block a row with one to eight vectors, and beyond
WIDTHS = [2, 7, 8, 32, 63, 64, 65, 127, 128, 129, 256, 257, 264, 512, 520, 1000, 1024, 1031, 1040,
          2047, 2048, 2056, 4096, 5000, 8192, 8200]


@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(ck, dt, wdt, width):
    compare(ck, *make(37, width, dt, wdt, width))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("width", [16384, 16392, 40001])
def test_wide_rows(ck, dt, width):
    compare(ck, *make(5, width, dt, F32, 1))


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 33, 1217, 20000])
@pytest.mark.parametrize("width", [40, 128, 1024])
def test_rows(ck, rows, width):
    compare(ck, *make(rows, width, BF, F32, rows))


def test_single_column(ck):
    """Width 1: the row is its own mean, y is the bias and dx is zero."""
    x, w, b, dy = make(9, 1, F32, F32, 3)
    y, mean, rstd = ck.layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    assert torch.equal(y.cpu(), b.expand(9, 1)) and torch.equal(mean.cpu(), x[:, 0])
    dx, dw, _ = ck.layernorm_bwd(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    assert float(dx.abs().max()) == 0 and float(dw.abs().max()) == 0


def test_without_weight_or_bias(ck):
    x, w, b, dy = make(50, 300, F32, F32, 5)
    compare(ck, x, None, None, dy)
    y, _, _ = ck.layernorm_fwd(x.cuda(), None, b.cuda(), eps=EPS)
    ref.check(y, ref.layer_norm(x, None, b, EPS)[0], tol(F32, 300), "y")
    m = ck.layernorm_fwd(x.cuda(), w.cuda(), eps=EPS)
    got = ck.layernorm_bwd(dy.cuda(), x.cuda(), m[1], m[2], w.cuda(), weight_grad=False)
    assert got[1] is None and got[2] is None


def test_large_offset_keeps_the_variance(ck):
    """A mean 1000 times the spread: the centred sum keeps what x - mean holds."""
    x, w, b, dy = make(20, 512, F32, F32, 7)
    x = x + 1000
    y, mean, rstd = ck.layernorm_fwd(x.cuda(), w.cuda(), b.cuda(), eps=EPS)
    # x - mean: the mean's own rounding is 1000 u of a spread near one
    ref.check(y, ref.layer_norm(x, w, b, EPS)[0], 4 * 1000 * 2 ** -24 + tol(F32, 512), "y")


def test_constant_rows(ck):
    x = torch.full((6, 256), 3.0)
    y, mean, rstd = ck.layernorm_fwd(x.cuda(), eps=EPS)
    assert float(y.abs().max()) == 0 and torch.equal(mean.cpu(), torch.full((6,), 3.0))
    assert torch.allclose(rstd.cpu(), torch.full((6,), EPS ** -0.5), rtol=1e-6)


def test_non_finite_rows_stay_alone(ck):
    x, w, b, _ = make(40, 128, BF, F32, 9)
    clean, _, _ = ck.layernorm_fwd(x.cuda(), w.cuda(), b.cuda())
    x[3, 5], x[8, 0] = float("inf"), float("nan")
    dirty, _, _ = ck.layernorm_fwd(x.cuda(), w.cuda(), b.cuda())
    keep = [i for i in range(40) if i not in (3, 8)]
    assert torch.equal(clean[keep], dirty[keep])
    assert torch.isnan(dirty[[3, 8]].float()).any(-1).all()


@pytest.mark.parametrize("dt", [BF, F32])
def test_misaligned_in_place_and_leading_axes(ck, dt):
    x, w, b, dy = make(24, 96, dt, F32, 11)
    buf = torch.empty(x.numel() + 1, dtype=dt, device="cuda")
    m = buf[1:].view(2, 3, 4, 96)
    m.copy_(x.view(2, 3, 4, 96))
    wy = ref.layer_norm(x, w, b, EPS)[0].view(2, 3, 4, 96)
    y, mean, rstd = ck.layernorm_fwd(m, w.cuda(), b.cuda(), eps=EPS)
    assert mean.shape == (2, 3, 4)
    ref.check(y, wy, tol(dt, 96), "y")
    g = dy.cuda().view(2, 3, 4, 96)
    dx, dw, db = ck.layernorm_bwd(g, m, mean, rstd, w.cuda())
    dx2, dw2, db2 = ck.layernorm_bwd(g, m, mean, rstd, w.cuda(), dx=g)
    assert dx2 is g and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    ck.layernorm_fwd(m, w.cuda(), b.cuda(), eps=EPS, y=m)
    assert torch.equal(m, y)


def test_no_rows(ck):
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = ck.layernorm_fwd(x)
    assert y.shape == (0, 64)
    _, dw, db = ck.layernorm_bwd(x, x, mean, rstd, torch.ones(64, device="cuda"))
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


def test_autograd_and_graph(ck):
    x, w, b, dy = (t.cuda() for t in make(300, 256, BF, F32, 13))
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    y = ck.layer_norm(*leaves, eps=EPS)
    y.backward(dy)
    m = ck.layernorm_fwd(x, w, b, eps=EPS)
    assert torch.equal(y, m[0])
    for t, r in zip(leaves, ck.layernorm_bwd(dy, x, m[1], m[2], w)):
        assert torch.equal(t.grad, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ck.layernorm_bwd(dy, x, m[1], m[2], w)
    dy.copy_(torch.randn_like(dy))
    graph.replay()
    torch.cuda.synchronize()
    for a, r in zip(got, ck.layernorm_bwd(dy, x, m[1], m[2], w)):
        assert torch.equal(a, r)


@pytest.mark.parametrize("dt,width", [(BF, 768), (BF, 1000), (BF, 1536), (BF, 2560), (BF, 5120), (BF, 12288), (BF, 16384), (F32, 400),
                                      (F32, 900), (F32, 5120), (F32, 8192)])
def test_more_rows_than_blocks(ck, dt, width):
    """Rows by a block each, several to a block: the ring comes round."""
    compare(ck, *make(2500 if width < 5000 else 700, width, dt, F32, width))
