"""Short causal convolution, forward, backward and by single tokens, against its 64-bit
reference."""
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


def make(B, T, D, W, dt, wdt, seed=0, cu=None, bias=True, h0=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    s = dict(x=r(B, T, D).to(dt), w=(r(D, W) * W ** -0.5).to(wdt), b=(0.3 * r(D)).to(wdt) if bias else None,
             h0=r(n, W - 1, D).to(dt) if h0 else None, dy=r(B, T, D).to(dt), dhT=r(n, W - 1, D).to(dt) if h0 else None)
    s["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    return s


def compare(ck, s, silu=True, last=None):
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    (B, T, D), W, dt, wdt = s["x"].shape, s["w"].shape[1], s["x"].dtype, s["w"].dtype
    last = T if last is None else last
    wy, wh, g, size = ref.conv(s["x"], s["w"], s["b"], s["h0"], s["cu"], silu, s["dy"], s["dhT"])
    y, hT = ck.conv_fwd(c["x"], c["w"], c["b"], h0=c["h0"], cu_seqlens=c["cu"], silu=silu)
    tol = ref.conv_tol(dt, W)
    ref.check(y[:, :last], wy[:, :last], tol, "y")
    assert torch.equal(hT.cpu().double(), wh)   # inputs, moved
    dx, dw, db, dh0 = ck.conv_bwd(c["dy"], c["x"], c["w"], c["b"], h0=c["h0"], dhT=c["dhT"],
                                  cu_seqlens=c["cu"], silu=silu)
    assert dw.dtype == wdt and (db is None) == (s["b"] is None)
    ref.check(dx[:, :last], g["dx"][:, :last], tol, "dx", size=size["dx"])
    ref.check(dh0, g["dh0"], tol, "dh0", size=size["dh0"])
    weights = (ref.rounding(BF) if wdt == BF else 0.0) + ref.conv_tol(F32, W) + 2 * (B * T) ** 0.5 * ref.U[F32]
    ref.check(dw, g["dw"], weights, "dw", size=size["dw"])
    if db is not None:
        ref.check(db, g["db"], weights, "db", size=size["db"])


@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, F32), (BF, BF), (F32, BF)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [1, 4, 7, 8, 40, 130, 264, 1000])
def test_widths(ck, D, W, dt, wdt):
    compare(ck, make(2, 19, D, W, dt, wdt, seed=D))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 63, 64, 65, 130, 257, 700])
@pytest.mark.parametrize("dt,D", [(BF, 72), (F32, 33)])
def test_lengths(ck, T, dt, D):
    compare(ck, make(3, T, D, 4, dt, F32, seed=T))


@pytest.mark.parametrize("bias,silu,h0", [(False, True, False), (True, False, True), (False, False, False)])
def test_without_parts(ck, bias, silu, h0):
    compare(ck, make(2, 50, 48, 4, BF, F32, bias=bias, h0=h0), silu=silu)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dt,D", [(BF, 64), (BF, 5), (F32, 36)])
def test_packed(ck, dt, D, W):
    """Empty sequences, ones shorter than the state, borders inside and at the end of a run."""
    cu = [0, 0, 1, 3, 6, 6, 70, 134, 135, 200, 200]
    compare(ck, make(1, 200, D, W, dt, F32, cu=cu))


@pytest.mark.parametrize("D", [64, 5])
def test_tokens_behind_the_last_sequence(ck, D):
    s = make(1, 90, D, 4, BF, F32, cu=[0, 20, 61])
    compare(ck, s, last=61)
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    y = torch.full((1, 90, D), 7.0, dtype=BF, device="cuda")
    ck.conv_fwd(c["x"], c["w"], c["b"], cu_seqlens=c["cu"], y=y)
    assert (y[:, 61:] == 7).all() and not (y[:, :61] == 7).all()


def test_many_short_sequences(ck):
    gen = torch.Generator().manual_seed(3)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), torch.randint(0, 4, (300,), generator=gen).cumsum(0)]).tolist()
    compare(ck, make(1, cu[-1], 24, 4, F32, F32, cu=cu))


def test_part_of_a_projection(ck):
    """x as a slice of a wider last axis, aligned and not."""
    s = make(2, 33, 64, 4, BF, F32)
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    want = ck.conv_fwd(c["x"], c["w"], c["b"], h0=c["h0"])
    grads = ck.conv_bwd(c["dy"], c["x"], c["w"], c["b"], h0=c["h0"], dhT=c["dhT"])
    for at in (0, 64, 3):
        wide = torch.randn(2, 33, 200, device="cuda").to(BF)
        wide[..., at:at + 64] = c["x"]
        part = wide[..., at:at + 64]
        got = ck.conv_fwd(part, c["w"], c["b"], h0=c["h0"])
        again = ck.conv_bwd(c["dy"], part, c["w"], c["b"], h0=c["h0"], dhT=c["dhT"])
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        for i, (a, b) in enumerate(zip(grads, again)):   # (dw: sums of other runs where x is not aligned)
            if at != 3 or i in (0, 3):
                assert torch.equal(a, b)
            else:
                ref.check(b, a.cpu().double(), 2 * ref.conv_tol(F32, 4), "weights")
        step = ck.conv_decode_step(part[:, 0], c["w"], c["h0"].clone(), c["b"])
        assert torch.equal(step, want[0][:, 0])


def test_steps_continue_a_prompt(ck):
    for dt, D in ((BF, 64), (F32, 30)):
        s = make(3, 21, D, 4, dt, F32)
        c = {k: None if v is None else v.cuda() for k, v in s.items()}
        y, hT = ck.conv_fwd(c["x"], c["w"], c["b"], h0=c["h0"])
        _, state = ck.conv_fwd(c["x"][:, :9].contiguous(), c["w"], c["b"], h0=c["h0"])
        for t in range(9, 21):
            assert torch.equal(ck.conv_decode_step(c["x"][:, t], c["w"], state, c["b"]), y[:, t])
        assert torch.equal(state, hT)


def test_no_tokens(ck):
    s = make(2, 0, 16, 4, BF, F32)
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    y, hT = ck.conv_fwd(c["x"], c["w"], c["b"], h0=c["h0"])
    assert y.shape == (2, 0, 16) and torch.equal(hT, c["h0"])
    _, dw, db, dh0 = ck.conv_bwd(c["dy"], c["x"], c["w"], c["b"], h0=c["h0"], dhT=c["dhT"])
    assert not dw.any() and not db.any() and torch.equal(dh0, c["dhT"])


def test_values_that_are_not_finite_stay_near(ck):
    """A token reaches its own channel's next W tokens and no other sequence."""
    s = make(1, 80, 16, 4, F32, F32, cu=[0, 40, 80])
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    run = lambda: ck.conv_fwd(c["x"], c["w"], c["b"], h0=c["h0"], cu_seqlens=c["cu"])[0]  # noqa: E731
    clean = run()
    c["x"][0, 10, 3] = float("nan")
    c["x"][0, 38, 5] = float("inf")
    dirty = run()
    bad = torch.zeros_like(clean, dtype=torch.bool)
    bad[0, 10:14, 3] = True
    bad[0, 38:40, 5] = True
    assert torch.equal(clean[~bad], dirty[~bad]) and torch.isnan(dirty[0, 10:14, 3]).all()


def test_large_arguments(ck):
    """silu far out: p, and zero."""
    x = torch.tensor([200.0, -200.0, 1e30, -1e30, 88.0, -88.0]).view(1, 6, 1).cuda()
    w = torch.tensor([[0.0, 1.0]]).cuda()
    y, _ = ck.conv_fwd(x, w)
    dx = ck.conv_bwd(torch.ones_like(x), x, w)[0]
    assert torch.equal(y.flatten()[[0, 2]], x.flatten()[[0, 2]])
    assert y.flatten()[[1, 3, 5]].abs().max() < 1e-30
    assert torch.equal(dx.flatten()[[0, 2]], torch.ones(2, device="cuda")) and dx.flatten()[[1, 3]].abs().max() < 1e-30


def test_same_bits_and_captured(ck):
    s = make(4, 300, 256, 4, BF, F32)
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    run = lambda: (*ck.conv_fwd(c["x"], c["w"], c["b"], h0=c["h0"]),  # noqa: E731
                   *ck.conv_bwd(c["dy"], c["x"], c["w"], c["b"], h0=c["h0"], dhT=c["dhT"]),
                   ck.conv_decode_step(c["x"][:, 0], c["w"], c["h0"].clone(), c["b"]))
    first = run()
    assert all(torch.equal(a, b) for a, b in zip(first, run()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    c["x"].copy_(torch.randn_like(c["x"]))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))
    assert not torch.equal(first[0], got[0])


def test_autograd(ck):
    s = make(2, 40, 24, 4, F32, F32)
    c = {k: None if v is None else v.cuda() for k, v in s.items()}
    leaves = [c[k].clone().requires_grad_() for k in ("x", "w", "b", "h0")]
    y, hT = ck.short_conv(leaves[0], leaves[1], leaves[2], leaves[3])
    ((y * c["dy"]).sum() + (hT * c["dhT"]).sum()).backward()
    want = ck.conv_bwd(c["dy"], c["x"], c["w"], c["b"], h0=c["h0"], dhT=c["dhT"])
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, want))
    # through the state alone, and through a weight that is used twice
    leaves = [c[k].clone().requires_grad_() for k in ("x", "w")]
    _, hT = ck.short_conv(leaves[0], leaves[1])
    hT.sum().backward()
    assert leaves[0].grad[:, :-3].abs().max() == 0 and leaves[0].grad[:, -3:].eq(1).all()
    w = c["w"].clone().requires_grad_()
    (ck.short_conv(c["x"], w)[0] + ck.short_conv(c["x"], w)[0]).backward(c["dy"])
    one = ck.conv_bwd(c["dy"], c["x"], c["w"])[1]
    assert torch.equal(w.grad, one + one)


def test_more_tokens_than_a_wave(ck):
    compare(ck, make(1, 40000, 8, 3, BF, F32, h0=False))
