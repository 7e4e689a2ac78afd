"""Selective scan, forward, backward and by single tokens, against its 64-bit reference."""
import math

import pytest
import torch

import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAMES = ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def make(B, T, D, N, dt, G=1, seed=0, cu=None, z=True, skip=True, bias=True, h0=True, softplus=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    n = B if cu is None else len(cu) - 1
    shape = (B, T, N) if G == 1 else (B, T, G, N)
    step = torch.exp(math.log(0.002) + math.log(100.0) * torch.rand(D, generator=gen))
    return dict(
        x=r(B, T, D).to(dt), dt=(r(B, T, D) if softplus else step * (0.5 + torch.rand(B, T, D, generator=gen))).to(dt),
        A=-torch.exp(0.8 * r(D, N)), B=r(*shape).to(dt), C=r(*shape).to(dt), D=r(D) if skip else None,
        z=r(B, T, D).to(dt) if z else None,
        bias=(step + torch.log(-torch.expm1(-step)) if softplus else 0.01 * r(D).abs()) if bias else None,
        h0=r(n, D, N) if h0 else None, cu=None if cu is None else torch.tensor(cu, dtype=torch.int32),
        softplus=softplus, dy=r(B, T, D).to(dt), dhT=r(n, D, N) if h0 else None)


def cuda(s):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}


def fwd(ck, c, **more):
    return ck.scan_fwd(c["x"], c["dt"], c["A"], c["B"], c["C"], D=c["D"], z=c["z"], dt_bias=c["bias"], h0=c["h0"],
                       cu_seqlens=c["cu"], softplus=c["softplus"], **more)


def bwd(ck, c, **more):
    return ck.scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"], D=c["D"], z=c["z"], dt_bias=c["bias"],
                       h0=c["h0"], dhT=c["dhT"], cu_seqlens=c["cu"], softplus=c["softplus"], **more)


def compare(ck, s, last=None):
    c = cuda(s)
    B, T, D = s["x"].shape
    dt = s["x"].dtype
    last = T if last is None else last
    wy, wh, want, size = ref.scan(*(s[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0", "cu", "softplus",
                                                   "dy", "dhT")))
    y, hT = fwd(ck, c)
    ref.check(y[:, :last], wy[:, :last], ref.scan_tol(dt, T), "y")
    ref.check(hT, wh, ref.scan_tol(F32, T), "hT")
    grads = dict(zip(NAMES, bwd(ck, c)))
    for name, given in (("dD", "D"), ("dz", "z"), ("ddt_bias", "bias")):
        assert (grads[name] is None) == (s[given] is None)
    for name, g in grads.items():
        if g is None:
            continue
        w = want[name]
        if name in ("dx", "ddt", "dz", "dB", "dC"):
            assert g.dtype == dt and g.shape == w.shape
            g, w = g[:, :last], w[:, :last]
            tol = ref.scan_tol(dt, T, True) if name[1] not in "BC" else ref.sum_tol(dt, T, D)
        else:
            assert g.dtype == F32
            tol = ref.scan_tol(F32, T, True) if name == "dh0" else ref.sum_tol(F32, T, B * T)
        ref.check(g, w, tol, name, size=size[name])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 31, 32, 33, 47, 64])
def test_states(ck, N, dt):
    compare(ck, make(2, 41, 40, N, dt, seed=N))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("D", [1, 5, 8, 24, 33, 64, 136, 200])
def test_channels(ck, D, N, dt):
    compare(ck, make(1, 35, D, N, dt, seed=D))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("N,dt", [(16, BF), (3, F32), (64, BF)])
def test_lengths(ck, T, N, dt):
    compare(ck, make(2, T, 24, N, dt, seed=T))


@pytest.mark.parametrize("G,D", [(2, 64), (3, 48), (4, 20), (5, 5)])
@pytest.mark.parametrize("N,dt", [(16, BF), (16, F32), (6, BF)])
def test_groups(ck, G, D, N, dt):
    compare(ck, make(2, 37, D, N, dt, G=G, seed=G))


@pytest.mark.parametrize("z,skip,bias,h0,softplus", [
    (False, True, True, True, True), (True, False, True, False, True), (True, True, False, True, True),
    (False, False, False, False, True), (True, True, True, True, False), (False, False, False, False, False)])
def test_without_parts(ck, z, skip, bias, h0, softplus):
    compare(ck, make(2, 50, 40, 16, BF, z=z, skip=skip, bias=bias, h0=h0, softplus=softplus))
    compare(ck, make(2, 50, 20, 5, F32, z=z, skip=skip, bias=bias, h0=h0, softplus=softplus))


# few channels: rows are cut into pieces that run side by side
@pytest.mark.parametrize("T", [200, 257, 640, 1000])
@pytest.mark.parametrize("N,dt,D", [(16, BF, 32), (16, F32, 30), (8, BF, 64), (64, F32, 8), (4, F32, 100)])
def test_pieces(ck, T, N, dt, D):
    compare(ck, make(1, T, D, N, dt, seed=T))
    compare(ck, make(3, T, D, N, dt, seed=T, h0=False))


PACKED = [0, 0, 1, 3, 40, 40, 41, 64, 128, 250, 250, 251, 700, 700]


@pytest.mark.parametrize("N,dt,D,G", [(16, BF, 32, 1), (16, F32, 24, 2), (5, BF, 9, 1), (64, BF, 16, 1), (4, F32, 136, 1),
                                      (32, BF, 40, 1), (8, F32, 16, 1)])
@pytest.mark.parametrize("h0", [True, False])
def test_packed(ck, N, dt, D, G, h0):
    """Empty sequences, single tokens, borders at a tile's, a chunk's and a piece's ends; one
    over many pieces."""
    compare(ck, make(1, 700, D, N, dt, G=G, cu=PACKED, h0=h0))


@pytest.mark.parametrize("N,D", [(16, 32), (3, 5)])
def test_tokens_behind_the_last_sequence(ck, N, D):
    s = make(1, 400, D, N, BF, cu=[0, 100, 290])
    compare(ck, s, last=290)
    c = cuda(s)
    y = torch.full((1, 400, D), 7.0, dtype=BF, device="cuda")
    fwd(ck, c, y=y)
    assert (y[:, 290:] == 7).all() and not (y[:, :290] == 7).any(-1).all()


@pytest.mark.parametrize("lengths", [[1] * 200, [0, 2] * 100, [0] * 150 + [5] + [0] * 150 + [300]])
def test_many_sequences(ck, lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    compare(ck, make(1, cu[-1], 16, 8, F32, cu=cu))


def test_one_wide_batch(ck):
    """More blocks than the card runs at once: one piece a row forward, two backward."""
    compare(ck, make(40, 33, 520, 16, BF, h0=False))


@pytest.mark.parametrize("D,N,dt,h0", [(520, 16, BF, True), (512, 8, F32, False)])
def test_wide_batch_of_longer_rows(ck, D, N, dt, h0):
    """Channels that fill the card: one piece a row in the backward pass too."""
    compare(ck, make(116, 45, D, N, dt, h0=h0))


@pytest.mark.parametrize("N,dt,D", [(16, BF, 32), (12, F32, 24), (5, BF, 9)])
def test_short_pieces(ck, N, dt, D):
    """Borders at and beside 32 tokens, the least of a piece in the backward pass."""
    compare(ck, make(1, 160, D, N, dt, cu=[0, 31, 32, 33, 96, 96, 127, 160]))
    compare(ck, make(2, 65, D, N, dt, h0=True))


def test_part_of_a_projection(ck):
    s = make(2, 45, 64, 16, BF, G=2)
    c = cuda(s)
    want = (*fwd(ck, c), *bwd(ck, c))
    wide = torch.randn(2, 45, 64 * 3 + 2 * 32 + 8, device="cuda").to(BF)
    at = 0
    parts = dict(c)
    for k in ("x", "dt", "z", "B", "C"):
        n = c[k].flatten(2).shape[-1]
        wide[..., at:at + n] = c[k].flatten(2)
        v = wide[..., at:at + n]
        parts[k] = v if k in ("x", "dt", "z") else v.unflatten(-1, (2, 16))
        at += n
    assert not parts["x"].is_contiguous() and not parts["B"].is_contiguous()
    for a, b in zip(want, (*fwd(ck, parts), *bwd(ck, parts))):
        assert torch.equal(a, b)
    odd = torch.randn(2, 45, 64 + 3, device="cuda").to(BF)
    odd[..., 3:] = c["x"]
    for a, b in zip(want, (*fwd(ck, dict(c, x=odd[..., 3:])), *bwd(ck, dict(c, x=odd[..., 3:])))):
        assert torch.equal(a, b)
    st = c["h0"].clone()
    first = ck.scan_decode_step(parts["x"][:, 0], parts["dt"][:, 0], c["A"], parts["B"][:, 0], parts["C"][:, 0], st,
                                D=c["D"], z=parts["z"][:, 0], dt_bias=c["bias"])
    ref.check(first, ref.d(want[0][:, 0]), 2 * ref.scan_tol(BF, 1), "step")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("N,D,G", [(16, 64, 1), (16, 100, 2), (1, 5, 1), (3, 7, 1), (4, 300, 1), (8, 33, 1), (12, 24, 3),
                                   (32, 70, 1), (64, 40, 1), (63, 9, 1)])
def test_steps(ck, N, D, G, dt):
    s = make(3, 6, D, N, dt, G=G, seed=N)
    c = cuda(s)
    wy, wh = ref.scan(*(s[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0", "cu")))
    state = c["h0"].clone()
    for t in range(6):
        y = ck.scan_decode_step(c["x"][:, t], c["dt"][:, t], c["A"], c["B"][:, t], c["C"][:, t], state, D=c["D"],
                                z=c["z"][:, t], dt_bias=c["bias"])
        ref.check(y, wy[:, t], ref.scan_tol(dt, 6), f"y of token {t}")
    ref.check(state, wh, ref.scan_tol(F32, 6), "state")


def test_step_without_parts_and_misaligned(ck):
    s = make(2, 1, 33, 8, F32, z=False, skip=False, bias=False, softplus=False)
    c = cuda(s)
    wy, wh = ref.scan(s["x"], s["dt"], s["A"], s["B"], s["C"], h0=s["h0"], softplus=False)
    buf = torch.empty(c["h0"].numel() + 1, device="cuda")
    state = buf[1:].view_as(c["h0"])
    state.copy_(c["h0"])
    y = ck.scan_decode_step(c["x"][:, 0], c["dt"][:, 0], c["A"], c["B"][:, 0], c["C"][:, 0], state, softplus=False)
    ref.check(y, wy[:, 0], ref.scan_tol(F32, 1), "y")
    ref.check(state, wh, ref.scan_tol(F32, 1), "state")


def test_steps_continue_a_prompt(ck):
    s = make(2, 30, 48, 16, F32)
    c = cuda(s)
    y, hT = fwd(ck, c)
    cut = dict(c, **{k: c[k][:, :17].contiguous() for k in ("x", "dt", "B", "C", "z")})
    _, state = fwd(ck, cut)
    for t in range(17, 30):
        o = ck.scan_decode_step(c["x"][:, t], c["dt"][:, t], c["A"], c["B"][:, t], c["C"][:, t], state, D=c["D"],
                                z=c["z"][:, t], dt_bias=c["bias"])
        ref.check(o, ref.d(y[:, t]), 2 * ref.scan_tol(F32, 30), f"token {t}")
    ref.check(state, ref.d(hT), 2 * ref.scan_tol(F32, 30), "state")


def test_no_tokens(ck):
    c = cuda(make(2, 0, 16, 4, BF))
    y, hT = fwd(ck, c)
    assert y.shape == (2, 0, 16) and torch.equal(hT, c["h0"])
    g = dict(zip(NAMES, bwd(ck, c)))
    assert torch.equal(g["dh0"], c["dhT"]) and not any(g[n].any() for n in ("dA", "dD", "ddt_bias"))
    c = cuda(make(1, 0, 16, 4, BF, cu=[0, 0, 0]))
    assert torch.equal(fwd(ck, c)[1], c["h0"]) and torch.equal(bwd(ck, c)[8], c["dhT"])


def test_small_and_large_steps(ck):
    """softplus far out on both sides; steps that decay a state to nothing, or not at all."""
    s = make(1, 12, 16, 4, F32, bias=False, h0=True)
    s["dt"] = torch.linspace(-30, 30, 12).view(1, 12, 1).expand(1, 12, 16).contiguous()
    compare(ck, s)
    s = make(1, 12, 16, 4, F32, softplus=False, bias=False)
    s["dt"][0, 3] = 0
    s["dt"][0, 7] = 200
    compare(ck, s)


def test_slow_decays_keep_their_precision(ck):
    """A memory of thousands of tokens, where a bias of the exponential would add up: the sum
    of 2000 decays' errors of one sign would be far outside the tolerance, which takes them
    as of changing sign."""
    s = make(1, 2000, 16, 4, F32, z=False, skip=False)
    s["A"] = -torch.full((16, 4), 0.05)
    compare(ck, s)


def test_values_that_are_not_finite_stay_in_their_sequence(ck):
    s = make(1, 600, 16, 16, F32, cu=[0, 200, 410, 600])
    c = cuda(s)
    clean = fwd(ck, c)
    clean_g = bwd(ck, c)
    c["x"][0, 250, 3] = float("nan")
    y, hT = fwd(ck, c)
    assert torch.isnan(y[0, 250:410, 3]).all() and torch.isnan(hT[1, 3]).all()
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 250:410, 3] = True
    assert torch.equal(y[~bad], clean[0][~bad]) and torch.equal(hT[[0, 2]], clean[1][[0, 2]])
    g = bwd(ck, c)
    for i in (0, 1, 3, 4, 6):   # dx, ddt, dB, dC, dz: of the other sequences' tokens
        for part in (slice(0, 200), slice(410, 600)):
            assert torch.equal(g[i][:, part], clean_g[i][:, part]), NAMES[i]
    assert torch.equal(g[8][[0, 2]], clean_g[8][[0, 2]])


def test_same_bits_and_captured(ck):
    c = cuda(make(2, 300, 96, 16, BF))
    run = lambda: (*fwd(ck, c), *bwd(ck, c))  # noqa: E731
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


def test_workspace_given(ck):
    c = cuda(make(1, 500, 64, 16, BF))
    want = (*fwd(ck, c), *bwd(ck, c))
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    for a, b in zip(want, (*fwd(ck, c, workspace=ws), *bwd(ck, c, workspace=ws))):
        assert torch.equal(a, b)
    with pytest.raises(ck.CkdaError) as e:
        bwd(ck, c, workspace=ws[:1024])
    assert e.value.code == 5


@pytest.mark.parametrize("D,T", [(64, 40), (64, 700)])
def test_autograd(ck, D, T):
    c = cuda(make(2, T, D, 16, F32))
    names = ("x", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    leaves = [c[k].clone().requires_grad_() for k in names]
    y, hT = ck.selective_scan(*leaves)
    torch.autograd.backward([y, hT], [c["dy"], c["dhT"]])
    for k, t, g in zip(names, leaves, bwd(ck, c)):
        assert torch.equal(t.grad, g), k
    del y, hT
    # B shared by two scans: its gradient is the sum of both
    B = c["B"].clone().requires_grad_()
    one = lambda: ck.selective_scan(c["x"], c["dt"], c["A"], B, c["C"])[0]  # noqa: E731
    (one() + one()).backward(c["dy"])
    g = ck.scan_bwd(c["dy"], c["x"], c["dt"], c["A"], c["B"], c["C"])[3]
    assert torch.equal(B.grad, g + g)


def test_differences(ck):
    """The gradients of a sum against differences of the forward in fp32: a step of 2^-6
    leaves 2^-12 of curvature and about 2^-24 / 2^-6 of rounding, on terms near one."""
    c = cuda(make(1, 24, 8, 4, F32))
    grads = dict(zip(("x", "dt", "A", "B", "C", "D", "z", "bias", "h0"), bwd(ck, c)))

    def loss():
        y, hT = fwd(ck, c)
        return float((y.double() * c["dy"].double()).sum() + (hT.double() * c["dhT"].double()).sum())
    size = 4 * (24 * 8) ** 0.5
    for name, g in grads.items():
        flat = c[name].view(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 3)):
            was = flat[i].item()
            flat[i] = was + 2.0 ** -6
            up = loss()
            flat[i] = was - 2.0 ** -6
            diff = (up - loss()) / 2 ** -5
            flat[i] = was
            got = float(g.reshape(-1)[i])
            assert abs(diff - got) <= (2 ** -12 + 2 ** -16) * size * max(1.0, abs(got)), (name, i, diff, got)
