"""The example blocks of a state space model: they train, and serving token by token agrees
with one call over the whole sequences; norm, convolution and scan together have the
gradients of their differences."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "state_space.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("state_space_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("more", [[], ["--states", "5", "--taps", "3", "--inner", "200"], ["--eight-bits"]])
def test_train_and_serve(example, more):
    losses, got, want = example.main(["--steps", "6", *more])
    assert torch.isfinite(losses).all()
    # Both sides round eight values in a row to bf16 in each of two blocks (norm, projection,
    # convolution, steps' two projections, scan, output projection, sum), by at most 2^-8 of
    # each, and may round apart in each; in 8 bits the norms' outputs too, each by up to 2^-4
    # on either side.
    far = 16 * 2 ** -8 + (2 * 2 ** -3 if "--eight-bits" in more else 0)
    assert (got.double() - want.double()).norm() <= far * want.double().norm()
    assert got.shape == (4, 20, 256)


@pytest.mark.parametrize("cu", [None, [0, 30, 30, 31, 70]])
def test_gradients_by_differences(example, cu):
    """Norm, convolution and scan in fp32 along a random direction, against a central
    difference in steps of h.  The loss has errors of a few 2^-24 of its terms' size, so the
    difference has at most that over h; a unit direction moves each row by a small part of
    itself, so the third derivative's term is below h^2 of that size."""
    gen = torch.Generator().manual_seed(3)
    B, T, D, N, G = 1, 70, 24, 6, 2
    mk = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    ck = example.ck
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    n = 1 if cu is None else len(cu) - 1
    leaves = [mk(B, T, 2 * D), mk(B, T, 2 * D), 1 + 0.1 * mk(2 * D), 0.5 * mk(D, 4), 0.1 * mk(D), mk(B, T, D) - 2,
              -mk(D, N).abs(), mk(B, T, G, N), mk(B, T, G, N), mk(D), 0.1 * mk(D), mk(n, 3, D), mk(n, D, N)]
    leaves = [t.requires_grad_() for t in leaves]
    r, rh, rc, rs = mk(B, T, D), mk(B, T, 2 * D), mk(n, 3, D), mk(n, D, N)

    def loss(u, h, w, cw, cb, dt, A, b, c, skip, bias, c0, s0):
        y, h = ck.rms_norm(u, w, h)
        x, cT = ck.short_conv(y[..., :D], cw, cb, c0, off)
        o, sT = ck.selective_scan(x, dt, A, b, c, skip, y[..., D:], bias, s0, off)
        return sum((p.double() * q.double()).sum() for p, q in ((o, r), (h, rh), (cT, rc), (sT, rs)))

    grads = torch.autograd.grad(loss(*leaves), leaves)
    h = 1e-2
    with torch.no_grad():
        scale = sum(t.double().square().sum() for t in (r, rh, rc, rs)).sqrt().item()
    for i, gr in enumerate(grads):
        u = mk(*leaves[i].shape)
        u /= u.norm()
        with torch.no_grad():
            up = [z if j != i else z + h * u for j, z in enumerate(leaves)]
            dn = [z if j != i else z - h * u for j, z in enumerate(leaves)]
            diff = ((loss(*up) - loss(*dn)) / (2 * h)).item()
        got = (gr.double() * u.double()).sum().item()
        # (terms here are products of up to three normal factors, four in size)
        assert abs(got - diff) <= 4 * scale * (16 * 2 ** -24 / h + h * h), (i, got, diff)


def test_one_graph_of_the_whole_pass(example):
    """Forward and backward of all three captured into one graph and replayed on new inputs."""
    ck = example.ck
    gen = torch.Generator().manual_seed(4)
    mk = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    D, N, T = 64, 16, 150
    u, h, w = mk(2, T, D).bfloat16(), mk(2, T, D).bfloat16(), mk(D)
    cw, A, b, c, dy = mk(D, 4), -mk(D, N).abs(), mk(2, T, N).bfloat16(), mk(2, T, N).bfloat16(), mk(2, T, D).bfloat16()

    def run():
        y, s, rstd = ck.rmsnorm_fwd(u, w, residual=h)
        x, _ = ck.conv_fwd(y, cw)
        o, _ = ck.scan_fwd(x, y, A, b, c, z=y)
        g = ck.scan_bwd(dy, x, y, A, b, c, z=y)
        dx, dw, _, _ = ck.conv_bwd(g[0], y, cw)
        return (o, *(t for t in g if t is not None), dx, dw, *ck.rmsnorm_bwd(dx, s, rstd, w, dh=s))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(2):
        u.copy_(torch.randn_like(u))
        dy.copy_(torch.randn_like(dy))
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(got, run()):
            assert torch.equal(a, e)


def test_calls_side_by_side_on_two_streams(example):
    """Every call on two streams at once, each with other inputs: the results of each alone."""
    ck = example.ck
    gen = torch.Generator().manual_seed(6)
    mk = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    D, N, T = 256, 16, 900

    def inputs():
        return dict(u=mk(2, T, D).bfloat16(), r=mk(2, T, D).bfloat16(), w=mk(D), cw=mk(D, 4), A=-mk(D, N).abs(),
                    b=mk(2, T, N).bfloat16(), c=mk(2, T, N).bfloat16(), dy=mk(2, T, D).bfloat16())

    def run(s):
        y, h, rstd = ck.rmsnorm_fwd(s["u"], s["w"], residual=s["r"])
        y8, scale, _, _ = ck.rmsnorm_fwd8(s["u"], s["w"], residual=s["r"], group=64)
        x, state = ck.conv_fwd(y, s["cw"])
        o, hT = ck.scan_fwd(x, y, s["A"], s["b"], s["c"], z=y)
        g = ck.scan_bwd(s["dy"], x, y, s["A"], s["b"], s["c"], z=y)
        back = ck.conv_bwd(g[0], y, s["cw"])
        return [o, hT, y8.float(), scale, state, *(t for t in (*g, *back) if t is not None),
                *ck.rmsnorm_bwd(back[0], h, rstd, s["w"], dh=h)]
    sets = [inputs(), inputs()]
    want = [run(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(run(s))
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(want[i % 2], outs):
            assert torch.equal(a, b)
