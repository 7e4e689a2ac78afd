"""What short convolution, selective scan and RMS norm refuse, on the host: argument errors
of the C ABI and of the binding, memory that no kernel may be given, streams, and second
derivatives.  No call here reaches the GPU."""
import contextlib
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
BAD, UNS, WS = 1, 2, 5
P = vp(4096)
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_ckda_gb300 import build
    build.build()
    import gated_delta_rule_ckda_gb300 as ck
    return ck.lib()


def far(i):
    """Addresses that do not overlap for the sizes below."""
    return vp(0x1000000 * (i + 1))


# ------------------------------------------------------------------------- C ABI
def conv_fwd(L, x=far(0), w=far(1), b=None, h0=None, y=far(2), hT=None, cu=None, seqs=0, B=2, T=8, D=16, W=4, ldx=16,
             io=1, wt=0):
    return L.ckda_conv_fwd(x, w, b, h0, y, hT, cu, seqs, B, T, D, W, ldx, io, wt, 1, None)


@pytest.mark.parametrize("bad,code", [
    (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(B=0), BAD), (dict(T=-1), BAD), (dict(D=0), BAD),
    (dict(io=7), BAD), (dict(wt=7), BAD), (dict(ldx=15), BAD), (dict(cu=P, seqs=0, B=1), BAD), (dict(cu=P, seqs=3, B=2), BAD),
    (dict(W=1), UNS), (dict(W=5), UNS), (dict(B=1 << 20, T=1 << 20), UNS), (dict(D=(1 << 24) + 1, ldx=1 << 25), UNS),
    (dict(y=far(0)), BAD), (dict(y=vp(0x1000000 + 100)), BAD), (dict(h0=far(5), hT=far(5)), BAD),
    (dict(h0=far(5), hT=vp(0x1000000 * 6 + 64)), BAD)])
def test_conv_fwd(L, bad, code):
    assert conv_fwd(L, **bad) == code


def conv_bwd(L, dy=far(0), x=far(1), w=far(2), dx=far(3), dw=far(4), db=None, B=2, T=8, D=16, W=4, ldx=16, io=1, wt=0,
             ws=far(9), size=1 << 20, cu=None, seqs=0, h0=None, dhT=None, dh0=None):
    return L.ckda_conv_bwd(dy, x, w, None, h0, dhT, dx, dw, db, dh0, cu, seqs, B, T, D, W, ldx, io, wt, 1, ws, size, None)


@pytest.mark.parametrize("bad,code", [
    (dict(dy=None), BAD), (dict(x=None), BAD), (dict(w=None), BAD), (dict(dx=None), BAD), (dict(dw=None), BAD),
    (dict(dx=far(0)), BAD), (dict(dx=far(1)), BAD), (dict(W=6), UNS), (dict(ws=None), WS), (dict(size=64), WS),
    (dict(ws=vp(0x1000008)), WS), (dict(io=3), BAD), (dict(cu=P, seqs=2, B=2), BAD),
    (dict(h0=far(20), dh0=far(20)), BAD), (dict(dhT=far(20), dh0=vp(0x1000000 * 21 + 64)), BAD)])
def test_conv_bwd(L, bad, code):
    assert conv_bwd(L, **bad) == code


@pytest.mark.parametrize("bad,code", [(dict(x=None), BAD), (dict(state=None), BAD), (dict(y=None), BAD), (dict(w=None), BAD),
                                      (dict(B=0), BAD), (dict(W=1), UNS), (dict(W=9), UNS), (dict(ldx=3), BAD)])
def test_conv_step(L, bad, code):
    a = dict(x=far(0), w=far(1), state=far(2), y=far(3), B=2, D=16, W=4, ldx=16)
    a.update(bad)
    assert L.ckda_conv_decode_step(a["x"], a["w"], None, a["state"], a["y"], a["B"], a["D"], a["W"], a["ldx"], 1, 0, 1,
                                   None) == code


def scan(L, which, **bad):
    a = dict(x=far(0), dt=far(1), A=far(2), Bm=far(3), C=far(4), z=None, h0=None, y=far(5), hT=None, cu=None, seqs=0, B=2,
             T=8, D=16, N=4, G=1, ldx=16, lddt=16, ldb=4, ldc=4, ldz=16, io=1, ws=far(9), size=1 << 30, dy=far(6),
             dx=far(7), ddt=far(8), dA=far(10), dB=far(11), dC=far(12), dz=None, dhT=None, dh0=None)
    a.update(bad)
    lds = [a[k] for k in ("ldx", "lddt", "ldb", "ldc", "ldz")]
    dims = [a[k] for k in ("B", "T", "D", "N", "G")]
    if which == "fwd":
        return L.ckda_scan_fwd(a["x"], a["dt"], a["A"], a["Bm"], a["C"], None, a["z"], None, a["h0"], a["y"], a["hT"],
                               a["cu"], a["seqs"], *dims, *lds, a["io"], 1, a["ws"], a["size"], None)
    if which == "bwd":
        return L.ckda_scan_bwd(a["dy"], a["x"], a["dt"], a["A"], a["Bm"], a["C"], None, a["z"], None, a["h0"], a["dhT"],
                               a["dx"], a["ddt"], a["dA"], a["dB"], a["dC"], None, a["dz"], None, a["dh0"], a["cu"],
                               a["seqs"], *dims, *lds, a["io"], 1, a["ws"], a["size"], None)
    return L.ckda_scan_decode_step(a["x"], a["dt"], a["A"], a["Bm"], a["C"], None, a["z"], None, a["hT"] or far(13), a["y"],
                                   a["B"], a["D"], a["N"], a["G"], *lds, a["io"], 1, None)


COMMON = [(dict(x=None), BAD), (dict(dt=None), BAD), (dict(A=None), BAD), (dict(Bm=None), BAD), (dict(C=None), BAD),
          (dict(B=0), BAD), (dict(D=0), BAD), (dict(N=0), BAD), (dict(G=0), BAD), (dict(G=3), BAD), (dict(io=5), BAD),
          (dict(N=65, ldb=65, ldc=65), UNS), (dict(ldx=8), BAD), (dict(lddt=8), BAD), (dict(ldb=3), BAD), (dict(ldc=3), BAD),
          (dict(z=far(14), dz=far(15), ldz=8), BAD), (dict(D=(1 << 20) + 1, ldx=1 << 21, lddt=1 << 21), UNS)]
ROWS = [(dict(T=-1), BAD), (dict(cu=P, seqs=0, B=1), BAD), (dict(cu=P, seqs=2, B=2), BAD), (dict(T=(1 << 30) + 1), UNS),
        (dict(B=1 << 12, T=1 << 20), UNS)]


@pytest.mark.parametrize("bad,code", COMMON + ROWS + [
    (dict(y=None), BAD), (dict(h0=far(20), hT=far(20)), BAD), (dict(h0=far(20), hT=vp(0x1000000 * 21 + 128)), BAD),
    (dict(T=4096, ws=None), WS), (dict(T=4096, size=16), WS), (dict(T=4096, ws=vp(0x1000008)), WS)])
def test_scan_fwd(L, bad, code):
    assert scan(L, "fwd", **bad) == code


@pytest.mark.parametrize("bad,code", COMMON + ROWS + [
    (dict(dy=None), BAD), (dict(dx=None), BAD), (dict(ddt=None), BAD), (dict(dA=None), BAD), (dict(dB=None), BAD),
    (dict(dC=None), BAD), (dict(z=far(14)), BAD), (dict(dz=far(14)), BAD), (dict(dhT=far(20), dh0=far(20)), BAD),
    (dict(ws=None), WS), (dict(size=16), WS), (dict(ws=vp(0x1000008)), WS)])
def test_scan_bwd(L, bad, code):
    assert scan(L, "bwd", **bad) == code


@pytest.mark.parametrize("bad,code", COMMON + [(dict(y=None), BAD), (dict(B=(1 << 30) + 1, D=1, ldx=1, lddt=1), UNS)])
def test_scan_step(L, bad, code):
    bad = {k: v for k, v in bad.items() if k != "dz"}
    assert scan(L, "step", **bad) == code


def test_rmsnorm(L):
    def f(x=far(0), res=None, w=None, h=None, y=far(1), rstd=far(2), rows=4, width=128, io=1, wt=0, eps=1e-5):
        return L.ckda_rmsnorm_fwd(x, res, w, h, y, rstd, rows, width, io, wt, eps, None)

    def f8(scale=far(3), group=0, width=128, h=None, res=None, y=far(1)):
        return L.ckda_rmsnorm_fwd8(far(0), res, None, h, y, scale, far(2), 4, width, group, 1, 0, 1e-5, None)

    def b(dy=far(0), h=far(1), rstd=far(2), dx=far(3), dw=far(4), rows=4, width=128, io=1, wt=0, ws=far(5), size=1 << 20):
        return L.ckda_rmsnorm_bwd(dy, h, rstd, None, None, dx, dw, rows, width, io, wt, ws, size, None)
    for bad, code in ((dict(x=None), BAD), (dict(y=None), BAD), (dict(rstd=None), BAD), (dict(res=P), BAD), (dict(h=P), BAD),
                      (dict(res=far(7), h=far(1)), BAD), (dict(rows=-1), BAD), (dict(width=0), BAD), (dict(io=4), BAD),
                      (dict(wt=4), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
                      (dict(rows=1 << 31), UNS), (dict(width=(1 << 30) + 1), UNS)):
        assert f(**bad) == code, bad
    assert f(rows=0, x=None, y=None) == 0
    for bad in (dict(scale=None), dict(group=16), dict(group=128, width=192), dict(group=-32), dict(res=far(7)),
                dict(h=far(1), res=far(7))):
        assert f8(**bad) == BAD, bad
    for bad, code in ((dict(dy=None), BAD), (dict(h=None), BAD), (dict(rstd=None), BAD), (dict(dx=None), BAD),
                      (dict(ws=None), WS), (dict(size=32), WS), (dict(ws=vp(0x1000008)), WS), (dict(rows=-1), BAD),
                      (dict(width=(1 << 30) + 1), UNS)):
        assert b(**bad) == code, bad


def test_workspace_sizes(L):
    assert L.ckda_scan_fwd_workspace_bytes(8, 2048, 4096, 16, 1) == 0        # enough channels: one pass
    assert L.ckda_scan_fwd_workspace_bytes(1, 32768, 64, 16, 1) > 0
    assert L.ckda_scan_bwd_workspace_bytes(1, 0, 16, 4, 1) > 0
    for f, n in ((L.ckda_scan_fwd_workspace_bytes, 5), (L.ckda_scan_bwd_workspace_bytes, 5)):
        for i in range(n):
            a = [1, 64, 16, 4, 1]
            a[i] = -1 if i == 1 else 0
            assert f(*a) == 0
        assert f(1, 64, 16, 4, 3) == 0
    assert L.ckda_conv_bwd_workspace_bytes(1, 64, 16, 1) == 0 and L.ckda_conv_bwd_workspace_bytes(1, 64, 16, 5) == 0
    # the states before every 4th token are most of the backward's
    n = L.ckda_scan_bwd_workspace_bytes(4, 2048, 4096, 16, 1)
    assert 4 * 512 * 4096 * 16 * 4 < n < 2 * 4 * 512 * 4096 * 16 * 4


# ------------------------------------------------------------------------ binding
def calls(ck, z):
    """Each call by name, on tensors of z(shape, dtype)."""
    x, w, b = z((1, 8, 16), BF), z((16, 4), F32), z((16,), F32)
    sc = dict(x=x, dt=z((1, 8, 16), BF), A=z((16, 4), F32), B=z((1, 8, 4), BF), C=z((1, 8, 4), BF), D=b, z=x, dt_bias=b)
    one = {k: (v[:, 0].contiguous() if v.dim() == 3 else v) for k, v in sc.items()}
    rows, rstd = z((6, 64), BF), z((6,), F32)
    states = [z((1, 3, 16), BF), z((1, 16, 4), F32)]
    kept = []

    def state(i):  # updated in place, so each call has its own, which lives as long as the calls
        kept.append(states[i].clone())
        return kept[-1]
    return {
        "conv_fwd": lambda **s: ck.conv_fwd(x, w, b, **s),
        "conv_bwd": lambda **s: ck.conv_bwd(x, x, w, b, **s),
        "conv_decode_step": lambda **s: ck.conv_decode_step(x[:, 0], w, state(0), b, **s),
        "scan_fwd": lambda **s: ck.scan_fwd(**sc, **s),
        "scan_bwd": lambda **s: ck.scan_bwd(x, **sc, **s),
        "scan_decode_step": lambda **s: ck.scan_decode_step(**one, state=state(1), **s),
        "rmsnorm_fwd": lambda **s: ck.rmsnorm_fwd(rows, residual=rows, **s),
        "rmsnorm_fwd8": lambda **s: ck.rmsnorm_fwd8(rows, residual=rows, group=32, **s),
        "rmsnorm_bwd": lambda **s: ck.rmsnorm_bwd(rows, rows, rstd, **s),
    }


NAMES = ["conv_fwd", "conv_bwd", "conv_decode_step", "scan_fwd", "scan_bwd", "scan_decode_step", "rmsnorm_fwd",
         "rmsnorm_fwd8", "rmsnorm_bwd"]


class NoLaunch:
    def __getattr__(self, fn):
        def called(*a):
            assert fn.endswith("_bytes"), f"{fn} was launched"
            return 1024
        return called


@pytest.fixture
def run(monkeypatch):
    import gated_delta_rule_ckda_gb300 as ck
    monkeypatch.setattr(ck, "lib", lambda: NoLaunch())
    ck._bytes.cache_clear()
    yield calls(ck, lambda shape, dt: torch.zeros(shape, dtype=dt))
    ck._bytes.cache_clear()


@pytest.mark.parametrize("name", NAMES)
def test_tensors_in_host_memory(run, name):
    with pytest.raises(ValueError, match="on cpu, expected CUDA"):
        run[name]()


@pytest.mark.parametrize("name", ["conv_bwd", "scan_fwd", "scan_bwd", "rmsnorm_bwd"])
def test_workspace_elsewhere(run, name):
    with pytest.raises(ValueError, match="workspace: on meta"):
        run[name](workspace=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
    with pytest.raises(ValueError, match="workspace: must be contiguous"):
        run[name](workspace=torch.empty(1 << 20, dtype=torch.uint8)[::2])


def z(*s, dt=BF):
    return torch.zeros(*s, dtype=dt)


@pytest.mark.parametrize("change,error", [
    (dict(x=z(2, 8, 16).half()), TypeError), (dict(x=z(8, 16)), ValueError), (dict(weight=z(16, 4, dt=torch.float16)), TypeError),
    (dict(weight=z(15, 4)), ValueError), (dict(weight=z(16)), ValueError), (dict(bias=z(16, dt=F32)), TypeError),
    (dict(bias=z(15)), ValueError), (dict(h0=z(2, 4, 16)), ValueError), (dict(h0=z(2, 3, 16, dt=F32)), TypeError),
    (dict(x=z(2, 16, 8).transpose(1, 2)), ValueError), (dict(x=z(1, 8, 16).expand(2, 8, 16)), ValueError),
    (dict(x=z(2, 9, 16)[:, :8]), ValueError), (dict(x=z(2, 8, 32)[..., ::2]), ValueError),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError), (dict(y=z(2, 8, 8)), ValueError),
    (dict(hT=z(2, 3, 8)), ValueError)])
def test_conv_arguments(run, change, error):
    import gated_delta_rule_ckda_gb300 as ck
    a = dict(x=z(2, 8, 16), weight=z(16, 4), bias=z(16))
    a.update(change)
    with pytest.raises(error) as e:
        ck.conv_fwd(**a)
    assert "expected CUDA" not in str(e.value)


@pytest.mark.parametrize("change,error", [
    (dict(x=z(2, 8, 16).half()), TypeError), (dict(x=z(8, 16)), ValueError), (dict(dt=z(2, 8, 15)), ValueError),
    (dict(dt=z(2, 8, 16, dt=F32)), TypeError), (dict(A=z(16, 4)), TypeError), (dict(A=z(15, 4, dt=F32)), ValueError),
    (dict(A=z(16, dt=F32)), ValueError), (dict(B=z(2, 8, 5)), ValueError), (dict(B=z(2, 8, 1, 4)), ValueError),
    (dict(B=z(2, 8, 3, 4), C=z(2, 8, 3, 4)), ValueError), (dict(B=z(2, 8, 2, 4), C=z(2, 8, 4, 4)), ValueError),
    (dict(B=z(2, 8, 4, dt=F32), C=z(2, 8, 4, dt=F32)), TypeError), (dict(D=z(16)), TypeError), (dict(D=z(8, dt=F32)), ValueError),
    (dict(dt_bias=z(16)), TypeError), (dict(z=z(2, 8, 8)), ValueError), (dict(h0=z(2, 16, 4)), TypeError),
    (dict(h0=z(3, 16, 4, dt=F32)), ValueError), (dict(x=z(2, 16, 8).transpose(1, 2)), ValueError),
    (dict(B=z(2, 8, 4, 2).transpose(2, 3), C=z(2, 8, 2, 4)), ValueError), (dict(z=z(2, 9, 16)[:, :8]), ValueError),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), ValueError)])
def test_scan_arguments(run, change, error):
    import gated_delta_rule_ckda_gb300 as ck
    a = dict(x=z(2, 8, 16), dt=z(2, 8, 16), A=z(16, 4, dt=F32), B=z(2, 8, 4), C=z(2, 8, 4))
    a.update(change)
    with pytest.raises(error) as e:
        ck.scan_fwd(**a)
    assert "expected CUDA" not in str(e.value)


@pytest.mark.parametrize("change,error", [
    (dict(x=z(4, 64).half()), TypeError), (dict(x=z(64, 4).T), ValueError), (dict(weight=z(63)), ValueError),
    (dict(residual=z(4, 32)), ValueError), (dict(residual=z(4, 64, dt=F32)), TypeError), (dict(h=z(4, 64)), ValueError),
    (dict(y=z(4, 32)), ValueError), (dict(rstd=z(4)), TypeError), (dict(x=z(()).reshape(())), ValueError)])
def test_rms_arguments(run, change, error):
    import gated_delta_rule_ckda_gb300 as ck
    a = dict(x=z(4, 64))
    a.update(change)
    with pytest.raises(error) as e:
        ck.rmsnorm_fwd(**a)
    assert "expected CUDA" not in str(e.value)
    for group in (16, 48, 128, -32):
        with pytest.raises(ValueError, match="group"):
            ck.rmsnorm_fwd8(z(4, 64), group=group)


class FakeStream:
    device, cuda_stream = torch.device("cuda", 0), 77


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream(name, monkeypatch):
    """With the library and torch's streams replaced: whatever the call allocates, it
    allocates with the given stream current, and launches there."""
    import gated_delta_rule_ckda_gb300 as ck

    class Lib:
        def __getattr__(self, fn):
            if fn.endswith("_bytes"):
                return lambda *a: 1024

            def launch(*a):
                launched.append((fn, current[-1]))
                return 0
            return launch

    side, here = FakeStream(), object()
    current, inside, launched = [here], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    run = calls(ck, lambda shape, dt: torch.zeros(shape, dtype=dt))[name]
    monkeypatch.setattr(ck, "lib", lambda: Lib())
    monkeypatch.setattr(ck, "_call", lambda fn, *a: fn())
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    for n in ("empty", "empty_like"):
        def alloc(*a, _make=getattr(torch, n), **kw):
            inside.append(current[-1])
            return _make(*a, **kw)
        monkeypatch.setattr(torch, n, alloc)
    ck._bytes.cache_clear()
    try:
        run(stream=side)
    finally:
        ck._bytes.cache_clear()
    assert inside and all(s is side for s in inside)
    assert len(launched) == 1 and launched[0][1] is side


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_memory_used_again_on_the_callers_stream(name):
    """The stream is held up while the caller's stream takes and fills memory of every size that
    the call could have given back: the results are those of a call without a stream."""
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator(device="cuda").manual_seed(5)
    run = calls(ck, lambda shape, dt: (0.3 * torch.randn(shape, generator=gen, device="cuda")).to(dt))[name]
    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = run(stream=side)
    for _ in range(3):
        for n in (256, 1024, 4096, 16384, 1 << 16, 1 << 18):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for a, b in zip(want if isinstance(want, tuple) else (want,), got if isinstance(got, tuple) else (got,)):
        assert (a is None and b is None) or torch.equal(a.float(), b.float())


# ------------------------------------------------------------- second derivatives
def one(name, ck, monkeypatch):
    """(function of x, x) with the calls behind it replaced by torch's."""
    like = torch.ones_like
    if name == "short_conv":
        monkeypatch.setattr(ck, "conv_fwd", lambda x, *a, **kw: (x * x, x[:, :1].clone()))
        monkeypatch.setattr(ck, "conv_bwd", lambda dy, x, w, *a, **kw: (2 * x * dy, like(w), None, None))
        w = torch.ones(4, 4)
        return lambda x: ck.short_conv(x, w)[0], torch.randn(1, 3, 4)
    if name == "selective_scan":
        monkeypatch.setattr(ck, "scan_fwd", lambda x, *a, **kw: (x * x, x[:, :1].clone()))
        monkeypatch.setattr(ck, "scan_bwd", lambda dy, x, dt, A, B, C, *a, **kw: (
            2 * x * dy, like(dt), like(A), like(B), like(C), None, None, None, None))
        dt, A, B = torch.ones(1, 3, 4), torch.ones(4, 2), torch.ones(1, 3, 2)
        return lambda x: ck.selective_scan(x, dt, A, B, B)[0], torch.randn(1, 3, 4)
    monkeypatch.setattr(ck, "rmsnorm_fwd", lambda x, *a, **kw: (x * x, x, x[..., 0]))
    monkeypatch.setattr(ck, "rmsnorm_bwd", lambda dy, h, *a, **kw: (2 * h * dy, None))
    return ck.rms_norm, torch.randn(3, 4)


@pytest.mark.parametrize("name", ["short_conv", "selective_scan", "rms_norm"])
def test_a_gradient_penalty_is_refused(name, monkeypatch):
    import gated_delta_rule_ckda_gb300 as ck
    f, x = one(name, ck, monkeypatch)
    x.requires_grad_()
    (g,) = torch.autograd.grad(f(x).sum(), x, create_graph=True)
    torch.testing.assert_close(g, 2 * x)
    with pytest.raises(RuntimeError, match="no second derivative"):
        (f(x).sum() + g.square().sum()).backward()
    x.grad = None
    f(x).sum().backward()
    torch.testing.assert_close(x.grad, 2 * x.detach())
    assert not x.grad.requires_grad
