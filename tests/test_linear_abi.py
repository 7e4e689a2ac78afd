"""Refusals of the linear-attention and layer-norm calls, on the host: bad
arguments return before anything is launched, and the binding raises before the
library is reached.  No call here reaches the GPU."""
import ctypes

import pytest
import torch

INV, UNS, WS = 1, 2, 5
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def ck():
    from gated_delta_rule_ckda_gb300 import build
    build.build()
    import gated_delta_rule_ckda_gb300 as ck
    return ck


def _fwd(L, **kw):
    p = lambda n, d=256: vp(kw.get(n, d))
    return L.ckda_linear_fwd(p("q"), p("k"), p("v"), p("g"), kw.get("per_head", 0), p("h0", None),
                             p("o"), p("hT", None), p("cu", None), kw.get("nseq", 0),
                             kw.get("B", 1), kw.get("H", 2), kw.get("Hk", 2), kw.get("T", 4),
                             kw.get("dk", 64), kw.get("dv", 64), kw.get("io", 1),
                             kw.get("scale", 1.0), p("ws", 4096), kw.get("wsb", 1 << 30), None)


def _bwd(L, **kw):
    p = lambda n, d=256: vp(kw.get(n, d))
    return L.ckda_linear_bwd(p("q"), p("k"), p("v"), p("g"), kw.get("per_head", 0), p("h0", None),
                             p("do"), p("dhT", None), p("dq"), p("dk"), p("dv"), p("dg"),
                             p("dh0", None), p("cu", None), kw.get("nseq", 0), kw.get("B", 1),
                             kw.get("H", 2), kw.get("Hk", 2), kw.get("T", 4), kw.get("ndk", 64),
                             kw.get("ndv", 64), kw.get("io", 1), kw.get("scale", 1.0),
                             p("ws", 4096), kw.get("wsb", 1 << 30), None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_linear_refusals(ck, call):
    L = ck.lib()
    nan = float("nan")
    bad = [dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(B=0), dict(H=0),
           dict(Hk=0), dict(H=3, Hk=2), dict(T=-1), dict(io=5), dict(scale=nan),
           dict(cu=256, nseq=2, B=2), dict(cu=256, nseq=0), dict(nseq=3, B=2)]
    for kw in bad:
        assert call(L, **kw) == INV, kw
    assert call(L, B=1 << 16, H=64, T=1 << 20) == UNS
    assert call(L, ws=None) == WS
    assert call(L, ws=4096 + 16) == WS
    assert call(L, wsb=128) == WS


def test_linear_width_limits(ck):
    L = ck.lib()
    assert _fwd(L, dk=129) == UNS and _fwd(L, dv=129) == UNS and _fwd(L, dk=0) == INV
    assert _bwd(L, ndk=129) == UNS and _bwd(L, ndv=129) == UNS and _bwd(L, ndv=0) == INV
    assert _fwd(L, o=None) == INV
    for n in ("do", "dq", "dk", "dv", "dg"):
        assert _bwd(L, **{n: None}) == INV


def test_step_refusals(ck):
    L = ck.lib()
    f = lambda **kw: L.ckda_linear_decode_step(
        *(vp(kw.get(n, 256)) for n in ("q", "k", "v", "g")), 0, vp(kw.get("state", 256)),
        vp(kw.get("o", 256)), kw.get("B", 1), kw.get("H", 4), kw.get("Hk", 2), kw.get("dk", 64),
        kw.get("dv", 64), kw.get("io", 0), kw.get("scale", 1.0), None)
    for n in ("q", "k", "v", "g", "state", "o"):
        assert f(**{n: None}) == INV
    assert f(B=0) == INV and f(Hk=3) == INV and f(io=9) == INV and f(scale=float("nan")) == INV
    assert f(dk=130) == UNS and f(dv=500) == UNS


def test_layernorm_refusals(ck):
    L = ck.lib()
    fw = lambda **kw: L.ckda_layernorm_fwd(
        *(vp(kw.get(n, 256)) for n in ("x", "w", "b", "y", "mean", "rstd")), kw.get("rows", 4),
        kw.get("width", 64), kw.get("io", 1), kw.get("wt", 0), kw.get("eps", 1e-5), None)
    for n in ("x", "y", "mean", "rstd"):
        assert fw(**{n: None}) == INV
    assert fw(rows=-1) == INV and fw(width=0) == INV and fw(io=2) == INV and fw(wt=-1) == INV
    assert fw(eps=-1.0) == INV and fw(eps=float("nan")) == INV and fw(rows=1 << 32) == UNS
    assert fw(rows=0, x=None, y=None) == 0          # nothing to do
    bw = lambda **kw: L.ckda_layernorm_bwd(
        *(vp(kw.get(n, 256)) for n in ("dy", "x", "mean", "rstd", "w", "dx", "dw", "db")),
        kw.get("rows", 4), kw.get("width", 64), kw.get("io", 1), kw.get("wt", 0),
        vp(kw.get("ws", 256)), kw.get("wsb", 1 << 20), None)
    for n in ("dy", "x", "mean", "rstd", "dx", "dw", "db"):
        assert bw(**{n: None}) == INV
    assert bw(width=0) == INV and bw(io=4) == INV
    assert bw(ws=None) == WS and bw(wsb=16) == WS and bw(ws=264) == WS


def test_binding_refuses(ck):
    """Shapes, types and strides are refused in Python, on CPU tensors."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    f32 = torch.float32
    ok = dict(q=z(2, 2, 8, 16), k=z(2, 2, 8, 16), v=z(2, 4, 8, 24), g=z(2, 4, 8, dt=f32))
    do = z(2, 4, 8, 24)
    bad = [dict(q=z(2, 2, 8, 16, dt=torch.float16)), dict(k=z(2, 2, 8, 17)),
           dict(k=z(2, 2, 8, 16, dt=f32)), dict(v=z(2, 3, 8, 24)), dict(g=z(2, 4, 8)),
           dict(g=z(2, 4, 9, dt=f32)), dict(g=z(5, dt=f32)), dict(h0=z(2, 4, 16, 24)),
           dict(h0=z(1, 4, 16, 24, dt=f32)), dict(q=z(2, 8, 2, 16).transpose(1, 2)),
           dict(cu_seqlens=z(3, dt=torch.int32))]
    for kw in bad:
        with pytest.raises((TypeError, ValueError)):
            ck.linear_fwd(**{**ok, **kw})
        with pytest.raises((TypeError, ValueError)):
            ck.linear_bwd(**{**ok, **kw}, do=do)
    one = {n: t[:1] for n, t in ok.items()}
    with pytest.raises(TypeError):
        ck.linear_fwd(**one, cu_seqlens=z(3, dt=torch.int64))
    with pytest.raises(ValueError):
        ck.linear_bwd(**ok, do=z(2, 4, 8, 16))
    s = dict(q=z(2, 2, 16), k=z(2, 2, 16), v=z(2, 4, 24), g=z(2, 4, dt=f32),
             state=z(2, 4, 16, 24, dt=f32))
    for kw in (dict(state=z(2, 4, 24, 16, dt=f32)), dict(state=z(2, 4, 16, 24)),
               dict(g=z(2, 4)), dict(q=z(2, 3, 16), k=z(2, 3, 16))):
        with pytest.raises((TypeError, ValueError)):
            ck.linear_decode_step(**{**s, **kw})
    for kw in (dict(x=z(4, 8, dt=torch.float64)), dict(weight=z(9)), dict(bias=z(8, dt=f32)),
               dict(x=z(8, 4).t()), dict(y=z(4, 8, dt=f32)), dict(mean=z(4))):
        with pytest.raises((TypeError, ValueError)):
            ck.layernorm_fwd(**{**dict(x=z(4, 8), weight=z(8)), **kw})
    b = dict(dy=z(4, 8), x=z(4, 8), mean=z(4, dt=f32), rstd=z(4, dt=f32), weight=z(8))
    for kw in (dict(dy=z(4, 9)), dict(mean=z(5, dt=f32)), dict(rstd=z(4)), dict(weight=z(7))):
        with pytest.raises((TypeError, ValueError)):
            ck.layernorm_bwd(**{**b, **kw})
