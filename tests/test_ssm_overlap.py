"""Outputs that share memory with inputs: convolution, scan and norm refuse what a block could
write while another still reads it, before anything is launched, and take the calls that
their documents allow, in place element for element."""
import ctypes

import pytest
import torch

import test_ssm_abi as abi
from test_ssm_abi import BAD, L, far, scan, vp  # noqa: F401

BF, F32 = torch.bfloat16, torch.float32


def at(i, off):
    return vp(0x1000000 * (i + 1) + off)


# ------------------------------------------------------------------------ refusals
# [2, 8, 16] in bf16: rows of 32 bytes, 512 in all; states of conv [2, 3, 16]
@pytest.mark.parametrize("bad", [
    dict(y=at(0, 2)), dict(y=at(0, -32)), dict(x=far(0), ldx=32, y=at(0, 512)), dict(h0=far(2)), dict(h0=at(2, 500)),
    dict(hT=far(2)), dict(hT=far(0)), dict(hT=at(0, 480))])
def test_conv_fwd(L, bad):  # noqa: F811
    assert abi.conv_fwd(L, **bad) == BAD


@pytest.mark.parametrize("bad", [
    dict(dx=at(0, 32)), dict(dx=at(1, -32)), dict(h0=far(3)), dict(dhT=at(3, 64)), dict(dh0=far(1)), dict(dh0=far(0)),
    dict(dh0=at(3, 100))])
def test_conv_bwd(L, bad):  # noqa: F811
    assert abi.conv_bwd(L, **bad) == BAD


@pytest.mark.parametrize("bad", [dict(y=at(0, 2)), dict(y=far(0), ldx=32), dict(y=far(2)), dict(y=at(2, 64)), dict(x=far(2))])
def test_conv_step(L, bad):  # noqa: F811
    a = dict(x=far(0), w=far(1), state=far(2), y=far(3), ldx=16)
    a.update(bad)
    assert L.ckda_conv_decode_step(a["x"], a["w"], None, a["state"], a["y"], 2, 16, 4, a["ldx"], 1, 0, 1, None) == BAD


@pytest.mark.parametrize("bad", [
    dict(y=at(0, 2)), dict(y=at(1, 480)), dict(y=far(0), ldx=24), dict(y=far(1), lddt=24), dict(z=far(14), y=at(14, -4)),
    dict(y=far(3)), dict(y=at(4, 100)), dict(h0=far(5)), dict(hT=far(5)), dict(hT=far(0)), dict(hT=far(1)), dict(hT=at(4, 64)),
    dict(D=4, ldx=4, lddt=4, y=far(3)), dict(h0=at(5, 16), hT=None)])
def test_scan_fwd(L, bad):  # noqa: F811
    assert scan(L, "fwd", **bad) == BAD


@pytest.mark.parametrize("bad", [
    dict(dx=at(0, 2)), dict(ddt=at(1, 480)), dict(dx=far(0), ldx=24), dict(dx=at(6, 32)), dict(z=far(14), dz=at(14, 32)),
    dict(dx=far(3)), dict(ddt=far(4)), dict(dB=far(0)), dict(dB=at(3, 8)), dict(dC=far(4), ldc=8), dict(dB=far(1)),
    dict(ddt=far(7)), dict(dB=far(7)), dict(dC=at(11, 8)), dict(z=far(14), dz=far(8)), dict(h0=far(20), dh0=at(20, 64)),
    dict(dh0=far(7)), dict(dh0=far(0)), dict(h0=far(20), dx=far(20)), dict(dhT=far(21), ddt=far(21)),
    dict(D=4, ldx=4, lddt=4, dx=far(3))])
def test_scan_bwd(L, bad):  # noqa: F811
    assert scan(L, "bwd", **bad) == BAD


@pytest.mark.parametrize("bad", [
    dict(y=at(0, 2)), dict(y=far(0), ldx=32), dict(y=at(1, -2)), dict(y=far(3)), dict(y=far(4)), dict(y=far(13)),
    dict(hT=far(0)), dict(hT=far(3)), dict(hT=at(5, -64)), dict(D=4, ldx=4, lddt=4, y=far(3))])
def test_scan_step(L, bad):  # noqa: F811
    assert scan(L, "step", **bad) == BAD


# [4, 128] in bf16: 1024 bytes
@pytest.mark.parametrize("bad", [
    dict(y=at(0, 2)), dict(y=at(0, -256)), dict(res=far(7), h=at(7, 256)), dict(res=far(7), h=at(0, 16)),
    dict(res=far(7), h=at(1, 256)), dict(res=far(7), h=far(8), y=at(7, 32))])
def test_norm(L, bad):  # noqa: F811
    a = dict(x=far(0), res=None, h=None, y=far(1))
    a.update(bad)
    assert L.ckda_rmsnorm_fwd(a["x"], a["res"], None, a["h"], a["y"], far(2), 4, 128, 1, 0, 1e-5, None) == BAD
    assert L.ckda_rmsnorm_fwd8(a["x"], a["res"], None, a["h"], a["y"], far(3), far(2), 4, 128, 0, 1, 0, 1e-5, None) == BAD


@pytest.mark.parametrize("y8,res,h", [(far(0), None, None), (at(0, 512), None, None), (far(7), far(7), far(8)),
                                      (at(8, 900), far(7), far(8))])
def test_norm_in_eight_bits(L, y8, res, h):  # noqa: F811
    assert L.ckda_rmsnorm_fwd8(far(0), res, None, h, y8, far(3), far(2), 4, 128, 0, 1, 0, 1e-5, None) == BAD


@pytest.mark.parametrize("i", [0, 1, 2])
@pytest.mark.parametrize("off", [2, 256, -256])
def test_norm_bwd(L, i, off):  # noqa: F811
    assert L.ckda_rmsnorm_bwd(far(0), far(1), far(5), None, far(2), at(i, off), None, 4, 128, 1, 0, None, 0, None) == BAD


# ------------------------------------------------------------------------ in place
def r(gen, *s, dt=F32):
    return torch.randn(*s, generator=gen).to(dt).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,D", [(BF, 256), (F32, 33)])
def test_steps_in_place(dt, D):
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator().manual_seed(1)
    x, w, state = r(gen, 9, D, dt=dt), r(gen, D, 4), r(gen, 9, 3, D, dt=dt)
    want, got = state.clone(), state.clone()
    y, z = ck.conv_decode_step(x, w, want), x.clone()
    assert ck.conv_decode_step(z, w, got, y=z) is z
    assert torch.equal(z, y) and torch.equal(got, want)
    A, B, h = -r(gen, D, 16).abs(), r(gen, 9, 16, dt=dt), r(gen, 9, D, 16)
    s = [r(gen, 9, D, dt=dt) for _ in range(3)]
    want = h.clone()
    y = ck.scan_decode_step(s[0], s[1], A, B, B, want, z=s[2])
    for i in range(3):
        c, got = [t.clone() for t in s], h.clone()
        ck.scan_decode_step(c[0], c[1], A, B, B, got, z=c[2], y=c[i])
        assert torch.equal(c[i], y) and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,rows,T,D,N", [(BF, 2, 50, 64, 16), (F32, 1, 900, 24, 8), (BF, 1, 700, 9, 5), (F32, 2, 700, 40, 64)])
def test_scan_in_place(dt, rows, T, D, N):
    """Forward through the binding; the gradients, whose memory it allocates, through the
    library: each in place of an input of its kind."""
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator().manual_seed(T)
    s = dict(x=r(gen, rows, T, D, dt=dt), dt=r(gen, rows, T, D, dt=dt), B=r(gen, rows, T, N, dt=dt), C=r(gen, rows, T, N, dt=dt),
             z=r(gen, rows, T, D, dt=dt), dy=r(gen, rows, T, D, dt=dt), h0=r(gen, rows, D, N), dhT=r(gen, rows, D, N))
    A, skip, bias = -r(gen, D, N).abs(), r(gen, D), r(gen, D)
    run = lambda c, **kw: ck.scan_fwd(c["x"], c["dt"], A, c["B"], c["C"], skip, c["z"], bias, c["h0"], **kw)  # noqa: E731
    y, hT = run(s)
    for k in ("x", "dt", "z"):
        c = {n: t.clone() for n, t in s.items()}
        got = run(c, y=c[k])
        assert got[0] is c[k] and torch.equal(got[0], y) and torch.equal(got[1], hT)
    want = ck.scan_bwd(s["dy"], s["x"], s["dt"], A, s["B"], s["C"], skip, s["z"], bias, s["h0"], s["dhT"])
    size = ck.lib().ckda_scan_bwd_workspace_bytes(rows, T, D, N, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for names in (("x", "dt", "z", "B", "C", "h0"), ("dy", "x", "dt", "C", "B", "h0"), ("z", "dy", "x", "B", "C", "h0")):
        c = {n: t.clone() for n, t in s.items()}
        dA, dskip, dbias = torch.empty_like(A), torch.empty_like(skip), torch.empty_like(bias)
        out = [c[n] for n in names]   # dx, ddt, dz, dB, dC, dh0
        p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        code = ck.lib().ckda_scan_bwd(
            p(c["dy"]), p(c["x"]), p(c["dt"]), p(A), p(c["B"]), p(c["C"]), p(skip), p(c["z"]), p(bias), p(c["h0"]),
            p(c["dhT"]), p(out[0]), p(out[1]), p(dA), p(out[3]), p(out[4]), p(dskip), p(out[2]), p(dbias), p(out[5]), None, 0,
            rows, T, D, N, 1, D, D, N, N, D, 1 if dt == BF else 0, 1, p(ws), size,
            ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert code == 0
        for a, b in zip((out[0], out[1], dA, out[3], out[4], dskip, out[2], dbias, out[5]), want):
            assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rows,width", [(3000, 256), (700, 1031), (4, 20000)])
def test_norm_in_place_of_the_residual(dt, rows, width):
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator().manual_seed(2)
    x, res, w = r(gen, rows, width, dt=dt), r(gen, rows, width, dt=dt), r(gen, width)
    want = ck.rmsnorm_fwd(x, w, residual=res)
    a, b = x.clone(), res.clone()
    y, h, rstd = ck.rmsnorm_fwd(a, w, residual=b, y=b)
    assert y is b and torch.equal(y, want[0]) and torch.equal(h, want[1]) and torch.equal(rstd, want[2])
    a, b = x.clone(), res.clone()
    y, h, _ = ck.rmsnorm_fwd(a, w, residual=b, y=b, h=a)
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
