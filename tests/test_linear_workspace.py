"""What the calls of linear attention ask for as workspace.  On the host, with an unloaded GPU:
no call here launches anything."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
BF16, F32 = 1, 0
WS = 5


@pytest.fixture(scope="module")
def ck():
    from gated_delta_rule_ckda_gb300 import build
    build.build()
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


@pytest.mark.parametrize("nseq,B,H,T", [(0, 4, 32, 8192), (0, 8, 16, 2048), (0, 1, 16, 37)])
def test_aligned_forward_that_is_not_cut_needs_the_status_only(ck, nseq, B, H, T):
    L = ck.lib()
    assert L.ckda_linear_fwd_aligned_workspace_bytes(nseq, B, H, T, 128, 128, BF16) == 256
    assert L.ckda_linear_fwd_aligned_workspace_bytes(nseq, B, H, T, 64, 64, BF16) == 256


@pytest.mark.parametrize("nseq,B,H,T", [(0, 4, 32, 8192), (0, 1, 16, 32768), (0, 2, 8, 0),
                                        (24, 1, 16, 50021), (3, 1, 2, 100)])
@pytest.mark.parametrize("dk,dv,io", [(128, 128, BF16), (64, 96, BF16), (100, 128, BF16),
                                      (48, 80, F32)])
def test_enough_for_any_pointer_is_enough_for_aligned_ones(ck, nseq, B, H, T, dk, dv, io):
    L = ck.lib()
    a = (nseq, B, H, T, dk, dv, io)
    b = (nseq, B, H, H, T, dk, dv, io)
    for direction, args in (("fwd", a), ("bwd", b)):
        any_, aligned = (getattr(L, f"ckda_linear_{direction}{n}_workspace_bytes")(*args)
                         for n in ("", "_aligned"))
        assert 256 <= aligned <= any_
        if io == F32 or dk % 8:
            assert aligned == any_


def test_a_call_asks_for_what_its_pointers_take(ck):
    """Refused short of its own path's bytes; where that is met, the null stream's launch is next
    (not reached here: the calls stop at the workspace's alignment)."""
    L = ck.lib()
    B, H, T, d = 4, 32, 8192, 128
    fwd = lambda base, ws, n: L.ckda_linear_fwd(
        vp(base), vp(base), vp(base), vp(256), 0, None, vp(base), None, None, 0, B, H, H, T, d, d,
        BF16, 1.0, vp(ws), n, None)
    need = L.ckda_linear_fwd_aligned_workspace_bytes(0, B, H, T, d, d, BF16)
    assert fwd(256, 4096, need - 1) == WS and fwd(258, 4096, need) == WS
    bwd = lambda base, n: L.ckda_linear_bwd(
        vp(base), vp(base), vp(base), vp(256), 0, None, vp(base), None, vp(256), vp(256), vp(256),
        vp(256), None, None, 0, B, H, H, T, d, d, BF16, 1.0, vp(4096), n, None)
    need = L.ckda_linear_bwd_aligned_workspace_bytes(0, B, H, H, T, d, d, BF16)
    assert bwd(256, need - 1) == WS and bwd(258, need) == WS


@pytest.mark.parametrize("shift", [0, 1])
def test_the_binding_takes_the_fewer_bytes(ck, monkeypatch, shift):
    L, asked = ck.lib(), []
    monkeypatch.setattr(ck, "_call", lambda fn, where, *a: asked.append(a[-1]))
    def z(*s, dt=torch.bfloat16):
        n = 1
        for x in s:
            n *= x
        return torch.zeros(n + 8, dtype=dt)[shift:shift + n].view(s)
    B, H, T, d = 1, 2, 1000, 64
    q, g = z(B, H, T, d), torch.zeros(B, H, T)
    ck.linear_fwd(q, q, q, g)
    ck.linear_bwd(q, q, q, g, q)
    name = "" if shift else "_aligned"
    assert asked == [
        getattr(L, f"ckda_linear_fwd{name}_workspace_bytes")(0, B, H, T, d, d, BF16),
        getattr(L, f"ckda_linear_bwd{name}_workspace_bytes")(0, B, H, H, T, d, d, BF16)]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [140, 1000])
def test_calls_on_workspaces_of_just_their_bytes(ck, T):
    """Aligned and unaligned bases, each on exactly what it asks for."""
    import linear_ref as ref
    gen = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = [r(1, 2, T, 64).bfloat16() for _ in range(4)]
    g, h0 = -0.1 * r(1, 2, T).abs(), r(1, 2, 64, 64)
    want = ref.linear(*x[:3], g, h0, scale=0.1, do=x[3])
    L = ck.lib()
    for shift in (0, 1):
        d = []
        for t in x:
            buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
            d.append(buf[shift:shift + t.numel()].view(t.shape).copy_(t))
        name = "" if shift else "_aligned"
        wf, wb = (torch.empty(getattr(L, f"ckda_linear_{n}{name}_workspace_bytes")(*a),
                              dtype=torch.uint8, device="cuda")
                  for n, a in (("fwd", (0, 1, 2, T, 64, 64, BF16)),
                               ("bwd", (0, 1, 2, 2, T, 64, 64, BF16))))
        o, hT = ck.linear_fwd(*d[:3], g.cuda(), h0.cuda(), scale=0.1, workspace=wf)
        grads = ck.linear_bwd(*d[:3], g.cuda(), d[3], h0=h0.cuda(), scale=0.1, workspace=wb)
        tol = ref.token_tol(torch.bfloat16, T)
        for n, a, b in zip(("o", "dq", "dk", "dv"), (o, *grads[:3]), (want[0], *want[2:5])):
            ref.check(a, b, tol, n)
        ref.check(hT, want[1], ref.state_tol(torch.bfloat16, T), "hT")
        ref.check(grads[3], want[5], ref.decay_tol(torch.bfloat16, T), "dg")
        ref.check(grads[4], want[6], ref.state_tol(torch.bfloat16, T), "dh0")


@pytest.mark.parametrize("dk,dv", [(64, 64), (8, 40), (128, 64), (72, 48), (64, 128), (128, 128)])
def test_states_of_narrow_heads_take_no_more_than_their_panels(ck, dk, dv):
    """A state crosses memory in two bf16 parts and both directions, rounded up to panels of 64
    channels by 64 values; for single tokens the rest of the workspace is small beside it."""
    L = ck.lib()
    B, H = 512, 32
    panels = -(-dk // 64) * -(-dv // 64)
    states = B * H * 2 * 2 * panels * 64 * 64 * 2
    need = L.ckda_linear_bwd_aligned_workspace_bytes(0, B, H, H, 1, dk, dv, BF16)
    assert states <= need <= 1.01 * states + 4096


def test_a_call_holds_no_large_workspace(ck, monkeypatch):
    """What a call made for itself: given back before the next is made, and at its end but for
    the status word where it is large.  What the caller gave stays the caller's."""
    import weakref
    made, real = [], torch.empty

    def empty(*a, **kw):
        t = real(*a, **kw)
        if kw.get("dtype") == torch.uint8:
            assert t.numel() <= 1 << 20 or all(w() is None for w in made), "still held"
            made.append(weakref.ref(t))
        return t
    monkeypatch.setattr(ck, "_call", lambda fn, where, *a: None)
    monkeypatch.setattr(ck, "_LARGE", 64 << 20, raising=False)
    monkeypatch.setattr(torch, "empty", empty)
    q, g = torch.zeros(1, 16, 4000, 128, dtype=torch.bfloat16), torch.zeros(1, 16, 4000)
    for _ in range(3):
        ck.linear_bwd(q, q, q, g, q)
        held = ck.linear_bwd.last_workspace
        assert held.numel() == 256 and held.untyped_storage().nbytes() == 256
        assert made[-1]() is None
    made.clear()
    for _ in range(2):  # a small one is held, without a copy
        ck.linear_bwd(q[:, :2, :300].contiguous(), *[q[:, :2, :300].contiguous()] * 2,
                      g[:, :2, :300].contiguous(), q[:, :2, :300].contiguous())
        assert made[-1]() is ck.linear_bwd.last_workspace
    mine = real(1 << 30, dtype=torch.uint8, device="cpu")
    ck.linear_bwd(q, q, q, g, q, workspace=mine)
    assert ck.linear_bwd.last_workspace is mine
    ck.linear_bwd.last_workspace = None


@pytest.mark.gpu
def test_status_of_a_call_that_gave_its_workspace_back(ck, monkeypatch):
    monkeypatch.setattr(ck, "_LARGE", 1 << 16)
    x = torch.randn(1, 2, 1000, 64, device="cuda").bfloat16()
    ck.linear_bwd(x, x, x, torch.zeros(1, 2, 1000, device="cuda"), x, scale=0.01)
    assert ck.linear_bwd.last_workspace.numel() == 256
    assert ck.fwd_status(ck.linear_bwd.last_workspace) == 0
