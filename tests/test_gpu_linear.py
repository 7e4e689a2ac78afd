"""Linear attention with a scalar decay per head against its 64-bit reference:
forward, backward and the single-token step."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def make(B, H, Hk, T, dk, dv, dt, seed, decay=0.3, h0=True, N=None):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)
    x = dict(q=r(B, Hk, T, dk).to(dt), k=r(B, Hk, T, dk).to(dt), v=r(B, H, T, dv).to(dt),
             g=-decay * torch.nn.functional.softplus(r(B, H, T)),
             h0=r(N or B, H, dk, dv) if h0 else None)
    extra = dict(do=r(B, H, T, dv).to(dt), dhT=r(N or B, H, dk, dv))
    return x, extra


def gpu(x):
    return {n: (t.cuda() if t is not None else None) for n, t in x.items()}


def compare(ck, x, extra, scale, cu=None, dh=True):
    """Forward and backward against the reference."""
    T, dt = x["q"].shape[2], x["q"].dtype
    d, e = gpu(x), gpu(extra)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, hT = ck.linear_fwd(**d, cu_seqlens=cud, scale=scale)
    assert ck.fwd_status(ck.linear_fwd.last_workspace) == 0
    dhT = extra["dhT"] if dh else None
    want = ref.linear(**x, cu=cu, scale=scale, do=extra["do"], dhT=dhT)
    ref.check(o, want[0], ref.token_tol(dt, T), "o")
    ref.check(hT, want[1], ref.state_tol(dt, T), "hT")
    got = ck.linear_bwd(d["q"], d["k"], d["v"], d["g"], e["do"], h0=d["h0"],
                        dhT=e["dhT"] if dh else None, cu_seqlens=cud, scale=scale)
    assert ck.fwd_status(ck.linear_bwd.last_workspace) == 0
    for name, t, w in zip(("dq", "dk", "dv"), got, want[2:]):
        assert t.dtype == dt
        ref.check(t, w, ref.token_tol(dt, T), name)
    ref.check(got[3], want[5], ref.decay_tol(dt, T), "dg")
    ref.check(got[4], want[6], ref.state_tol(dt, T), "dh0")


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 130])
def test_lengths(ck, dt, T):
    compare(ck, *make(2, 2, 2, T, 32, 48, dt, T), scale=32 ** -0.5)


@pytest.mark.parametrize("dk,dv", [(1, 1), (5, 3), (16, 128), (128, 16), (33, 65), (127, 128), (100, 7)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_widths(ck, dk, dv, dt):
    compare(ck, *make(1, 2, 1, 70, dk, dv, dt, 7), scale=1.0)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64), (8, 8), (96, 40), (72, 128), (120, 16)])
@pytest.mark.parametrize("T", [1, 37, 128, 129, 300])
def test_tensor_core_widths(ck, dk, dv, T):
    compare(ck, *make(1, 2, 2, T, dk, dv, BF, T + dk), scale=dk ** -0.5)


@pytest.mark.parametrize("T", [127, 255, 256, 257, 511, 640])
def test_tensor_core_lengths(ck, T):
    compare(ck, *make(2, 1, 1, T, 128, 128, BF, T), scale=128 ** -0.5)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("H,Hk", [(4, 1), (6, 2), (4, 4)])
@pytest.mark.parametrize("d", [20, 64])
def test_shared_key_heads(ck, dt, H, Hk, d):
    compare(ck, *make(2, H, Hk, 150, d, d, dt, H), scale=0.2)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("d", [24, 100, 128])
def test_packed_with_empty_and_single_token_sequences(ck, dt, d):
    cu = [0, 0, 1, 1, 66, 70, 70, 198, 327, 327]
    compare(ck, *make(1, 4, 2, 327, d, d, dt, 11, N=len(cu) - 1), scale=d ** -0.5, cu=cu)


@pytest.mark.parametrize("dt", [F32, BF])
def test_no_initial_state_and_no_state_gradient(ck, dt):
    x, e = make(2, 3, 3, 200, 64, 64, dt, 13, h0=False)
    compare(ck, x, e, scale=0.125, dh=False)


@pytest.mark.parametrize("dt,d", [(F32, 48), (BF, 128)])
@pytest.mark.parametrize("decay", [0.0, 0.001, 0.05, 3.0, 30.0])
def test_decays_from_none_to_strong(ck, dt, d, decay):
    compare(ck, *make(1, 2, 2, 400, d, d, dt, 17, decay=decay), scale=d ** -0.5)


@pytest.mark.parametrize("dt,d", [(F32, 48), (BF, 128), (BF, 50)])
def test_resets(ck, dt, d):
    """g = -inf forgets the state: at the first token, inside a chunk, at its
    border, twice in a row."""
    x, e = make(1, 2, 2, 300, d, d, dt, 19)
    for t in (0, 50, 127, 128, 129, 255, 299):
        x["g"][0, 0, t] = -float("inf")
    x["g"][0, 1, :] = -float("inf")
    compare(ck, x, e, scale=d ** -0.5)


@pytest.mark.parametrize("dt,d", [(F32, 40), (BF, 64), (BF, 128)])
def test_decay_of_a_head(ck, dt, d):
    x, e = make(2, 4, 2, 260, d, d, dt, 23)
    x["g"] = -torch.tensor([0.0, 0.01, 0.2, 2.0])
    compare(ck, x, e, scale=d ** -0.5)


@pytest.mark.parametrize("dt,d", [(F32, 40), (BF, 128)])
def test_neighbours_do_not_leak(ck, dt, d):
    """Infinities and NaN in one packed sequence leave the others' bits alone."""
    cu = [0, 75, 90, 260]
    x, e = make(1, 2, 2, 260, d, d, dt, 29, N=3)
    d0, e0 = gpu(x), gpu(e)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    run = lambda d_, e_: (*ck.linear_fwd(**d_, cu_seqlens=cud),
                          *ck.linear_bwd(d_["q"], d_["k"], d_["v"], d_["g"], e_["do"], h0=d_["h0"],
                                         dhT=e_["dhT"], cu_seqlens=cud))
    clean = run(d0, e0)
    for t in (d0["q"], d0["k"], d0["v"], e0["do"]):
        t[:, :, 75:90, ::2] = float("nan")
        t[:, :, 75:90, 1::2] = float("inf")
    d0["g"][:, :, 75:90] = float("nan")
    dirty = run(d0, e0)
    for a, b in zip(clean, dirty):
        if a.shape[0] == 3:
            assert torch.equal(a[[0, 2]], b[[0, 2]])
        else:
            assert torch.equal(a[:, :, :75], b[:, :, :75]) and torch.equal(a[:, :, 90:], b[:, :, 90:])
    assert torch.isnan(dirty[0][:, :, 75:90].float()).all()


@pytest.mark.parametrize("dt,d", [(F32, 33), (BF, 128)])
def test_state_carries_over_calls(ck, dt, d):
    """A sequence in two calls, the state handed on in place, is the sequence in one."""
    x, _ = make(1, 2, 2, 333, d, d, dt, 31)
    want = ref.linear(**x, scale=0.1)
    s = gpu(x)
    st = s["h0"].clone()
    outs = []
    for t0, t1 in ((0, 200), (200, 333)):
        p = {n: s[n][:, :, t0:t1].contiguous() for n in ("q", "k", "v", "g")}
        outs.append(ck.linear_fwd(**p, h0=st, hT=st, scale=0.1)[0])
    ref.check(torch.cat(outs, 2), want[0], ref.token_tol(dt, 333), "o")
    ref.check(st, want[1], ref.state_tol(dt, 333), "state")


@pytest.mark.parametrize("dt", [F32, BF])
def test_misaligned_inputs(ck, dt):
    """Contiguous tensors whose base is not 16-byte aligned."""
    x, e = make(1, 2, 2, 140, 64, 64, dt, 37)
    d, eo = gpu(x), gpu(e)

    def shift(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)
    m = {n: shift(d[n]) for n in ("q", "k", "v", "g", "h0")}
    want = ref.linear(**x, scale=0.1, do=e["do"], dhT=e["dhT"])
    o, hT = ck.linear_fwd(**m, scale=0.1)
    ref.check(o, want[0], ref.token_tol(dt, 140), "o")
    ref.check(hT, want[1], ref.state_tol(dt, 140), "hT")
    got = ck.linear_bwd(m["q"], m["k"], m["v"], m["g"], shift(eo["do"]), h0=m["h0"],
                        dhT=shift(eo["dhT"]), scale=0.1)
    for name, t, w in zip(("dq", "dk", "dv"), got, want[2:]):
        ref.check(t, w, ref.token_tol(dt, 140), name)
    ref.check(got[3], want[5], ref.decay_tol(dt, 140), "dg")
    ref.check(got[4], want[6], ref.state_tol(dt, 140), "dh0")


@pytest.mark.parametrize("dt,d", [(F32, 48), (BF, 128)])
def test_same_bits_again_and_on_another_stream(ck, dt, d):
    x, e = make(2, 4, 2, 700, d, d, dt, 41)
    d0, e0 = gpu(x), gpu(e)
    run = lambda: (*ck.linear_fwd(**d0), *ck.linear_bwd(d0["q"], d0["k"], d0["v"], d0["g"], e0["do"],
                                                        h0=d0["h0"], dhT=e0["dhT"]))
    first = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = run()
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_empty(ck):
    x, e = make(2, 2, 2, 0, 64, 64, BF, 43)
    d, eo = gpu(x), gpu(e)
    o, hT = ck.linear_fwd(**d)
    assert o.shape == (2, 2, 0, 64) and torch.equal(hT, d["h0"])
    *_, dg, dh0 = ck.linear_bwd(d["q"], d["k"], d["v"], d["g"], eo["do"], h0=d["h0"], dhT=eo["dhT"])
    assert dg.numel() == 0 and torch.equal(dh0, eo["dhT"])


@pytest.mark.parametrize("dt,d", [(F32, 32), (BF, 128)])
def test_autograd(ck, dt, d):
    x, e = make(1, 4, 2, 200, d, d, dt, 47)
    leaves = {n: t.cuda().requires_grad_() for n, t in x.items()}
    o, hT = ck.linear_attention(**leaves, scale=0.1)
    ((o.float() * e["do"].cuda().float()).sum() + (hT * e["dhT"].cuda()).sum()).backward()
    eo, d0 = gpu(e), gpu(x)
    want = ck.linear_bwd(d0["q"], d0["k"], d0["v"], d0["g"], eo["do"], h0=d0["h0"], dhT=eo["dhT"],
                         scale=0.1)
    for (n, t), w in zip(leaves.items(), want):
        assert torch.equal(t.grad, w), n
    # only the final state used; a decay shared over the batch through expand
    per = (-torch.rand(4, device="cuda")).requires_grad_()
    _, hT = ck.linear_attention(leaves["q"], leaves["k"], leaves["v"], per, scale=0.1)
    hT.sum().backward()
    assert per.grad.shape == (4,) and torch.isfinite(per.grad).all()


def test_graph_replay(ck):
    x, e = make(1, 4, 4, 300, 128, 128, BF, 53)
    d, eo = gpu(x), gpu(e)
    hT, o = torch.empty_like(d["h0"]), torch.empty_like(d["v"])
    ws = torch.empty(ck.linear_fwd_workspace_bytes(1, 4, 300, 128, 128), dtype=torch.uint8, device="cuda")
    ck.linear_fwd(**d, o=o, hT=hT, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ck.linear_fwd(**d, o=o, hT=hT, workspace=ws)
        back = ck.linear_bwd(d["q"], d["k"], d["v"], d["g"], eo["do"], h0=d["h0"], dhT=eo["dhT"])
    d["v"].copy_(torch.randn_like(d["v"]))
    graph.replay()
    torch.cuda.synchronize()
    o2, hT2 = ck.linear_fwd(**d)
    assert torch.equal(o, o2) and torch.equal(hT, hT2)
    for a, b in zip(back, ck.linear_bwd(d["q"], d["k"], d["v"], d["g"], eo["do"], h0=d["h0"], dhT=eo["dhT"])):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------- step
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 1, 1, 128, 128), (3, 4, 2, 128, 128), (2, 2, 2, 5, 3),
                                          (1, 6, 2, 127, 33), (40, 8, 8, 64, 128), (400, 1, 1, 20, 36),
                                          (1, 4, 1, 128, 60), (7, 45, 15, 96, 4)])
def test_step(ck, dt, B, H, Hk, dk, dv):
    x, _ = make(B, H, Hk, 3, dk, dv, dt, B + dk)
    want_o, want_h = ref.linear(**x, scale=0.3)
    st = x["h0"].cuda()
    outs = []
    for t in range(3):
        p = {n: x[n][:, :, t].contiguous().cuda() for n in ("q", "k", "v", "g")}
        outs.append(ck.linear_decode_step(**p, state=st, scale=0.3))
    ref.check(torch.stack(outs, 2), want_o, ref.token_tol(dt, 3), "o")
    ref.check(st, want_h, ref.state_tol(F32, 3), "state")


def test_step_reset_and_decay_of_a_head(ck):
    x, _ = make(2, 3, 3, 1, 64, 64, BF, 3)
    x["g"] = torch.tensor([-float("inf"), 0.0, -0.5])
    want_o, want_h = ref.linear(**x)
    st = x["h0"].cuda()
    p = {n: x[n][:, :, 0].contiguous().cuda() for n in ("q", "k", "v")}
    o = ck.linear_decode_step(**p, g=x["g"].cuda(), state=st)
    ref.check(o[:, :, None], want_o, ref.token_tol(BF, 1), "o")
    ref.check(st, want_h, ref.state_tol(F32, 1), "state")


def test_step_misaligned_state(ck):
    x, _ = make(1, 2, 2, 1, 32, 32, F32, 5)
    buf = torch.empty(x["h0"].numel() + 1, device="cuda")
    st = buf[1:].view(x["h0"].shape)
    st.copy_(x["h0"])
    want_o, want_h = ref.linear(**x)
    p = {n: x[n][:, :, 0].contiguous().cuda() for n in ("q", "k", "v", "g")}
    o = ck.linear_decode_step(**p, state=st)
    ref.check(o[:, :, None], want_o, ref.token_tol(F32, 1), "o")
    ref.check(st, want_h, ref.state_tol(F32, 1), "state")


# --------------------------------------------------------------- cut sequences
@pytest.mark.parametrize("T", [1152, 2000, 3071])
@pytest.mark.parametrize("d", [64, 128])
def test_few_heads_are_cut_into_segments(ck, T, d):
    """Far fewer heads than SMs: the sequence runs as segments and a scan joins their states."""
    x, e = make(1, 2, 1, T, d, d, BF, T, decay=0.02)
    x["g"][0, 0, T // 2] = -float("inf")
    compare(ck, x, e, scale=d ** -0.5)


def test_no_states_at_either_end_of_segments(ck):
    x, e = make(2, 1, 1, 1500, 128, 72, BF, 3, decay=0.01, h0=False)
    compare(ck, x, e, scale=0.1, dh=False)


def test_long_packed_sequences_are_cut(ck):
    cu = [0, 40, 1940, 1940, 3300, 3301]
    compare(ck, *make(1, 2, 1, 3301, 64, 96, BF, 5, decay=0.02, N=5), scale=0.125, cu=cu)


def test_cut_sequence_updates_its_state_in_place(ck):
    """hT may be h0, although different segments read the one and write the other."""
    x, _ = make(1, 2, 2, 2500, 64, 64, BF, 7, decay=0.01)
    want = ref.linear(**x, scale=0.1)
    s = gpu(x)
    o, _ = ck.linear_fwd(**s, hT=s["h0"], scale=0.1)
    ref.check(o, want[0], ref.token_tol(BF, 2500), "o")
    ref.check(s["h0"], want[1], ref.state_tol(BF, 2500), "state")


@pytest.mark.parametrize("T", [1, 100, 300])
def test_more_heads_than_sms(ck, T):
    """A CTA goes through several short sequences; widths and tails among them."""
    x, e = make(41, 8, 4, T, 64, 40, BF, T)
    d, eo = gpu(x), gpu(e)
    o, hT = ck.linear_fwd(**d, scale=0.125)
    grads = ck.linear_bwd(d["q"], d["k"], d["v"], d["g"], eo["do"], h0=d["h0"], dhT=eo["dhT"], scale=0.125)
    for b in (0, 18, 37, 40):   # sequences of different rounds
        y = {n: t[b:b + 1] for n, t in x.items()}
        z = {n: t[b:b + 1] for n, t in e.items()}
        want = ref.linear(**y, scale=0.125, **z)
        ref.check(o[b:b + 1], want[0], ref.token_tol(BF, T), "o")
        ref.check(hT[b:b + 1], want[1], ref.state_tol(BF, T), "hT")
        for name, t, w in zip(("dq", "dk", "dv"), grads, want[2:]):
            ref.check(t[b:b + 1], w, ref.token_tol(BF, T), name)
        ref.check(grads[3][b:b + 1], want[5], ref.decay_tol(BF, T), "dg")
        ref.check(grads[4][b:b + 1], want[6], ref.state_tol(BF, T), "dh0")


def test_many_packed_sequences(ck):
    gen = torch.Generator().manual_seed(9)
    cu = [0] + torch.randint(0, 200, (60,), generator=gen).cumsum(0).tolist()
    compare(ck, *make(1, 6, 3, cu[-1], 64, 64, BF, 11, N=60), scale=0.125, cu=cu)


def test_values_that_are_not_finite_keep_to_their_tokens(ck):
    """On CUDA cores: a NaN of v, k or q reaches only what the formula says."""
    T, at = 200, 70
    x, e = make(1, 2, 2, T, 20, 36, F32, 43)
    d, e = gpu(x), gpu(e)
    c, h0, do, dhT = [d[n] for n in "qkvg"], d["h0"], e["do"], e["dhT"]
    plain = ck.linear_fwd(*c, h0, scale=0.2)[0]
    for i in range(3):
        y = [z.clone() for z in c]
        y[i][:, :, at] = float("nan")
        o = ck.linear_fwd(*y, h0, scale=0.2)[0]
        torch.testing.assert_close(o[:, :, :at], plain[:, :, :at], rtol=0, atol=0)
        assert torch.isnan(o[:, :, at]).any()
        dq, dk, dv, dg, _ = ck.linear_bwd(*y, do, h0=h0, dhT=dhT, scale=0.2)
        if i > 0:  # k, v: queries before
            assert torch.isfinite(dq[:, :, :at]).all()
        if i != 1:  # q, v: keys behind
            assert torch.isfinite(dk[:, :, at + 1:]).all()
        assert torch.isfinite(dv[:, :, at + 1:]).all()


CHAINS = [("cut", BF, 2, 2, 1500, 64, None), ("packed", BF, 4, 2, 1700, 128, [0, 3, 3, 1500, 1700]),
          ("shared", BF, 4, 1, 260, 64, None), ("pieces", F32, 4, 2, 500, 40, None),
          ("packed pieces", F32, 2, 2, 500, 24, [0, 0, 130, 131, 500])]


@pytest.mark.parametrize("name,dt,H,Hk,T,d,cu", CHAINS, ids=[c[0] for c in CHAINS])
def test_calls_of_several_kernels(ck, name, dt, H, Hk, T, d, cu):
    """Kernels of a call may start under the one before: calls back to back on one
    workspace, and replayed from a graph, give the bits of calls apart."""
    N = 1 if cu is None else len(cu) - 1
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    inputs, apart = [], []
    nseq = 0 if cu is None else N
    per_head = -torch.rand(H, device="cuda") * 0.1

    def run(x, e, wf=None, wb=None):
        return [*ck.linear_fwd(**x, cu_seqlens=cud, workspace=wf),
                *ck.linear_bwd(x["q"], x["k"], x["v"], x["g"], e["do"], h0=x["h0"], dhT=e["dhT"],
                               cu_seqlens=cud, workspace=wb)]

    for seed in range(4):
        x, e = make(1, H, Hk, T, d, d, dt, seed, N=N)
        x, e = gpu(x), gpu(e)
        if seed % 2:
            x["g"] = per_head
        inputs.append((x, e))
        apart.append(run(x, e))
        torch.cuda.synchronize()
    wf = torch.empty(ck.linear_fwd_workspace_bytes(1, H, T, d, d, dt, nseq), dtype=torch.uint8, device="cuda")
    wb = torch.empty(ck.linear_bwd_workspace_bytes(1, H, Hk, T, d, d, dt, nseq), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        together = [run(x, e, wf, wb) for x, e in inputs]
        for a, b in zip(apart, together):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = [run(x, e, wf, wb) for x, e in inputs]
    for _ in range(3):
        for outs in replayed:
            for t in outs:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(apart, replayed):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
