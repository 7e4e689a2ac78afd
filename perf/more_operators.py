"""Cases of a state space block's operators: inputs, plain forms, calls, exact values.

Short causal convolution of each channel (W taps, W - 1 inputs of state):

    p_t = bias + sum_j weight_j x_{t-W+1+j},    y_t = silu(p_t) or p_t

the selective scan behind it (N states to a channel, step sizes, inputs and readouts by token):

    delta_t = softplus(dt_t + dt_bias),    h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
    y_t = (<C_t, h_t> + D x_t) silu(z_t)

and the root-mean-square norm before a block, with the residual's addition and an output in 8 bits:

    h = x + residual,    y = h rstd weight,    rstd = 1 / sqrt(mean(h^2) + eps)

each forward and backward, the first two also one token at a time on a resident state.  `own`
selects the framework's kernels (True) or the plain form in elementary torch operations (False).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
E4M3_MAX = 448.0
LEAST = 2.0 ** -100              # what a scale's largest value is taken for at least
MOST_CONV = 50021 * 4096         # token-channels of the largest convolution
MOST_FWD = 8 * 2048 * 4096 * 16  # token-channel-states of the largest scan
MOST_BWD = 4 * 2048 * 4096 * 16
MOST_NORM = 16384 * 4096


def listed():
    return [
        # ragged prompts packed together, before the scan of each
        dict(name="conv_packed", op="conv_fwd", B=1, T=50021, D=4096, W=4, dtype="bf16", wdtype="fp32", bias=1, silu=1, h0=0, seqs=24),
        # a training batch
        dict(name="conv_bwd", op="conv_bwd", B=8, T=2048, D=4096, W=4, dtype="bf16", wdtype="fp32", bias=1, silu=1, h0=0, seqs=0),
        # one user's next token: latency counts
        dict(name="conv_step", op="conv_step", B=1, D=4096, W=4, dtype="bf16", wdtype="fp32", bias=1, silu=1),
        # one user's short prompt, continued from a state
        dict(name="scan_short", op="scan_fwd", B=1, T=37, D=2048, N=16, G=1, dtype="bf16", z=1, h0=1, seqs=0),
        # a training batch
        dict(name="scan_batch", op="scan_fwd", B=8, T=2048, D=4096, N=16, G=1, dtype="bf16", z=1, h0=0, seqs=0),
        # long documents of ragged lengths packed together: few channels for the whole card
        dict(name="scan_long", op="scan_fwd", B=1, T=32768, D=2048, N=16, G=1, dtype="bf16", z=1, h0=0, seqs=3),
        # training
        dict(name="scan_bwd", op="scan_bwd", B=4, T=2048, D=4096, N=16, G=1, dtype="bf16", z=1, h0=0, seqs=0),
        # fp32 gradients of a small odd model, two groups of channels, initial state trained
        dict(name="scan_bwd_fp32", op="scan_bwd", B=2, T=1001, D=480, N=12, G=2, dtype="fp32", z=0, h0=1, seqs=0),
        # the serving batch
        dict(name="scan_step", op="scan_step", B=256, D=4096, N=16, G=1, dtype="bf16", z=1),
        # the norm before a projection in 8 bits, for a few tokens being decoded
        dict(name="rms_tokens", op="rms_fwd8", rows=7, width=2048, dtype="bf16", wdtype="bf16", residual=1, group=128),
        # the same for a prefill batch, a scale for each row
        dict(name="rms_batch", op="rms_fwd8", rows=16384, width=4096, dtype="bf16", wdtype="fp32", residual=1, group=0),
        # training, the residual stream's gradient passed on
        dict(name="rms_bwd", op="rms_bwd", rows=16384, width=4096, dtype="bf16", wdtype="fp32", residual=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_fwd", "conv_bwd", "conv_step", "scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step",
                     "rms_fwd", "rms_fwd8", "rms_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    wdtype = dtype if rng.random() < 0.5 else "fp32"
    if op.startswith("rms"):
        group = rng.choice([0, 0, 32, 64, 128]) if op == "rms_fwd8" else 0
        width = group * _log_int(rng, 1, 16384 // group) if group else _log_int(rng, 32, 16384)
        case = dict(op=op, rows=_log_int(rng, 1, MOST_NORM // width), width=width, dtype=dtype, wdtype=wdtype, residual=rng.randint(0, 1))
        return dict(case, group=group) if op == "rms_fwd8" else case
    # channels in whole vectors mostly, any number of them else
    D = 8 * _log_int(rng, 1, 1024) if rng.random() < 0.75 else _log_int(rng, 1, 8192)
    if op.startswith("conv"):
        case = dict(op=op, D=D, W=rng.choice([2, 3, 4, 4, 4]), dtype=dtype, wdtype=wdtype, bias=rng.randint(0, 1), silu=rng.choice([0, 1, 1]))
        if op == "conv_step":
            return dict(case, B=_log_int(rng, 1, max(1, min(1024, (1 << 20) // D))))
        most = (MOST_CONV if op == "conv_fwd" else 8 * 2048 * 4096) // D // (2 if dtype == "fp32" else 1)
    else:
        N = rng.choice([16, 16, 16, 8, 32, rng.randint(1, 64)])
        G = rng.choice([1, 1, 1, 2, 4])
        D = G * max(1, D // G)
        case = dict(op=op, D=D, N=N, G=G, dtype=dtype, z=rng.choice([0, 1, 1]))
        if op == "scan_step":
            return dict(case, B=_log_int(rng, 1, max(1, min(1024, (1 << 24) // (D * N)))))
        most = (MOST_FWD if op == "scan_fwd" else MOST_BWD) // (D * N) // (2 if dtype == "fp32" else 1)
    T = _log_int(rng, 1, max(1, min(32768, most)))
    packed = rng.random() < 0.3
    B = 1 if packed else _log_int(rng, 1, max(1, min(64, most // T)))
    return dict(case, B=B, T=T, h0=rng.randint(0, 1), seqs=_log_int(rng, 1, max(1, min(32, T // 4))) if packed else 0)


# ------------------------------------------------------------------------------------- inputs
def _offsets(case, seed):
    """Offsets of the packed sequences: ragged lengths, zero among them, the same total for every seed."""
    n, T = case["seqs"], case["T"]
    r = torch.Generator().manual_seed(int(seed) * 7919 + n)
    cuts = torch.sort(torch.randint(0, T + 1, (n - 1,), generator=r)).values
    return torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([T])])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device=DEV)

    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op.startswith("rms"):
        n, d, wdt = case["rows"], case["width"], DTYPES[case["wdtype"]]
        # a residual stream with a spread of its own in each row, and what a block adds to it
        spread = 0.5 + rand(n, 1)
        s["x"] = ((randn(n, d) * spread) if not case["residual"] else 0.5 * randn(n, d)).to(dt)
        s["w"] = (1 + 0.1 * randn(d)).to(wdt)
        s["res"] = (randn(n, d) * spread).to(dt) if case["residual"] else None
        if op == "rms_bwd":   # of the sum that the forward pass left
            s["h"] = (s["x"].float() + s["res"].float()).to(dt) if case["residual"] else s["x"]
            s["rstd"] = (s["h"].double().square().mean(-1) + EPS).rsqrt().float()
            s["dy"] = randn(n, d).to(dt)
            s["dh"] = randn(n, d).to(dt) if case["residual"] else None
        return s
    lead = (case["B"],) if op.endswith("step") else (case["B"], case["T"])
    D, count = case["D"], case["B"]
    s["cu"] = None
    if case.get("seqs"):
        count = case["seqs"]
        s["cu"] = _offsets(case, seed).to(torch.int32).to(DEV)
    back = op.endswith("bwd")
    if op.startswith("conv"):
        W, wdt = case["W"], DTYPES[case["wdtype"]]
        s["x"] = randn(*lead, D).to(dt)
        s["w"] = (randn(D, W) * W ** -0.5).to(wdt)
        s["b"] = (0.1 * randn(D)).to(wdt) if case["bias"] else None
        if op == "conv_step":
            s["state"] = randn(count, W - 1, D).to(dt)
            return s
        s["h0"] = randn(count, W - 1, D).to(dt) if case["h0"] else None
        if back:
            s["dy"] = randn(*lead, D).to(dt)
            s["dhT"] = randn(count, W - 1, D).to(dt) if case["h0"] else None
        return s
    N, G = case["N"], case["G"]
    s["x"] = torch.nn.functional.silu(randn(*lead, D)).to(dt)
    s["dt"] = randn(*lead, D).to(dt)
    # step sizes from 0.001 to 0.1 by channel, decay rates by state
    step = torch.exp(math.log(0.001) + math.log(100.0) * rand(D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(0.2 * randn(D, N))
    s["B"], s["C"] = randn(*lead, G, N).to(dt), randn(*lead, G, N).to(dt)
    s["D"] = 1 + 0.1 * randn(D)
    s["z"] = randn(*lead, D).to(dt) if case["z"] else None
    if op == "scan_step":
        s["state"] = randn(count, D, N)
        return s
    s["h0"] = randn(count, D, N) if case["h0"] else None
    if back:
        s["dy"] = randn(*lead, D).to(dt)
        s["dhT"] = randn(count, D, N) if case["h0"] else None
    return s


# -------------------------------------------------------------------------------- plain forms
def _borders(s):
    """Of every token: its place in its sequence, its sequence; of every sequence: batch row, first
    token and length.  Dense rows are sequences of one length."""
    c, cu = s["case"], s["cu"]
    t = torch.arange(c["T"], device=DEV)
    if cu is None:
        row = torch.arange(c["B"], device=DEV)
        return t.expand(c["B"], -1), row[:, None].expand(-1, c["T"]), row, torch.zeros_like(row), torch.full_like(row, c["T"])
    cu = cu.long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return (t - cu[seq])[None], seq[None], torch.zeros_like(cu[1:]), cu[:-1], cu[1:] - cu[:-1]


def _silu_grad(p):
    g = torch.sigmoid(p)
    return g * (1 + p * (1 - g))


def _taps(s):
    """The W inputs of every token, x_{t-W+1} to x_t: before a sequence's start its state, or zero."""
    W, x = s["case"]["W"], s["x"].float()
    place, seq = _borders(s)[:2]
    back = torch.arange(W - 1, -1, -1, device=DEV)
    t = torch.arange(x.shape[1], device=DEV)
    at = (t[:, None] - back).clamp(min=0)                    # [T, W]
    before = place[..., None] - back                         # [B, T, W], < 0: in the state
    taps = x[:, at]                                          # [B, T, W, D]
    if s["h0"] is None:
        return torch.where((before >= 0)[..., None], taps, 0)
    b, i, j = (before < 0).nonzero(as_tuple=True)
    taps[b, i, j] = s["h0"].float()[seq[b, i], before[b, i, j] + W - 1]
    return taps


def _conv_state(s):
    """The last W - 1 inputs of every sequence, its initial state's where it has fewer."""
    W, x = s["case"]["W"], s["x"]
    _, _, row, first, length = _borders(s)
    at = length[:, None] - (W - 1) + torch.arange(W - 1, device=DEV)
    own_rows = x[row[:, None], (first[:, None] + at).clamp(0, x.shape[1] - 1)]
    old = torch.zeros_like(own_rows) if s["h0"] is None else s["h0"].gather(1, (at + W - 1).clamp(0, W - 2)[..., None].expand_as(s["h0"]))
    return torch.where((at >= 0)[..., None], own_rows, old)


def _plain_conv_fwd(s):
    p = (_taps(s) * s["w"].float().T).sum(-2)
    if s["b"] is not None:
        p = p + s["b"].float()
    if s["case"]["silu"]:
        p = p * torch.sigmoid(p)
    return {"y": p.to(s["x"].dtype), "hT": _conv_state(s)}


def _plain_conv_bwd(s):
    c, w, dt = s["case"], s["w"].float(), s["x"].dtype
    W, B, T, D = c["W"], c["B"], c["T"], c["D"]
    taps, dp = _taps(s), s["dy"].float()
    if c["silu"]:
        p = (taps * w.T).sum(-2)
        dp = dp * _silu_grad(p if s["b"] is None else p + s["b"].float())
    out = {"dw": (dp[..., None, :] * taps).double().sum((0, 1)).T.to(s["w"].dtype)}
    if s["b"] is not None:
        out["db"] = dp.double().sum((0, 1)).to(s["w"].dtype)
    place, seq, row, first, length = _borders(s)
    # input i feeds tap W - 1 - k of token i + k, where that is in its sequence
    end = torch.where(place >= 0, length[seq], 0)
    reach = torch.arange(W, device=DEV)
    t = torch.arange(T, device=DEV)
    at = (t[:, None] + reach).clamp(max=T - 1)
    inside = (place[..., None] + reach < end[..., None])[..., None]
    dx = (torch.where(inside, dp[:, at], 0) * w.T.flip(0)).sum(-2)
    if s["dhT"] is not None:
        left = place - end + W - 1                           # the row of the final state that holds the input
        b, i = (left >= 0).nonzero(as_tuple=True)
        dx[b, i] += s["dhT"].float()[seq[b, i], left[b, i]]
    out["dx"] = dx.to(dt)
    if s["h0"] is not None:
        r = torch.arange(W - 1, device=DEV)
        # row r of the initial state feeds tap r - k of token k
        k = torch.arange(W - 1, device=DEV)
        use = (k[None] <= r[:, None])[None] & (k[None, None] < length[:, None, None])
        rows = dp[row[:, None], (first[:, None] + k).clamp(max=T - 1)]      # [seqs, W - 1, D]
        tap = w.T[(r[:, None] - k[None]).clamp(min=0)]                      # [W - 1, W - 1, D]
        dh0 = (torch.where(use[..., None], rows[:, None], 0) * tap).sum(2)
        if s["dhT"] is not None:
            kept = r[None] - length[:, None]                                # rows that a short sequence hands on
            old = s["dhT"].float().gather(1, kept.clamp(min=0)[..., None].expand_as(dh0))
            dh0 = dh0 + torch.where((kept >= 0)[..., None], old, 0)
        out["dh0"] = dh0.to(dt)
    return out


def _plain_conv_step(s):
    w, st = s["w"].float(), s["state"]
    taps = torch.cat([st, s["x"][:, None]], 1)
    p = (taps.float() * w.T).sum(1)
    if s["b"] is not None:
        p = p + s["b"].float()
    if s["case"]["silu"]:
        p = p * torch.sigmoid(p)
    st.copy_(taps[:, 1:])
    return {"y": p.to(s["x"].dtype), "state": st}


def _steps(s):
    """Step sizes, and the argument of their softplus."""
    raw = s["dt"].float() + s["dt_bias"]
    return torch.where(raw > 0, raw, 0) + torch.log1p(torch.exp(-raw.abs())), raw


def _channels(x, D):
    """[..., G, N] -> [..., D, N]: the group of each channel."""
    return x.float().repeat_interleave(D // x.shape[-2], -2)


def _run_through(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1, spans of tokens joined to twice as long ones."""
    n = 1
    while n < a.shape[1]:
        b = torch.cat([b[:, :n], torch.addcmul(b[:, n:], a[:, n:], b[:, :-n])], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _scan_states(s, delta, decay):
    """h_t of every token, and the decays that stop at a sequence's start."""
    c = s["case"]
    place, seq = _borders(s)[:2]
    b = (delta * s["x"].float())[..., None] * _channels(s["B"], c["D"])
    start = (place == 0)[..., None, None]
    if s["h0"] is not None:
        i, t = (place == 0).nonzero(as_tuple=True)
        b[i, t] += decay[i, t] * s["h0"][seq[i, t]]
    inner = torch.where(start, 0, decay)
    return _run_through(inner, b), inner


def _plain_scan_fwd(s):
    c, x = s["case"], s["x"].float()
    delta, _ = _steps(s)
    h, _ = _scan_states(s, delta, torch.exp(delta[..., None] * s["A"]))
    y = (h * _channels(s["C"], c["D"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    _, _, row, first, length = _borders(s)
    hT = h[row, (first + length - 1).clamp(min=0)]
    empty = s["h0"] if s["h0"] is not None else torch.zeros_like(hT)
    hT = torch.where((length > 0)[:, None, None], hT, empty)
    return {"y": y.to(s["x"].dtype), "hT": hT}


def _grouped(x, G):
    """Sums over the channels of each group: [..., D, N] -> [..., G, N]."""
    return x.unflatten(-2, (G, x.shape[-2] // G)).sum(-2)


def _plain_scan_bwd(s):
    c, x, dt = s["case"], s["x"].float(), s["x"].dtype
    D, G = c["D"], c["G"]
    place, seq, row, first, length = _borders(s)
    delta, raw = _steps(s)
    decay = torch.exp(delta[..., None] * s["A"])
    h, inner = _scan_states(s, delta, decay)
    Bc, Cc, out = _channels(s["B"], D), _channels(s["C"], D), {}
    dy = s["dy"].float()
    if s["z"] is not None:
        z = s["z"].float()
        out["dz"] = (dy * ((h * Cc).sum(-1) + s["D"] * x) * _silu_grad(z)).to(dt)
        dy = dy * z * torch.sigmoid(z)
    out["dC"] = _grouped(dy[..., None] * h, G).to(dt)
    # g_t = dy_t C_t + a_{t+1} g_{t+1}
    g = dy[..., None] * Cc
    if s["dhT"] is not None:
        full = length > 0
        g[row[full], (first + length - 1)[full]] += s["dhT"][full]
    after = torch.cat([inner[:, 1:], torch.zeros_like(inner[:, :1])], 1)
    g = _run_through(after.flip(1), g.flip(1)).flip(1)
    old = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    old = torch.where((place == 0)[..., None, None], 0, old)
    if s["h0"] is not None:
        i, t = (place == 0).nonzero(as_tuple=True)
        old[i, t] = s["h0"][seq[i, t]]
        full = length > 0
        out["dh0"] = torch.zeros_like(s["h0"]) if s["dhT"] is None else s["dhT"].clone()
        out["dh0"][full] = (decay * g)[row[full], first[full]]
    out["dB"] = _grouped((delta * x)[..., None] * g, G).to(dt)
    gB = (g * Bc).sum(-1)
    out["dx"] = (delta * gB + s["D"] * dy).to(dt)
    old = g * decay * old
    ddelta = (old * s["A"]).sum(-1) + gB * x
    ddt = ddelta * torch.sigmoid(raw)
    out["ddt"] = ddt.to(dt)
    out["ddt_bias"] = ddt.double().sum((0, 1)).float()
    out["dA"] = (old * delta[..., None]).sum((0, 1), dtype=torch.float64).float()
    out["dD"] = (dy * x).double().sum((0, 1)).float()
    return out


def _plain_scan_step(s):
    c, x, st = s["case"], s["x"].float(), s["state"]
    delta, _ = _steps(s)
    st.mul_(torch.exp(delta[..., None] * s["A"])).add_((delta * x)[..., None] * _channels(s["B"], c["D"]))
    y = (st * _channels(s["C"], c["D"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype), "state": st}


def _plain_rms_fwd(s):
    out, h, dt = {}, s["x"], s["x"].dtype
    if s["res"] is not None:
        h = out["h"] = (h.float() + s["res"].float()).to(dt)
    h = h.float()
    rstd = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    out["rstd"] = rstd[:, 0]
    y = h * rstd * s["w"].float()
    if s["case"]["op"] == "rms_fwd":
        out["y"] = y.to(dt)
        return out
    group = s["case"]["group"] or y.shape[1]
    y = y.unflatten(1, (-1, group))
    most = y.abs().amax(-1).clamp(min=LEAST)
    out["scale"] = most / E4M3_MAX if s["case"]["group"] else most[:, 0] / E4M3_MAX
    q = (y * (E4M3_MAX / most)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    out["y"] = q.flatten(1).to(torch.float8_e4m3fn)   # e4m3 values, in units of their scale
    return out


def _plain_rms_bwd(s):
    rstd, dy = s["rstd"][:, None], s["dy"].float()
    xh = s["h"].float() * rstd
    t = dy * s["w"].float()
    dx = rstd * (t - xh * (t * xh).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0, dtype=torch.float64).to(s["w"].dtype)}


PLAIN = {"conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd, "conv_step": _plain_conv_step,
         "scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step,
         "rms_fwd": _plain_rms_fwd, "rms_fwd8": _plain_rms_fwd, "rms_bwd": _plain_rms_bwd}


# ------------------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import gated_delta_rule_ckda_gb300 as ck
        silu = bool(s["case"].get("silu"))
        if op == "conv_fwd":
            y, hT = ck.conv_fwd(s["x"], s["w"], s["b"], h0=s["h0"], cu_seqlens=s["cu"], silu=silu)
            return {"y": y, "hT": hT}
        if op == "conv_bwd":
            dx, dw, db, dh0 = ck.conv_bwd(s["dy"], s["x"], s["w"], s["b"], h0=s["h0"], dhT=s["dhT"],
                                          cu_seqlens=s["cu"], silu=silu, store_dh0=s["h0"] is not None)
            out = {"dx": dx, "dw": dw, "db": db, "dh0": dh0}
        elif op == "conv_step":
            y = ck.conv_decode_step(s["x"], s["w"], s["state"], s["b"], silu=silu)
            return {"y": y, "state": s["state"]}
        elif op == "scan_fwd":
            y, hT = ck.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                h0=s["h0"], cu_seqlens=s["cu"])
            return {"y": y, "hT": hT}
        elif op == "scan_bwd":
            g = ck.scan_bwd(s["dy"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                            h0=s["h0"], dhT=s["dhT"], cu_seqlens=s["cu"], store_dh0=s["h0"] is not None)
            out = dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0"), g))
        elif op == "scan_step":
            y = ck.scan_decode_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
            return {"y": y, "state": s["state"]}
        elif op == "rms_fwd":
            y, h, rstd = ck.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS)
            out = {"y": y, "h": h if s["res"] is not None else None, "rstd": rstd}
        elif op == "rms_fwd8":
            y, scale, h, rstd = ck.rmsnorm_fwd8(s["x"], s["w"], residual=s["res"], eps=EPS, group=s["case"]["group"])
            out = {"y": y, "scale": scale, "h": h if s["res"] is not None else None, "rstd": rstd}
        else:
            dx, dw = ck.rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["w"], dh=s["dh"])
            out = {"dx": dx, "dw": dw}
        return {k: v for k, v in out.items() if v is not None}
    return PLAIN[op](s)


def work(case):
    """Inputs read once, outputs written once; the operations of the formulas, token by token."""
    size = {"bf16": 2, "fp32": 4}
    io, op = size[case["dtype"]], case["op"]
    if op.startswith("rms"):
        n, d, w, r = case["rows"], case["width"], size[case["wdtype"]], case["residual"]
        if op == "rms_bwd":
            return {"bytes": (3 + r) * n * d * io + 2 * d * w + 4 * n, "flops": 10 * n * d}
        out = n * d * io if op == "rms_fwd" else n * d + 4 * n * (d // case["group"] if case["group"] else 1)
        return {"bytes": (1 + 2 * r) * n * d * io + out + d * w + 4 * n, "flops": 6 * n * d}
    B, D = case["B"], case["D"]
    count = case.get("seqs") or B
    rows = B * case.get("T", 1)
    back, step = op.endswith("bwd"), op.endswith("step")
    h0 = 1 if step else case["h0"]
    if op.startswith("conv"):
        W, w = case["W"], size[case["wdtype"]]
        states = count * (W - 1) * D * io * (3 * h0 if back else 1 + h0)
        return {"bytes": rows * D * io * (3 if back else 2) + states + D * (W + case["bias"]) * w * (2 if back else 1),
                "flops": rows * D * (2 * W + 4) * (3 if back else 1)}
    N, G, z = case["N"], case["G"], case["z"]
    states = count * D * N * 4 * (3 * h0 if back else 1 + h0)
    weights = 4 * D * (N + 2)
    if back:   # x, dt, dy, (z) in, dx, ddt, (dz) out
        return {"bytes": rows * io * ((5 + 2 * z) * D + 4 * G * N) + states + 2 * weights, "flops": rows * D * (20 * N + 12)}
    return {"bytes": rows * io * ((3 + z) * D + 2 * G * N) + states + weights, "flops": rows * D * (7 * N + 8)}


# ------------------------------------------------------------------------------- 64-bit values
def _sequences(case, s):
    if s["cu"] is None:
        return [(slice(None), 0, case["T"], slice(None))]   # every batch row at once
    cu = s["cu"].tolist()
    return [(slice(0, 1), cu[i], cu[i + 1], slice(i, i + 1)) for i in range(len(cu) - 1)]


def _exact_conv(case, s):
    """Each sequence behind its state, the taps as a product along time; gradients by autograd."""
    W, back = case["W"], case["op"] == "conv_bwd"
    d = {n: s[n].double() for n in ("x", "w", "b", "h0", "dy", "dhT") if s.get(n) is not None}
    leaves = {n: d[n].clone().requires_grad_(back) for n in ("w", "b") if n in d}
    y, hT = torch.zeros_like(d["x"]), d["x"].new_zeros(case["seqs"] or case["B"], W - 1, case["D"])
    out = {"dx": torch.zeros_like(d["x"]), "dw": torch.zeros_like(d["w"])}
    if "b" in d:
        out["db"] = torch.zeros_like(d["b"])
    if "h0" in d:
        out["dh0"] = torch.zeros_like(d["h0"])
    for rows, t0, t1, n in _sequences(case, s):
        first = d["h0"][n] if "h0" in d else torch.zeros_like(hT[n])
        line = torch.cat([first, d["x"][rows, t0:t1]], 1)
        if not back:
            hT[n] = line[:, line.shape[1] - (W - 1):]
        if t1 == t0:
            if back and "h0" in d:
                out["dh0"][n] = d["dhT"][n]
            continue
        line.requires_grad_(back)
        p = torch.einsum("btdw,dw->btd", line.unfold(1, W, 1), leaves["w"])
        if "b" in d:
            p = p + leaves["b"]
        if case["silu"]:
            p = p / (1 + torch.exp(-p))
        if not back:
            y[rows, t0:t1] = p
            continue
        loss = (p * d["dy"][rows, t0:t1]).sum()
        if "dhT" in d:
            loss = loss + (line[:, line.shape[1] - (W - 1):] * d["dhT"][n]).sum()
        got = torch.autograd.grad(loss, [line, *leaves.values()])
        out["dx"][rows, t0:t1] = got[0][:, W - 1:]
        if "h0" in d:
            out["dh0"][n] = got[0][:, :W - 1]
        for name, g in zip(leaves, got[1:]):
            out["d" + name] += g
    return out if back else {"y": y, "hT": hT}


def _exact_scan(case, s):
    """Token after token, and for the gradients the same tokens from the last to the first."""
    B, T, D, N, G = (case[n] for n in ("B", "T", "D", "N", "G"))
    back = case["op"] == "scan_bwd"
    d = {n: s[n].double() for n in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0", "dy", "dhT") if s.get(n) is not None}
    raw = d["dt"] + d["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    A, per = d["A"], D // G
    wide = lambda v: v[..., :, None, :].expand(*v.shape[:-2], G, per, N).reshape(*v.shape[:-2], D, N)  # noqa: E731
    count = case["seqs"] or B
    hT = A.new_zeros(count, D, N)
    y = torch.zeros_like(d["x"])
    grads = {n: torch.zeros_like(d[k]) for n, k in (("dx", "x"), ("ddt", "x"), ("dB", "B"), ("dC", "C"), ("dA", "A"))}
    if "h0" in d:
        grads["dh0"] = torch.zeros_like(d["h0"])
    for rows, t0, t1, n in _sequences(case, s):
        h = d["h0"][n] if "h0" in d else torch.zeros_like(hT[n])
        seen = []
        for t in range(t0, t1):
            if back:
                seen.append(h)
            step = delta[rows, t, :, None]
            h = torch.exp(step * A) * h + step * d["x"][rows, t, :, None] * wide(d["B"][rows, t])
            y[rows, t] = torch.einsum("bdn,bdn->bd", h, wide(d["C"][rows, t]))
        hT[n] = h
        if not back:
            continue
        g = d["dhT"][n] if "dhT" in d else torch.zeros_like(h)
        for t in range(t1 - 1, t0 - 1, -1):
            old, step, x = seen.pop(), delta[rows, t, :, None], d["x"][rows, t, :, None]
            up = d["dy"][rows, t, :, None]
            if "z" in d:
                z = d["z"][rows, t, :, None]
                up = up * z / (1 + torch.exp(-z))
            Bw, Cw = wide(d["B"][rows, t]), wide(d["C"][rows, t])
            g = g + up * Cw
            decay = torch.exp(step * A)
            grads["dC"][rows, t] = (up * h).unflatten(1, (G, per)).sum(2)
            grads["dB"][rows, t] = (g * step * x).unflatten(1, (G, per)).sum(2)
            grads["dx"][rows, t] = (g * step * Bw).sum(-1) + d["D"] * up[..., 0]
            through = g * decay * old
            grads["ddt"][rows, t] = (through * A + g * x * Bw).sum(-1)
            grads["dA"] += (through * step).sum(0)
            g, h = g * decay, old
        if "h0" in d:
            grads["dh0"][n] = g
    y = y + d["D"] * d["x"]
    gate = d["z"] / (1 + torch.exp(-d["z"])) if "z" in d else 1.0
    if not back:
        return {"y": y * gate, "hT": hT}
    grads["dD"] = torch.einsum("btd,btd->d", d["dy"] * gate, d["x"])
    grads["ddt"] = grads["ddt"] / (1 + torch.exp(-raw))
    grads["ddt_bias"] = grads["ddt"].sum((0, 1))
    if "z" in d:
        p = 1 / (1 + torch.exp(-d["z"]))
        grads["dz"] = d["dy"] * y * p * (1 + d["z"] - d["z"] * p)
    return grads


def exact(case, seed):
    op = case["op"]
    if op in ("scan_fwd", "scan_bwd") and case["T"] * (3 if op == "scan_bwd" else 1) > 40000:
        return None
    s = prepare(case, seed)
    if op in ("conv_fwd", "conv_bwd"):
        return _exact_conv(case, s)
    if op in ("scan_fwd", "scan_bwd"):
        return _exact_scan(case, s)
    if op == "conv_step":
        line = torch.cat([s["state"], s["x"][:, None]], 1).double()
        p = torch.einsum("bwd,dw->bd", line, s["w"].double())
        if s["b"] is not None:
            p = p + s["b"].double()
        return {"y": p / (1 + torch.exp(-p)) if case["silu"] else p, "state": line[:, 1:]}
    if op == "scan_step":
        one = {**s, "h0": s["state"], **{n: (s[n][:, None] if s[n] is not None else None) for n in ("x", "dt", "B", "C", "z")}}
        got = _exact_scan({**case, "op": "scan_fwd", "T": 1, "seqs": 0}, one)
        return {"y": got["y"][:, 0], "state": got["hT"]}
    w = s["w"].double()
    if op == "rms_bwd":
        dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
        xh = s["h"].double() * rstd
        t = dy * w
        dx = (t - torch.einsum("nd,nd->n", t, xh)[:, None] / t.shape[1] * xh) * rstd
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": torch.einsum("nd,nd->d", dy, xh)}
    out, h = {}, s["x"].double()
    if s["res"] is not None:   # the norm is of the sum as it is stored
        out["h"] = h + s["res"].double()
        h = out["h"].to(s["x"].dtype).double()
    rstd = 1 / torch.sqrt(torch.einsum("nd,nd->n", h, h) / h.shape[1] + EPS)
    out["rstd"] = rstd
    out["y"] = h * rstd[:, None] * w
    if op == "rms_fwd8":
        y = out["y"].reshape(h.shape[0], -1, case["group"] or h.shape[1])
        scale = torch.linalg.vector_norm(y, math.inf, -1).clamp(min=LEAST) / E4M3_MAX
        out["y"] = (y / scale[..., None]).reshape(h.shape)
        out["scale"] = scale if case["group"] else scale[:, 0]
    return out
