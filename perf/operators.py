"""Cases of the linear-attention and layer-norm operators: inputs, plain forms, calls, exact values.

Linear attention with a scalar decay for each head, state H in R^{dk x dv}:

    H_t = exp(g_t) H_{t-1} + k_t v_t^T,    o_t = H_t^T (scale q_t)

as a chunked forward over prompts, its backward pass, and one step on a resident state; and layer
norm, forward and backward.  `own` selects the framework's kernels (True) or the plain form in
elementary torch operations (False).
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64          # chunk of the plain form
EPS = 1e-5          # layer norm
MOST_TOKEN_HEADS = 4 * 32 * 8192
EXACT_PAIRS = 3.0e9   # (query, key) pairs that the 64-bit quadratic form takes on


def listed():
    return [
        # a short prompt of one user: latency counts
        dict(name="fwd_short", op="linear_fwd", B=1, H=16, Hk=16, T=37, dk=128, dv=128, dtype="bf16", h0=1, seqs=0),
        # the long training and prefill batch, state carried in
        dict(name="fwd_batch", op="linear_fwd", B=4, H=32, Hk=32, T=8192, dk=128, dv=128, dtype="bf16", h0=1, seqs=0),
        # one long document: fewer heads than SMs
        dict(name="fwd_long", op="linear_fwd", B=1, H=16, Hk=16, T=32768, dk=128, dv=128, dtype="bf16", h0=0, seqs=0),
        # prompts of ragged lengths packed together, keys and queries shared by pairs of heads
        dict(name="fwd_packed", op="linear_fwd", B=1, H=16, Hk=8, T=50021, dk=64, dv=128, dtype="bf16", h0=0, seqs=24),
        # training, the batch of the moderate forward workload
        dict(name="bwd_batch", op="linear_bwd", B=8, H=16, Hk=16, T=2048, dk=128, dv=128, dtype="bf16", h0=0, seqs=0),
        # fp32 gradients of a small odd model, keys shared by three heads, initial state trained
        dict(name="bwd_fp32", op="linear_bwd", B=2, H=6, Hk=2, T=1001, dk=48, dv=80, dtype="fp32", h0=1, seqs=0),
        # one user's next token
        dict(name="step_one", op="linear_step", B=1, H=16, Hk=16, dk=128, dv=128, dtype="bf16"),
        # the serving batch
        dict(name="step_batch", op="linear_step", B=256, H=32, Hk=32, dk=128, dv=128, dtype="bf16"),
        # the norm before a layer for a few tokens being decoded
        dict(name="norm_tokens", op="norm_fwd", rows=7, width=2048, dtype="bf16", wdtype="bf16"),
        # the norm of every head's output over a long batch
        dict(name="norm_heads", op="norm_fwd", rows=1048576, width=128, dtype="bf16", wdtype="fp32"),
        # a training batch at the width of 32 heads of 128
        dict(name="norm_bwd_wide", op="norm_bwd", rows=16384, width=4096, dtype="bf16", wdtype="fp32"),
        # fp32 rows of an odd width
        dict(name="norm_bwd_odd", op="norm_bwd", rows=2999, width=1031, dtype="fp32", wdtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "linear_bwd", "linear_step", "norm_fwd", "norm_bwd"])
    if op in ("norm_fwd", "norm_bwd"):
        width = _log_int(rng, 32, 16384)
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        rows = _log_int(rng, 1, min(1048576, 67108864 // width))
        return dict(op=op, rows=rows, width=width, dtype=dtype, wdtype=dtype if rng.random() < 0.5 else "fp32")
    group = rng.choice([1, 1, 2, 4])
    Hk = _log_int(rng, 1, 32 // group)
    H = Hk * group
    if op == "linear_step":
        dk, dv = (rng.choice([32, 64, 96, 128, 128, rng.randint(16, 128)]) for _ in range(2))
        return dict(op=op, B=_log_int(rng, 1, 8192 // H), H=H, Hk=Hk, dk=dk, dv=dv, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if rng.random() < 0.75:   # heads of eight channels each and more, in bf16
        dtype, most = "bf16", MOST_TOKEN_HEADS if op == "linear_fwd" else 8 * 16 * 2048
        dk, dv = (rng.choice([64, 128, 128, 8 * rng.randint(2, 16)]) for _ in range(2))
    else:                     # odd widths, or fp32
        dtype, most = rng.choice(["fp32", "fp32", "bf16"]), 2 * 16 * 2048
        dk, dv = (rng.choice([32, 64, rng.randint(5, 128)]) for _ in range(2))
    T = _log_int(rng, 1, min(32768, most // H))
    packed = rng.random() < 0.3
    B = 1 if packed else _log_int(rng, 1, max(1, min(64, most // (H * T))))
    return dict(op=op, B=B, H=H, Hk=Hk, T=T, dk=dk, dv=dv, dtype=dtype, h0=rng.randint(0, 1),
                seqs=_log_int(rng, 1, max(1, min(32, T // 4))) if packed else 0)


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

    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        n, d, wdt = case["rows"], case["width"], DTYPES[case["wdtype"]]
        # activations of a residual stream: an offset and a spread of their own in each row
        s["x"] = (randn(n, d) * (0.5 + torch.rand(n, 1, generator=gen, device=DEV)) + 0.3 * randn(n, 1)).to(dt)
        s["w"] = (1 + 0.1 * randn(d)).to(wdt)
        s["b"] = (0.1 * randn(d)).to(wdt)
        if case["op"] == "norm_bwd":
            x = s["x"].double()
            mean = x.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(-1) + EPS).rsqrt().float()
            s["dy"] = randn(n, d).to(dt)
        return s
    B, H, Hk, dk, dv = case["B"], case["H"], case["Hk"], case["dk"], case["dv"]
    s["scale"] = dk ** -0.5
    # decays from a head's own rate, long memory to short, and a gate of the token
    rate = torch.exp(torch.linspace(math.log(0.003), math.log(0.7), H, device=DEV))
    if case["op"] == "linear_step":
        s["q"], s["k"], s["v"] = randn(B, Hk, dk).to(dt), randn(B, Hk, dk).to(dt), randn(B, H, dv).to(dt)
        s["g"] = -rate * torch.nn.functional.softplus(randn(B, H))
        s["state"] = randn(B, H, dk, dv)
        return s
    T = case["T"]
    s["q"], s["k"], s["v"] = randn(B, Hk, T, dk).to(dt), randn(B, Hk, T, dk).to(dt), randn(B, H, T, dv).to(dt)
    s["g"] = -rate[:, None] * torch.nn.functional.softplus(randn(B, H, T))
    s["cu"] = None
    N = B
    if case["seqs"]:
        N = case["seqs"]
        off = _offsets(case, seed)
        s["cu"] = off.to(torch.int32).to(DEV)
        s["longest"] = int((off[1:] - off[:-1]).max())
    s["h0"] = randn(N, H, dk, dv) if case["h0"] else None
    if case["op"] == "linear_bwd":
        s["do"] = randn(B, H, T, dv).to(dt)
        s["dhT"] = randn(N, H, dk, dv) if case["h0"] else None
    return s


# -------------------------------------------------------------------------------- plain forms
def _chunks(x, n):
    """[B, H, T, ...] padded with zeros to n chunks: [B, H, n, CHUNK, ...]."""
    pad = n * CHUNK - x.shape[2]
    x = torch.cat([x, x.new_zeros(*x.shape[:2], pad, *x.shape[3:])], 2) if pad else x
    return x.reshape(*x.shape[:2], n, CHUNK, *x.shape[3:])


def _decays(g, n):
    """Of chunked log decays: from key to query inside a chunk, into a chunk, out of it, and between
    the states at chunk borders (n + 1 by n + 1).  The angles are summed in 64 bits."""
    L = _chunks(g.double(), n).cumsum(-1)
    i = torch.arange(CHUNK, device=g.device)
    late = i[:, None] >= i[None, :]
    inside = torch.where(late, L[..., :, None] - L[..., None, :], -math.inf).exp().float()
    total = L[..., -1:]
    M = torch.cat([torch.zeros_like(total[..., 0, :]), total[..., 0].cumsum(-1)], -1)
    c = torch.arange(n + 1, device=g.device)
    border = torch.where(c[:, None] >= c[None, :], M[..., :, None] - M[..., None, :], -math.inf).exp().float()
    return inside, L.exp().float()[..., None], (total - L).exp().float()[..., None], border


def _states(border, h0, F):
    """The states at chunk borders from the initial one and each chunk's own contribution."""
    B, H, n, dk, dv = F.shape
    first = h0 if h0 is not None else F.new_zeros(B, H, dk, dv)
    return (border @ torch.cat([first[:, :, None], F], 2).flatten(3)).view(B, H, n + 1, dk, dv)


def _plain_fwd(q, k, v, g, h0, scale):
    T, n = q.shape[2], -(-q.shape[2] // CHUNK)
    inside, into, out, border = _decays(g, n)
    q, k, v = _chunks(q * scale, n), _chunks(k, n), _chunks(v, n)
    Hs = _states(border, h0, (k * out).mT @ v)
    o = ((q @ k.mT) * inside) @ v + (q * into) @ Hs[:, :, :-1]
    return o.flatten(2, 3)[:, :, :T], Hs[:, :, -1]


def _plain_bwd(q, k, v, g, do, h0, dhT, scale):
    T, n = q.shape[2], -(-q.shape[2] // CHUNK)
    inside, into, out, border = _decays(g, n)
    q, k, v, do = _chunks(q, n), _chunks(k, n), _chunks(v, n), _chunks(do, n)
    Hs = _states(border, h0, (k * out).mT @ v)
    FG = (q * into * scale).mT @ do
    last = dhT if dhT is not None else FG.new_zeros(FG.shape[0], FG.shape[1], *FG.shape[3:])
    Gs = (border.mT @ torch.cat([FG, last[:, :, None]], 2).flatten(3)).view_as(Hs)
    G = Gs[:, :, 1:]
    A = (q @ k.mT) * inside * scale
    dA = (do @ v.mT) * inside * scale
    dq = dA @ k + (do @ Hs[:, :, :-1].mT) * into * scale
    dk = dA.mT @ q + (v @ G.mT) * out
    dv = A.mT @ do + (k @ G) * out
    x = (q.double() * dq).sum(-1) - (k.double() * dk).sum(-1)
    dg = x.flip(-1).cumsum(-1).flip(-1) + (Hs[:, :, 1:].double() * G).sum((-1, -2))[..., None]
    back = [t.flatten(2, 3)[:, :, :T] for t in (dq, dk, dv, dg)]
    return (*back, Gs[:, :, 0])


def _heads(x, H):
    return x.float().repeat_interleave(H // x.shape[1], 1)


def _shared(x, Hk):
    return x.unflatten(1, (Hk, x.shape[1] // Hk)).sum(2)


def _unpack(s):
    """Index of token t of sequence n in the packed axis, and whether it is one."""
    cu = s["cu"].long()
    t = torch.arange(s["longest"], device=cu.device)
    at = cu[:-1, None] + t[None, :]
    valid = at < cu[1:, None]
    return torch.where(valid, at, 0), valid


def _plain_linear(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    B, H, Hk, T, dk, dv = (c[n] for n in ("B", "H", "Hk", "T", "dk", "dv"))
    x = [_heads(s["q"], H), _heads(s["k"], H), s["v"].float(), s["g"]]
    back = c["op"] == "linear_bwd"
    if back:
        x.append(s["do"].float())
    if s["cu"] is not None:   # one padded row of the batch for each packed sequence
        at, valid = _unpack(s)
        fill = lambda t: torch.where(valid[:, None] if t.dim() == 3 else valid[:, None, :, None], t[0][:, at].transpose(0, 1), 0)  # noqa: E731
        x = [fill(t) for t in x]
    if back:
        *tok, dh0 = _plain_bwd(*x, s["h0"], s["dhT"], s["scale"])
    else:
        o, hT = _plain_fwd(*x, s["h0"], s["scale"])
        tok = [o]
    if s["cu"] is not None:
        where = at[valid]

        def pack(t):
            y = t.new_empty(1, H, T, *t.shape[3:])
            y[0, :, where] = t.transpose(0, 1)[:, valid]
            return y
        tok = [pack(t) for t in tok]
    if not back:
        return {"o": tok[0].to(dt), "hT": hT}
    dq, dk_, dv_, dg = tok
    out = {"dq": _shared(dq, Hk).to(dt), "dk": _shared(dk_, Hk).to(dt), "dv": dv_.to(dt), "dg": dg.float()}
    if s["h0"] is not None:
        out["dh0"] = dh0
    return out


def _plain_step(s):
    H, st = s["case"]["H"], s["state"]
    k, q = _heads(s["k"], H), _heads(s["q"], H) * s["scale"]
    st.mul_(s["g"].exp()[..., None, None]).add_(k[..., :, None] * s["v"].float()[..., None, :])
    o = (q[..., None, :] @ st)[..., 0, :]
    return {"o": o.to(s["v"].dtype), "state": st}


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    rstd = ((x - mean).square().mean(-1, keepdim=True) + EPS).rsqrt()
    y = (x - mean) * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    wdy = dy * s["w"].float()
    dx = rstd * (wdy - wdy.mean(-1, keepdim=True) - xh * (wdy * xh).mean(-1, keepdim=True))
    dw = (dy * xh).sum(0, dtype=torch.float64)
    db = dy.sum(0, dtype=torch.float64)
    return {"dx": dx.to(s["x"].dtype), "dw": dw.to(s["w"].dtype), "db": db.to(s["w"].dtype)}


# ------------------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import gated_delta_rule_ckda_gb300 as ck
        if op == "linear_fwd":
            o, hT = ck.linear_fwd(s["q"], s["k"], s["v"], s["g"], h0=s["h0"], cu_seqlens=s["cu"], scale=s["scale"])
            return {"o": o, "hT": hT}
        if op == "linear_bwd":
            dq, dk, dv, dg, dh0 = ck.linear_bwd(s["q"], s["k"], s["v"], s["g"], s["do"], h0=s["h0"], dhT=s["dhT"],
                                                cu_seqlens=s["cu"], scale=s["scale"], store_dh0=s["h0"] is not None)
            out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg}
            if dh0 is not None:
                out["dh0"] = dh0
            return out
        if op == "linear_step":
            o = ck.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"])
            return {"o": o, "state": s["state"]}
        if op == "norm_fwd":
            y, mean, rstd = ck.layernorm_fwd(s["x"], s["w"], s["b"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = ck.layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
        return {"dx": dx, "dw": dw, "db": db}
    if op in ("linear_fwd", "linear_bwd"):
        return _plain_linear(s)
    if op == "linear_step":
        return _plain_step(s)
    return _plain_norm_fwd(s) if op == "norm_fwd" else _plain_norm_bwd(s)


def work(case):
    """Inputs read once, outputs written once; the operations of the token-by-token recurrence (a
    state update and a readout for each token, three times that for the gradients)."""
    size = {"bf16": 2, "fp32": 4}
    io = size[case["dtype"]]
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        n, d, w = case["rows"], case["width"], size[case["wdtype"]]
        if op == "norm_fwd":
            return {"bytes": 2 * n * d * io + 2 * d * w + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * io + 3 * d * w + 8 * n, "flops": 14 * n * d}
    B, H, Hk, dk, dv = (case[n] for n in ("B", "H", "Hk", "dk", "dv"))
    if op == "linear_step":
        return {"bytes": 8 * B * H * dk * dv + B * (2 * Hk * dk + 2 * H * dv) * io + 4 * B * H, "flops": 5 * B * H * dk * dv}
    T, N = case["T"], case["seqs"] or B
    st = 4 * N * H * dk * dv
    if op == "linear_fwd":
        return {"bytes": B * T * ((2 * Hk * dk + 2 * H * dv) * io + 4 * H) + st * (1 + case["h0"]), "flops": 5 * B * H * T * dk * dv}
    return {"bytes": B * T * ((4 * Hk * dk + 3 * H * dv) * io + 8 * H) + 3 * st * case["h0"], "flops": 16 * B * H * T * dk * dv}


# ------------------------------------------------------------------------------- 64-bit values
def _exact_head(q, k, v, g, h0, scale):
    """One head of one sequence by the sum over all pairs: o_t = scale sum_{j<=t} exp(sum_{j<s<=t} g_s) (q_t.k_j) v_j."""
    T = q.shape[0]
    L = torch.cumsum(g, 0)
    gap = L[:, None] - L[None, :]
    gap = gap.masked_fill(torch.ones(T, T, dtype=torch.bool, device=g.device).triu(1), -math.inf)
    o = ((q @ k.T) * torch.exp(gap)) @ v
    left = torch.exp(L[-1] - L)[:, None]
    hT = (k * left).T @ v
    if h0 is not None:
        o = o + torch.exp(L)[:, None] * (q @ h0)
        hT = hT + torch.exp(L[-1]) * h0
    return o * scale, hT


def _exact_linear(case, s):
    B, H, Hk, T = case["B"], case["H"], case["Hk"], case["T"]
    back = case["op"] == "linear_bwd"
    cu = s["cu"].tolist() if s["cu"] is not None else None
    seqs = [(0, cu[i], cu[i + 1], i) for i in range(len(cu) - 1)] if cu else [(b, 0, T, b) for b in range(B)]
    if sum((t1 - t0) ** 2 for _, t0, t1, _ in seqs) * H * (4 if back else 1) > EXACT_PAIRS or max(t1 - t0 for _, t0, t1, _ in seqs) > 10000:
        return None
    d = {n: (s[n].double() if s.get(n) is not None else None) for n in ("q", "k", "v", "g", "h0", "do", "dhT")}
    zeros = lambda n: torch.zeros_like(d[n])  # noqa: E731
    if not back:
        out = {"o": zeros("v"), "hT": d["v"].new_zeros(len(seqs), H, case["dk"], case["dv"])}
    else:
        out = {"dq": zeros("q"), "dk": zeros("k"), "dv": zeros("v"), "dg": zeros("g")}
        if d["h0"] is not None:
            out["dh0"] = zeros("h0")
    for b, t0, t1, n in seqs:
        for h in range(H):
            hk = h * Hk // H
            ins = [d["q"][b, hk, t0:t1], d["k"][b, hk, t0:t1], d["v"][b, h, t0:t1], d["g"][b, h, t0:t1]]
            h0 = d["h0"][n, h] if d["h0"] is not None else None
            if t1 == t0:   # an empty sequence hands its state on
                if h0 is not None:
                    if back:
                        out["dh0"][n, h] = d["dhT"][n, h]
                    else:
                        out["hT"][n, h] = h0
                continue
            if not back:
                o, hT = _exact_head(*ins, h0, s["scale"])
                out["o"][b, h, t0:t1], out["hT"][n, h] = o, hT
                continue
            ins = [t.clone().requires_grad_() for t in ins] + ([h0.clone().requires_grad_()] if h0 is not None else [])
            o, hT = _exact_head(*ins[:4], ins[4] if h0 is not None else None, s["scale"])
            loss = (o * d["do"][b, h, t0:t1]).sum()
            if d["dhT"] is not None:
                loss = loss + (hT * d["dhT"][n, h]).sum()
            grads = torch.autograd.grad(loss, ins)
            out["dq"][b, hk, t0:t1] += grads[0]
            out["dk"][b, hk, t0:t1] += grads[1]
            out["dv"][b, h, t0:t1] = grads[2]
            out["dg"][b, h, t0:t1] = grads[3]
            if h0 is not None:
                out["dh0"][n, h] = grads[4]
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("linear_fwd", "linear_bwd"):
        return _exact_linear(case, s)
    if op == "linear_step":
        group = case["H"] // case["Hk"]
        k, q = (torch.stack([s[n][:, h // group] for h in range(case["H"])], 1).double() for n in ("k", "q"))
        st = torch.exp(s["g"].double())[:, :, None, None] * s["state"].double() + torch.einsum("bhi,bhj->bhij", k, s["v"].double())
        return {"o": s["scale"] * torch.einsum("bhi,bhij->bhj", q, st), "state": st}
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    if op == "norm_fwd":
        var, mean = torch.var_mean(x, -1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        return {"y": torch.addcmul(b, (x - mean[:, None]) * rstd[:, None], w), "mean": mean, "rstd": rstd}
    xh = (x - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
    dy = s["dy"].double()
    t = dy * w
    a, c = t.sum(-1) / x.shape[-1], torch.einsum("nd,nd->n", t, xh) / x.shape[-1]
    dx = (t - a[:, None] - xh * c[:, None]) * s["rstd"].double()[:, None]
    return {"dx": dx, "dw": torch.einsum("nd,nd->d", dy, xh), "db": dy.sum(0)}
