"""Linear attention with a scalar decay per head and layer norm in 64 bits, on
the CPU: the token-by-token recurrence and, for the gradients, the same
recurrence run backward.  Shares nothing with the CUDA path."""
import torch


def _head(q, k, v, g, h0, scale):
    H = torch.zeros(q.shape[1], v.shape[1], dtype=torch.float64) if h0 is None else h0.clone()
    o, states = [], [H]
    for t in range(q.shape[0]):
        H = torch.exp(g[t]) * H + torch.outer(k[t], v[t])
        states.append(H)
        o.append(scale * (q[t] @ H))
    return (torch.stack(o) if o else v.clone()), states


def _head_bwd(q, k, v, g, states, do, dhT, scale):
    G = torch.zeros_like(states[-1]) if dhT is None else dhT.clone()
    dq, dk, dv, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    for t in range(q.shape[0] - 1, -1, -1):
        G = G + scale * torch.outer(q[t], do[t])       # dL/dH_t
        dq[t] = scale * (states[t + 1] @ do[t])
        dk[t] = G @ v[t]
        dv[t] = k[t] @ G
        a = torch.exp(g[t])
        dg[t] = a * (states[t] * G).sum()
        G = a * G
    return dq, dk, dv, dg, G


def units(q, v, cu):
    """(batch row, first token, end, sequence) of each sequence."""
    if cu is None:
        return [(b, 0, q.shape[2], b) for b in range(q.shape[0])]
    c = [int(x) for x in cu]
    return [(0, c[i], c[i + 1], i) for i in range(len(c) - 1)]


def linear(q, k, v, g, h0=None, cu=None, scale=1.0, do=None, dhT=None):
    """(o, hT), or with do (o, hT, dq, dk, dv, dg, dh0); all float64 on the CPU."""
    d = lambda x: None if x is None else x.detach().cpu().double()
    per_head = g.dim() == 1
    q, k, v, g, h0, do, dhT = (d(x) for x in (q, k, v, g, h0, do, dhT))
    H, Hk = v.shape[1], q.shape[1]
    gf = g[None, :, None].expand(v.shape[:3]) if per_head else g
    seqs = units(q, v, cu)
    o = torch.zeros_like(v)
    hT = torch.zeros(len(seqs), H, q.shape[3], v.shape[3], dtype=torch.float64)
    grads = [torch.zeros_like(x) for x in (q, k, v, gf)] + [torch.zeros_like(hT)]
    for b, t0, t1, n in seqs:
        for h in range(H):
            x = (q[b, h * Hk // H, t0:t1], k[b, h * Hk // H, t0:t1], v[b, h, t0:t1],
                 gf[b, h, t0:t1])
            o[b, h, t0:t1], states = _head(*x, None if h0 is None else h0[n, h], scale)
            hT[n, h] = states[-1]
            if do is None:
                continue
            r = _head_bwd(*x, states, do[b, h, t0:t1], None if dhT is None else dhT[n, h], scale)
            grads[0][b, h * Hk // H, t0:t1] += r[0]
            grads[1][b, h * Hk // H, t0:t1] += r[1]
            grads[2][b, h, t0:t1] = r[2]
            grads[3][b, h, t0:t1] = r[3]
            grads[4][n, h] = r[4]
    if do is None:
        return o, hT
    if per_head:
        grads[3] = grads[3].sum((0, 2))
    return (o, hT, *grads)


def layer_norm(x, w, b, eps):
    x = x.detach().cpu().double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mean) * rstd
    if w is not None:
        y = y * w.detach().cpu().double()
    if b is not None:
        y = y + b.detach().cpu().double()
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_bwd(dy, x, mean, rstd, w):
    dy, x, mean, rstd = (t.detach().cpu().double() for t in (dy, x, mean, rstd))
    xh = (x - mean[..., None]) * rstd[..., None]
    t = dy if w is None else dy * w.detach().cpu().double()
    dx = rstd[..., None] * (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True))
    D = x.shape[-1]
    return dx, (dy * xh).reshape(-1, D).sum(0), dy.reshape(-1, D).sum(0)


# ------------------------------------------------------------------ tolerances
# u = eps / 2 of a type bounds one rounding's relative error; spread over a
# half step its rms is u / sqrt(3).
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def far(got, ref, size=0.0):
    """(rms of the error over s, largest |error| over max(|ref|, s)), s the rms of
    ref or, where that is more, the size of the terms that it is a difference of."""
    g, r = got.detach().cpu().double(), ref
    assert g.shape == r.shape, (g.shape, r.shape)
    if r.numel() == 0:
        return 0.0, 0.0
    assert torch.isfinite(g).all()
    e, s = (g - r).abs(), r.square().mean().sqrt().clamp(min=size)
    if s == 0:
        return (0.0, 0.0) if e.max() == 0 else (float("inf"), float("inf"))
    return float(e.square().mean().sqrt() / s), float((e / torch.clamp(r.abs(), min=s)).max())


def check(got, ref, rms_tol, what, size=0.0):
    """Root mean square within rms_tol and no element 8 times as far: errors
    are sums of many roundings, near normal, so the largest of 10^6 is within
    about 5 of their rms; an element in the tail of ref has larger terms."""
    rms, big = far(got, ref, size)
    assert rms <= rms_tol and big <= 8 * rms_tol, f"{what}: rms {rms:.2e}, max {big:.2e} (tolerance {rms_tol:.2e})"


def token_tol(io, T):
    """o, dq, dk, dv.  bf16: the operand that is rounded (a probability or the
    state) and the result, two roundings of rms u / sqrt 3 in quadrature, and a
    quarter on top for what they share.  fp32: a random walk over the tokens
    and the 128 columns of a readout."""
    if io == torch.bfloat16:
        return 1.25 * (2 / 3) ** 0.5 * U[io]
    return 4 * (T + 128) ** 0.5 * U[io]


def state_tol(io, T):
    """hT and dh0, fp32.  bf16 I/O: the decayed keys enter in two bf16 parts,
    what is left is u^2 at most; either way a walk over the tokens."""
    return (U[io] ** 2 if io == torch.bfloat16 else 0.0) + 4 * (T + 128) ** 0.5 * U[torch.float32]


def decay_tol(io, T):
    """dg, fp32: differences of sums that are up to 8 times what is left."""
    return 8 * state_tol(io, T)


def smoke_error(ck, dev):
    """Largest rms error over tolerance of a small forward, its gradients, a step
    and a layer norm with its gradients, times the bf16 tolerance of an output."""
    gen = torch.Generator().manual_seed(11)
    B, H, Hk, T, d, bf = 1, 4, 2, 200, 64, torch.bfloat16
    mk = lambda *s: torch.randn(*s, generator=gen)
    q, k, v, do = (mk(B, n, T, d).to(bf) for n in (Hk, Hk, H, H))
    g, h0, dhT = -0.1 * mk(B, H, T).abs(), mk(B, H, d, d), mk(B, H, d, d)
    c = [x.to(dev) for x in (q, k, v, g, do, h0, dhT)]
    o, hT = ck.linear_fwd(*c[:4], c[5], scale=0.125)
    grads = ck.linear_bwd(*c[:5], h0=c[5], dhT=c[6], scale=0.125)
    for call in (ck.linear_fwd, ck.linear_bwd):
        st = ck.fwd_status(call.last_workspace)
        if st != 0:
            raise RuntimeError(f"linear attention: device status {ck.STATUS.get(st, st)}")
    ref = linear(q, k, v, g, h0, None, 0.125, do, dhT)
    tol = [token_tol(bf, T), state_tol(bf, T), *[token_tol(bf, T)] * 3, decay_tol(bf, T),
           state_tol(bf, T)]
    worst = [far(a, r)[0] / t for a, r, t in zip((o, hT, *grads), ref, tol)]
    state, x = hT.clone(), [y[:, :, -1].contiguous() for y in c[:4]]
    so = ck.linear_decode_step(*x, state, scale=0.125)
    one = linear(*(y[:, :, -1:] for y in (q, k, v, g)), hT, None, 0.125)
    worst += [far(so, one[0][:, :, 0])[0] / token_tol(bf, 1), far(state, one[1])[0] / state_tol(bf, 1)]
    w, b = 1 + 0.1 * mk(d), mk(d)
    y, mean, rstd = ck.layernorm_fwd(c[2], w.to(dev), b.to(dev))
    n = layer_norm(v, w, b, 1e-5)
    dx, dw, db = ck.layernorm_bwd(c[4], c[2], mean, rstd, w.to(dev))
    m = layer_norm_bwd(do, v, n[1], n[2], w)
    worst += [far(y, n[0])[0] / token_tol(bf, 1), far(dx, m[0])[0] / token_tol(bf, 1),
              far(dw, m[1])[0] / state_tol(bf, T * H), far(db, m[2])[0] / state_tol(bf, T * H)]
    return max(worst) * token_tol(bf, 1)
