"""Short causal convolution, selective scan and RMS norm in 64 bits, on the CPU: token by
token, and for the gradients the same tokens run backward.  Shares nothing with the CUDA
path.  Gradients come with the size of the terms that they are sums of (the root of the sum
of their squares): where terms cancel, errors go by that."""
import torch

import linear_ref
from linear_ref import U, check  # noqa: F401

BF, F32 = torch.bfloat16, torch.float32


def d(t):
    return None if t is None else t.detach().cpu().double()


def sequences(x, cu):
    """(batch row, first token, end, sequence) of each sequence."""
    if cu is None:
        return [(b, 0, x.shape[1], b) for b in range(x.shape[0])]
    c = [int(v) for v in cu]
    return [(0, c[i], c[i + 1], i) for i in range(len(c) - 1)]


def act(p, silu):
    return p / (1 + torch.exp(-p)) if silu else p


def act_grad(p, silu):
    if not silu:
        return torch.ones_like(p)
    g = 1 / (1 + torch.exp(-p))
    return g * (1 + p * (1 - g))


# ----------------------------------------------------------------- short convolution
def conv(x, w, b=None, h0=None, cu=None, silu=True, dy=None, dhT=None):
    """(y, hT), or with dy (y, hT, dx, dw, db, dh0) and the gradients' sizes in a dict."""
    x, w, b, h0, dy, dhT = (d(t) for t in (x, w, b, h0, dy, dhT))
    D, W = w.shape
    seqs = sequences(x, cu)
    y, hT = torch.zeros_like(x), x.new_zeros(len(seqs), W - 1, D)
    out = {n: torch.zeros(s, dtype=torch.float64) for n, s in (
        ("dx", x.shape), ("dw", w.shape), ("db", (D,)), ("dh0", hT.shape))}
    sq = {n: torch.zeros_like(t) for n, t in out.items()}

    def add(name, at, v):
        out[name][at] += v
        sq[name][at] += v * v

    for row, t0, t1, n in seqs:
        line = torch.cat([hT[n] * 0 if h0 is None else h0[n], x[row, t0:t1]])
        hT[n] = line[len(line) - (W - 1):]
        for t in range(t1 - t0):
            p = (line[t:t + W].T * w).sum(1) + (0 if b is None else b)
            y[row, t0 + t] = act(p, silu)
            if dy is None:
                continue
            dp = dy[row, t0 + t] * act_grad(p, silu)
            add("db", slice(None), dp)
            for j in range(W):
                add("dw", (slice(None), j), dp * line[t + j])
                i = t + j - (W - 1)
                add("dx" if i >= 0 else "dh0", (row, t0 + i) if i >= 0 else (n, t + j), dp * w[:, j])
        if dy is not None and dhT is not None:
            for r in range(W - 1):
                i = t1 - t0 - (W - 1) + r
                add("dx" if i >= 0 else "dh0", (row, t0 + i) if i >= 0 else (n, i + W - 1), dhT[n, r])
    if dy is None:
        return y, hT
    return y, hT, out, {n: float(s.mean().sqrt()) if s.numel() else 0.0 for n, s in sq.items()}


# -------------------------------------------------------------------- selective scan
def scan(x, dt, A, B, C, D=None, z=None, bias=None, h0=None, cu=None, softplus=True, dy=None, dhT=None):
    """(y, hT), or with dy (y, hT, gradients, their sizes), B and C [.., G, N] or [.., N]."""
    x, dt, A, B, C, D, z, bias, h0, dy, dhT = (d(t) for t in (x, dt, A, B, C, D, z, bias, h0, dy, dhT))
    shape = B.shape
    if B.dim() == 3:
        B, C = B[:, :, None], C[:, :, None]
    width, N = A.shape
    G = B.shape[2]
    wide = lambda v: v.repeat_interleave(width // G, 0)  # noqa: E731
    seqs = sequences(x, cu)
    raw = dt if bias is None else dt + bias
    delta = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    inner, hT = torch.zeros_like(x), A.new_zeros(len(seqs), width, N)
    skip = A.new_zeros(width) if D is None else D
    out = {n: torch.zeros(s, dtype=torch.float64) for n, s in (
        ("dx", x.shape), ("ddt", x.shape), ("dA", A.shape), ("dB", B.shape), ("dC", B.shape),
        ("dD", (width,)), ("dz", x.shape), ("ddt_bias", (width,)), ("dh0", hT.shape))}
    sq = {n: torch.zeros_like(t) for n, t in out.items()}
    grouped = lambda v: v.unflatten(0, (G, width // G)).sum(1)  # noqa: E731
    gate = torch.ones_like(x) if z is None else act(z, True)
    for row, t0, t1, n in seqs:
        h = A.new_zeros(width, N) if h0 is None else h0[n]
        states = [h]
        for t in range(t0, t1):
            h = torch.exp(delta[row, t, :, None] * A) * h + (delta[row, t] * x[row, t])[:, None] * wide(B[row, t])
            states.append(h)
            inner[row, t] = (h * wide(C[row, t])).sum(1) + skip * x[row, t]
        hT[n] = h
        if dy is None:
            continue
        g = A.new_zeros(width, N) if dhT is None else dhT[n]
        for t in range(t1 - 1, t0 - 1, -1):
            now, old = states[t - t0 + 1], states[t - t0]
            up, step, xt, Bw, Cw = dy[row, t] * gate[row, t], delta[row, t], x[row, t], wide(B[row, t]), wide(C[row, t])
            g = g + up[:, None] * Cw
            a = torch.exp(step[:, None] * A)

            def put(name, terms, how):
                out[name][row, t] = how(terms)
                sq[name][row, t] = how(terms * terms)
            put("dC", up[:, None] * now, grouped)
            put("dB", g * (step * xt)[:, None], grouped)
            last = lambda v: v.sum(1)  # noqa: E731
            put("dx", torch.cat([g * Bw * step[:, None], (skip * up)[:, None]], 1), last)
            through = g * a * old
            slope = 1 / (1 + torch.exp(-raw[row, t])) if softplus else torch.ones_like(step)
            terms = torch.cat([through * A, g * Bw * xt[:, None]], 1) * slope[:, None]
            put("ddt", terms, last)
            out["ddt_bias"] += terms.sum(1)
            sq["ddt_bias"] += (terms * terms).sum(1)
            out["dA"] += through * step[:, None]
            sq["dA"] += (through * step[:, None]) ** 2
            out["dD"] += up * xt
            sq["dD"] += (up * xt) ** 2
            if z is not None:
                terms = torch.cat([now * Cw, (skip * xt)[:, None]], 1) * (dy[row, t] * act_grad(z[row, t], True))[:, None]
                put("dz", terms, last)
            g = g * a
        out["dh0"][n] = g
        sq["dh0"][n] = g * g
    if dy is None:
        return inner * gate, hT
    for n in ("dB", "dC"):
        out[n] = out[n].reshape(shape)
    return inner * gate, hT, out, {n: float(s.mean().sqrt()) if s.numel() else 0.0 for n, s in sq.items()}


# ------------------------------------------------------------------------- RMS norm
def rms(h, w, eps):
    """(y, rstd) of the stored sum."""
    h = d(h)
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    y = h * rstd[..., None]
    return (y if w is None else y * d(w)), rstd


def rms_bwd(dy, h, rstd, w, dh):
    dy, h, rstd, w, dh = (d(t) for t in (dy, h, rstd, w, dh))
    xh = h * rstd[..., None]
    t = dy if w is None else dy * w
    dx = rstd[..., None] * (t - xh * (t * xh).mean(-1, keepdim=True))
    size = float((rstd[..., None] * t).square().mean().sqrt()) if dx.numel() else 0.0
    return (dx if dh is None else dx + dh), (dy * xh).reshape(-1, h.shape[-1]).sum(0), size


# ------------------------------------------------------------------------ tolerances
# Root-mean-square errors, relative to the result's or its terms' rms; check() allows a
# single element 8 times that.  One rounding to a type moves each value by at most u of it,
# so the rms too: u / sqrt(3), as of many even errors, does not hold where a few values
# make up the rms.
def rounding(dt):
    return U[dt]


def conv_tol(dt, W):
    """fp32 between: W products and sums on terms up to 2 sqrt(W) / W of the whole each, the
    exponential (2 + 1.2 |p| units of 2^-23, |p| about 2), the quotient (2 of them), one on
    top: 2 W + 2 (2 + 2.4 + 2) + 1 units of u, 2 W + 14.  A slope of silu has two more products."""
    return (rounding(dt) if dt == BF else 0.0) + (2 * W + 14 + 4) * U[F32]


def scan_tol(dt, T, back=False):
    """The steps: softplus by an exponential, a quotient and eight more, 16 u.  A decay's
    exponent delta A: the step's 16 u, two products, 18 u in all times |delta A|, and the
    exponential itself 2 units of 2^-23, 4 u.  A state is a sum over about 1 / |delta A|
    tokens (T at most), through which the first add up to 18 u and the second, of changing
    sign, to 4 u sqrt(T); its own products and sums 2 u sqrt(T).  The readout, gate and skip
    16 u more.  A gradient is of two such factors, a state and a gradient's own."""
    t = (16 + 18 + 6 * T ** 0.5 + 16) * U[F32]
    return (rounding(dt) if dt == BF else 0.0) + (2 * t + 8 * U[F32] if back else t)


def sum_tol(dt, T, rows):
    """A gradient summed over `rows` tokens in fp32 behind that."""
    return (rounding(dt) if dt == BF else 0.0) + scan_tol(F32, T, True) + 2 * rows ** 0.5 * U[F32]


def rms_tol(dt, width):
    """fp32 sums of `width` squares and four products."""
    return (rounding(dt) if dt == BF else 0.0) + (8 + 2 * width ** 0.5) * U[F32]


far = linear_ref.far


def smoke_error(ck, dev):
    """Largest rms error over tolerance of a small convolution, scan and norm, their gradients
    and a step each, times the bf16 tolerance of an output of the norm."""
    gen = torch.Generator().manual_seed(17)
    B, T, D, W, N = 2, 70, 64, 4, 16
    mk = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, u, dt, z, dy, b, c = (mk(B, T, n).to(BF) for n in (D, D, D, D, D, N, N))
    w, A, skip, h0 = 1 + 0.1 * mk(D), -mk(D, N).abs(), mk(D), mk(B, D, N)
    cw, cb, c0 = 0.5 * mk(D, W), 0.1 * mk(D), mk(B, W - 1, D).to(BF)
    g = lambda *v: [t.to(dev) for t in v]  # noqa: E731
    worst = []

    def compare(got, want, tol):
        worst.append(far(got, want)[0] / tol)

    y, h, rstd = ck.rmsnorm_fwd(*g(x, w, u))
    compare(y, rms(h, w, 1e-5)[0], rms_tol(BF, D))
    dx, dw = ck.rmsnorm_bwd(dy.to(dev), h, rstd, w.to(dev), u.to(dev))
    want = rms_bwd(dy, h, rms(h, w, 1e-5)[1], w, u)
    compare(dx, want[0], 2 * rms_tol(BF, D))
    compare(dw, want[1], sum_tol(F32, T, B * T))

    y, hT = ck.conv_fwd(*g(x, cw, cb, c0))
    grads = ck.conv_bwd(*g(dy, x, cw, cb, c0))
    want = conv(x, cw, cb, c0, dy=dy)
    compare(y, want[0], conv_tol(BF, W))
    compare(hT, want[1], U[BF])
    for got, n in zip(grads, ("dx", "dw", "db", "dh0")):
        compare(got, want[2][n], 2 * conv_tol(got.dtype, W) + 2 * T ** 0.5 * U[F32])
    state = hT.clone()
    one = conv(x[:, -1:], cw, cb, hT)
    compare(ck.conv_decode_step(*g(x[:, -1], cw), state, cb.to(dev)), one[0][:, 0], conv_tol(BF, W))
    compare(state, one[1], U[BF])

    y, hT = ck.scan_fwd(*g(x, dt, A, b, c, skip, z), h0=h0.to(dev))
    grads = ck.scan_bwd(*g(dy, x, dt, A, b, c, skip, z), h0=h0.to(dev))
    want = scan(x, dt, A, b, c, skip, z, h0=h0, dy=dy)
    compare(y, want[0], scan_tol(BF, T))
    compare(hT, want[1], scan_tol(F32, T))
    for got, n in zip(grads, ("dx", "ddt", "dA", "dB", "dC", "dD", "dz", "", "dh0")):
        if n:
            compare(got, want[2][n], sum_tol(got.dtype, T, B * T))
    state = hT.clone()
    one = scan(*(t[:, -1:] for t in (x, dt)), A, *(t[:, -1:] for t in (b, c)), skip, z[:, -1:], h0=hT)
    got = ck.scan_decode_step(*g(x[:, -1], dt[:, -1], A, b[:, -1], c[:, -1]), state, *g(skip, z[:, -1]))
    compare(got, one[0][:, 0], scan_tol(BF, 1))
    compare(state, one[1], scan_tol(F32, 1))
    return max(worst) * rms_tol(BF, D)
