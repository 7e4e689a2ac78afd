"""Blocks of a selective state space model, trained and then served, on the library's calls.

Each block, on a residual stream h:

    h, y = h + u, norm(h + u)                      rms_norm with the residual's addition
    x, z = y W_in                                  (parts of one projection)
    x = silu(conv(x))                              short_conv
    r, B, C = x W_x,   dt = r W_dt
    u = scan(x, dt, A, B, C, D, z) W_out           selective_scan

Training uses the autograd functions: a student learns to reproduce fixed random blocks.
Serving runs prompts of different lengths in one packed call of each operator, keeps every
prompt's two states a block, and continues token by token in a CUDA graph with
`conv_decode_step` and `scan_decode_step`; the same tokens in one call over the whole
sequences must give the same outputs.  With --eight-bits, the served blocks' norms put out
8 bits with a scale for each row (rmsnorm_fwd8), for the projection behind them.

    python examples/state_space.py --steps 60
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_ckda_gb300 as ck  # noqa: E402

BF = torch.bfloat16


class StateSpaceBlock(torch.nn.Module):
    """width -> inner channels of `states` states, convolved over `taps` tokens."""

    def __init__(self, width, inner, states, taps, rank, generator):
        super().__init__()
        self.inner, self.states, self.taps, self.rank = inner, states, taps, rank

        def weight(rows, cols, scale=1.0):
            return torch.nn.Parameter(
                (scale * torch.randn(rows, cols, generator=generator) / rows ** 0.5).cuda())

        self.norm = torch.nn.Parameter(torch.ones(width, device="cuda"))
        self.w_in, self.w_out = weight(width, 2 * inner), weight(inner, width)
        self.w_x, self.w_dt = weight(inner, rank + 2 * states), weight(rank, inner)
        self.conv_w = torch.nn.Parameter((torch.randn(inner, taps, generator=generator) / taps ** 0.5).cuda())
        self.conv_b = torch.nn.Parameter(torch.zeros(inner, device="cuda"))
        # steps from 0.001 to 0.1, decay rates of 1, 2, 3, ...
        step = torch.exp(math.log(0.001) + math.log(100.0) * torch.rand(inner, generator=generator))
        self.dt_bias = torch.nn.Parameter((step + torch.log(-torch.expm1(-step))).cuda())
        self.log_a = torch.nn.Parameter(torch.arange(1.0, states + 1).log().repeat(inner, 1).cuda())
        self.skip = torch.nn.Parameter(torch.ones(inner, device="cuda"))

    def _steps(self, x):
        """dt, B, C of x's tokens; B and C are parts of one projection."""
        p = x @ self.w_x.to(BF)
        dt = p[..., :self.rank] @ self.w_dt.to(BF)
        return dt, p[..., self.rank:self.rank + self.states], p[..., self.rank + self.states:]

    def _in(self, u, h, eight):
        """(x and z in one, new residual stream)."""
        if eight:
            y, scale, h, _ = ck.rmsnorm_fwd8(u, self.norm, residual=h)
            return (y.to(BF) @ self.w_in.to(BF)) * scale[..., None].to(BF), h
        y, h = ck.rms_norm(u, self.norm, h)
        return y @ self.w_in.to(BF), h

    def forward(self, u, h, cu_seqlens=None, eight=False):
        """u, h bf16 [B, T, width] -> (u, h, (convolution's state, scan's state))."""
        xz, h = self._in(u, h, eight)
        x, conv = ck.short_conv(xz[..., :self.inner], self.conv_w, self.conv_b, cu_seqlens=cu_seqlens)
        dt, b, c = self._steps(x)
        y, scan = ck.selective_scan(x, dt, -self.log_a.exp(), b, c, self.skip, xz[..., self.inner:],
                                    self.dt_bias, cu_seqlens=cu_seqlens)
        return y @ self.w_out.to(BF), h, (conv, scan)

    @torch.no_grad()
    def step(self, u, h, state, eight=False):
        """One token of each sequence: u, h [B, width], both states updated in place."""
        conv, scan = state
        xz, h = self._in(u, h, eight)
        x = ck.conv_decode_step(xz[..., :self.inner], self.conv_w, conv, self.conv_b)
        dt, b, c = self._steps(x)
        y = ck.scan_decode_step(x, dt, -self.log_a.exp(), b, c, scan, self.skip, xz[..., self.inner:],
                                self.dt_bias)
        return y @ self.w_out.to(BF), h


class Blocks(torch.nn.Module):
    def __init__(self, count, *shape):
        super().__init__()
        self.blocks = torch.nn.ModuleList(StateSpaceBlock(*shape) for _ in range(count))

    def forward(self, x, cu_seqlens=None, eight=False):
        u, h, states = torch.zeros_like(x), x, []
        for block in self.blocks:
            u, h, state = block(u, h, cu_seqlens, eight)
            states.append(state)
        return h + u, states

    def step(self, x, states, eight=False):
        u, h = torch.zeros_like(x), x
        for block, state in zip(self.blocks, states):
            u, h = block.step(u, h, state, eight)
        return h + u


def train(student, teacher, steps, batch, tokens, width, generator, lr=3e-3):
    """Losses of `steps` Adam steps towards the teacher's outputs."""
    opt = torch.optim.Adam(student.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(batch, tokens, width, generator=generator).to(BF).cuda()
        with torch.no_grad():
            want = teacher(x)[0]
        loss = (student(x)[0] - want).float().square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).cpu()


@torch.no_grad()
def serve(model, lengths, new_tokens, width, generator, eight=False):
    """Outputs of new_tokens tokens after prompts of the given lengths: token by token from
    the prompts' states, and in one packed call over everything."""
    seqs = [torch.randn(n + new_tokens, width, generator=generator).to(BF).cuda() for n in lengths]

    def packed(parts):
        cu = [0]
        for p in parts:
            cu.append(cu[-1] + len(p))
        return model(torch.cat(parts)[None], torch.tensor(cu, dtype=torch.int32, device="cuda"), eight)

    _, states = packed([s[:n] for s, n in zip(seqs, lengths)])  # the prompts
    start = [tuple(t.clone() for t in s) for s in states]
    token = torch.zeros(len(seqs), width, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.step(token, states, eight)  # (libraries set themselves up before a capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model.step(token, states, eight)
    for state, old in zip(states, start):
        for t, o in zip(state, old):
            t.copy_(o)
    outs = []
    for t in range(new_tokens):
        token.copy_(torch.stack([s[n + t] for s, n in zip(seqs, lengths)]))
        graph.replay()
        outs.append(out.clone())
    whole, _ = packed(seqs)
    ends, at = [], 0
    for s in seqs:
        at += len(s)
        ends.append(whole[0, at - new_tokens:at])
    return torch.stack(outs, 1), torch.stack(ends)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--tokens", type=int, default=300)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--inner", type=int, default=512)
    p.add_argument("--states", type=int, default=16)
    p.add_argument("--taps", type=int, default=4)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--blocks", type=int, default=2)
    p.add_argument("--prompts", type=int, nargs="+", default=[1, 37, 300, 129])
    p.add_argument("--new-tokens", type=int, default=20)
    p.add_argument("--eight-bits", action="store_true")
    a = p.parse_args(argv)
    gen = torch.Generator().manual_seed(1)
    shape = (a.width, a.inner, a.states, a.taps, a.rank, gen)
    teacher, student = Blocks(a.blocks, *shape), Blocks(a.blocks, *shape)
    losses = train(student, teacher, a.steps, a.batch, a.tokens, a.width, gen)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    got, want = serve(student, a.prompts, a.new_tokens, a.width, gen, a.eight_bits)
    err = ((got.float() - want.float()).norm() / want.float().norm()).item()
    print(f"served {len(a.prompts)} prompts, {a.new_tokens} tokens each: "
          f"{err:.2e} (relative, rms) from one call over the whole sequences")
    return losses, got, want


if __name__ == "__main__":
    main()
