"""A layer of linear attention, trained and then served, on the library's calls.

    x + W_o norm_h(attend(norm(x) W_q, norm(x) W_k, norm(x) W_v, decay(norm(x))))

norm is layer norm over the channels, norm_h the same over each head's output,
attend the recurrence H_t = exp(g_t) H_{t-1} + k_t v_t^T, o_t = H_t^T q_t.

Training uses the autograd functions `layer_norm` and `linear_attention`: a
student learns to reproduce a fixed random layer.  Serving runs prompts of
different lengths in one packed call of `linear_fwd`, keeps each one's state,
and continues token by token with `linear_decode_step` in a CUDA graph; the
same tokens in one call over the whole sequences must give the same outputs.

    python examples/linear_attention.py --steps 60
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_ckda_gb300 as ck  # noqa: E402


class LinearAttentionLayer(torch.nn.Module):
    """width -> heads of dv channels reading key heads of dk channels."""

    def __init__(self, width, heads, key_heads, dk, dv, generator):
        super().__init__()
        self.heads, self.key_heads, self.dk, self.dv = heads, key_heads, dk, dv

        def weight(rows, cols):
            return torch.nn.Parameter(
                (torch.randn(rows, cols, generator=generator) / rows ** 0.5).cuda())

        self.wq, self.wk = weight(width, key_heads * dk), weight(width, key_heads * dk)
        self.wv, self.wo = weight(width, heads * dv), weight(heads * dv, width)
        self.wg = weight(width, heads)
        # decays from a few tokens to a few hundred
        self.bias_g = torch.nn.Parameter(torch.linspace(-6.0, -1.0, heads, device="cuda"))
        for name, n in (("norm", width), ("norm_h", dv)):
            setattr(self, name + "_w", torch.nn.Parameter(torch.ones(n, device="cuda")))
            setattr(self, name + "_b", torch.nn.Parameter(torch.zeros(n, device="cuda")))

    def _project(self, y):
        """q, k, v of y's leading shape and (heads, channels); g fp32."""
        lead, t = y.shape[:-1], torch.bfloat16
        q = (y @ self.wq.to(t)).view(*lead, self.key_heads, self.dk)
        k = (y @ self.wk.to(t)).view(*lead, self.key_heads, self.dk)
        v = (y @ self.wv.to(t)).view(*lead, self.heads, self.dv)
        g = -F.softplus((y @ self.wg.to(t)).float() + self.bias_g)
        return q, k, v, g

    def forward(self, x, h0=None, cu_seqlens=None):
        """x bf16 [B, T, width] -> (y, states of the sequences' ends)."""
        q, k, v, g = self._project(ck.layer_norm(x, self.norm_w, self.norm_b))
        q, k, v, g = (z.transpose(1, 2).contiguous() for z in (q, k, v, g))
        o, hT = ck.linear_attention(q, k, v, g, h0, cu_seqlens, scale=self.dk ** -0.5)
        o = ck.layer_norm(o, self.norm_h_w, self.norm_h_b)
        return x + o.transpose(1, 2).flatten(2) @ self.wo.to(x.dtype), hT

    @torch.no_grad()
    def step(self, x, state):
        """One token of each sequence: x [B, width], state updated in place."""
        y = ck.layernorm_fwd(x, self.norm_w, self.norm_b)[0]
        q, k, v, g = self._project(y)
        o = ck.linear_decode_step(q, k, v, g, state, scale=self.dk ** -0.5)
        o = ck.layernorm_fwd(o, self.norm_h_w, self.norm_h_b)[0]
        return x + o.flatten(1) @ self.wo.to(x.dtype)


def train(student, teacher, steps, batch, tokens, width, generator, lr=3e-3):
    """Losses of `steps` Adam steps towards the teacher's outputs."""
    opt = torch.optim.Adam(student.parameters(), lr=lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(batch, tokens, width, generator=generator).bfloat16().cuda()
        with torch.no_grad():
            want = teacher(x)[0] - x
        loss = (student(x)[0] - x - want).float().square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).cpu()


@torch.no_grad()
def serve(layer, lengths, new_tokens, width, generator):
    """Outputs of new_tokens tokens after prompts of the given lengths: token by
    token from the prompts' states, and in one packed call over everything."""
    seqs = [torch.randn(n + new_tokens, width, generator=generator).bfloat16().cuda()
            for n in lengths]

    def packed(parts):
        cu = [0]
        for p in parts:
            cu.append(cu[-1] + len(p))
        return layer(torch.cat(parts)[None], cu_seqlens=torch.tensor(
            cu, dtype=torch.int32, device="cuda"))

    _, state = packed([s[:n] for s, n in zip(seqs, lengths)])  # the prompts
    token = torch.empty(len(seqs), width, dtype=torch.bfloat16, device="cuda")
    start = state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(token.zero_(), state)  # (libraries set themselves up before a capture)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(token, state)
    state.copy_(start)
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
    p.add_argument("--tokens", type=int, default=500)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--heads", type=int, default=4)
    p.add_argument("--key-heads", type=int, default=2)
    p.add_argument("--dk", type=int, default=64)
    p.add_argument("--dv", type=int, default=64)
    p.add_argument("--prompts", type=int, nargs="+", default=[1, 37, 300, 129])
    p.add_argument("--new-tokens", type=int, default=20)
    a = p.parse_args(argv)
    gen = torch.Generator().manual_seed(1)
    shape = (a.width, a.heads, a.key_heads, a.dk, a.dv)
    teacher = LinearAttentionLayer(*shape, gen)
    student = LinearAttentionLayer(*shape, gen)
    losses = train(student, teacher, a.steps, a.batch, a.tokens, a.width, gen)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    got, want = serve(student, a.prompts, a.new_tokens, a.width, gen)
    err = ((got.float() - want.float()).norm() / want.float().norm()).item()
    print(f"served {len(a.prompts)} prompts, {a.new_tokens} tokens each: "
          f"{err:.2e} (relative, rms) from one call over the whole sequences")
    return losses, got, want


if __name__ == "__main__":
    main()
