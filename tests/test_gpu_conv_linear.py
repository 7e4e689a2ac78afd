"""Short convolution in front of q, k and v of linear attention: a projection's parts, tokens
as rows, convolved and brought to [B, H, T, d] for the attention; outputs against both
references, gradients by differences, and token by token from both states."""
import pytest
import torch

import linear_ref
import ssm_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ck():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_ckda_gb300 as ck
    ck.lib()
    return ck


def heads(t, H):
    """[B, T, H d] -> [B, H, T, d], copied."""
    return t.unflatten(-1, (H, -1)).transpose(1, 2).contiguous()


def layer(ck, qkv, w, g, off, H):
    """qkv [B, T, 3 H d] -> outputs, states of the attention and of the convolution."""
    c, conv = ck.short_conv(qkv, w, cu_seqlens=off)
    q, k, v = (heads(t, H) for t in c.chunk(3, -1))
    o, hT = ck.linear_attention(q, k, v, g, cu_seqlens=off)
    return o, hT, conv


@pytest.mark.parametrize("cu", [None, [0, 1, 40, 40, 131]])
@pytest.mark.parametrize("dt", [BF, F32])
def test_outputs(ck, dt, cu):
    gen = torch.Generator().manual_seed(1)
    B, T, H, d = (2, 90, 3, 64) if cu is None else (1, 131, 3, 64)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    qkv, w, g = r(B, T, 3 * H * d).to(dt), 0.3 * r(3 * H * d, 4), -0.1 * r(B, H, T).abs()
    off = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, hT, conv = layer(ck, qkv.cuda(), w.cuda(), g.cuda(), off, H)
    c, state = ref.conv(qkv, w, None, None, cu)
    assert torch.equal(conv.cpu().double(), state)
    got_c = ck.conv_fwd(qkv.cuda(), w.cuda(), cu_seqlens=off)[0]
    ref.check(got_c, c, ref.conv_tol(dt, 4), "convolution")
    # the attention is of the convolution's outputs as they are stored
    q, k, v = (heads(t, H).cpu() for t in got_c.chunk(3, -1))
    want, states = linear_ref.linear(q, k, v, g, None, cu)
    linear_ref.check(o, want, linear_ref.token_tol(dt, T), "o")
    linear_ref.check(hT, states, linear_ref.state_tol(dt, T), "hT")


def test_gradients_by_differences(ck):
    """In fp32 along a random direction of unit length: over a step of h the loss has errors of a
    few 2^-24 of its terms over h, and a third derivative's term of h^2 of them."""
    gen = torch.Generator().manual_seed(2)
    B, T, H, d, h = 1, 60, 2, 16, 1e-2
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    off = torch.tensor([0, 25, 60], dtype=torch.int32, device="cuda")
    leaves = [r(B, T, 3 * H * d).requires_grad_(), (0.3 * r(3 * H * d, 4)).requires_grad_(),
              (-0.1 * r(B, H, T).abs()).requires_grad_()]
    ro, rh, rc = r(B, H, T, d), r(2, H, d, d), r(2, 3, 3 * H * d)

    def loss(qkv, w, g):
        o, hT, conv = layer(ck, qkv, w, g, off, H)
        return sum((p.double() * q.double()).sum() for p, q in ((o, ro), (hT, rh), (conv, rc)))

    def terms(qkv, w, g):
        o, hT, conv = layer(ck, qkv, w, g, off, H)
        return sum((p.double() * q.double()).square().sum() for p, q in ((o, ro), (hT, rh), (conv, rc))).sqrt().item()
    grads = torch.autograd.grad(loss(*leaves), leaves)
    with torch.no_grad():
        scale = terms(*leaves)
    for i, gr in enumerate(grads):
        u = r(*leaves[i].shape)
        u /= u.norm()
        with torch.no_grad():
            up = [t if j != i else t + h * u for j, t in enumerate(leaves)]
            dn = [t if j != i else t - h * u for j, t in enumerate(leaves)]
            diff = ((loss(*up) - loss(*dn)) / (2 * h)).item()
        got = (gr.double() * u.double()).sum().item()
        assert abs(got - diff) <= 4 * scale * (16 * 2 ** -24 / h + h * h), (i, got, diff)


def test_steps_continue_a_prompt(ck):
    gen = torch.Generator().manual_seed(3)
    B, T, H, d, cut = 3, 30, 4, 64, 21
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    qkv, w, g = r(B, T, 3 * H * d), 0.3 * r(3 * H * d, 4), -0.1 * r(B, H, T).abs()
    o, hT, conv = layer(ck, qkv, w, g, None, H)
    _, state, taps = layer(ck, qkv[:, :cut].contiguous(), w, g[..., :cut].contiguous(), None, H)
    for t in range(cut, T):
        c = ck.conv_decode_step(qkv[:, t], w, taps)
        q, k, v = (p.unflatten(-1, (H, d)).contiguous() for p in c.chunk(3, -1))
        y = ck.linear_decode_step(q, k, v, g[..., t].contiguous(), state)
        linear_ref.check(y, o[:, :, t].double().cpu(), 2 * linear_ref.token_tol(F32, T), f"token {t}")
    assert torch.equal(taps, conv)
    linear_ref.check(state, hT.double().cpu(), 2 * linear_ref.state_tol(F32, T), "state")
