"""Calls on a stream of the caller's choice: what a call allocates belongs to that stream."""
import contextlib

import pytest
import torch

BF, F32 = torch.bfloat16, torch.float32


def calls(ck, z):
    """Each call by name, on tensors of z(shape, dtype) that live as long as the calls."""
    lin = dict(q=z((1, 2, 8, 16), BF), k=z((1, 2, 8, 16), BF), v=z((1, 4, 8, 24), BF),
               g=z((1, 4, 8), F32))
    do = z((1, 4, 8, 24), BF)
    rule = [z(s, BF) for s in ((1, 2, 8, 64), (1, 2, 8, 64), (1, 2, 8, 128), (1, 2, 8, 64),
                               (1, 2, 8))]
    rule_do = z((1, 2, 8, 128), BF)
    x, one = z((4, 32), BF), z((4,), F32)
    kr, br = z((3, 32), BF), z((3,), BF)
    step = dict(q=z((1, 2, 16), BF), k=z((1, 2, 16), BF), v=z((1, 4, 24), BF), g=z((1, 4), F32))
    rule_step = [t[:, :, 0].contiguous() for t in rule]
    states = [z((1, 4, 16, 24), F32), z((1, 2, 64, 128), F32)]
    kept = []

    def state(i):  # updated in place, so each call has its own
        kept.append(states[i].clone())
        return kept[-1]
    return {
        "linear_fwd": lambda **s: ck.linear_fwd(**lin, **s),
        "linear_bwd": lambda **s: ck.linear_bwd(**lin, do=do, **s),
        "linear_decode_step": lambda **s: ck.linear_decode_step(**step, state=state(0), **s),
        "layernorm_fwd": lambda **s: ck.layernorm_fwd(x, **s),
        "layernorm_bwd": lambda **s: ck.layernorm_bwd(x, x, one, one, **s),
        "fwd": lambda **s: ck.fwd(*rule, **s),
        "fwd_raw": lambda **s: ck.fwd_raw(*rule, **s),
        "bwd": lambda **s: ck.bwd(*rule, do=rule_do, **s),
        "decode_step": lambda **s: ck.decode_step(*rule_step, state(1), **s),
        "prep": lambda **s: ck.prep(kr, kr, br, **s),
        "prep_bwd": lambda **s: ck.prep_bwd(kr, kr, br, kr, kr, br, **s),
    }


NAMES = ["linear_fwd", "linear_bwd", "linear_decode_step", "layernorm_fwd", "layernorm_bwd", "fwd",
         "fwd_raw", "bwd", "decode_step", "prep", "prep_bwd"]


class FakeStream:
    device, cuda_stream = torch.device("cuda", 0), 77


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream(name, monkeypatch):
    """On the CPU, with the library and torch's streams replaced: whatever the call allocates,
    it allocates with the given stream current, and launches there."""
    import gated_delta_rule_ckda_gb300 as ck

    class Lib:
        def __getattr__(self, fn):
            if fn.endswith("_bytes"):
                return lambda *a: 1024
            def launch(*a):
                launched.append((fn, current[-1]))
                return 0
            return launch

    side, here = FakeStream(), object()
    current, inside, launched = [here], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    run = calls(ck, lambda shape, dt: torch.zeros(shape, dtype=dt))[name]
    monkeypatch.setattr(ck, "lib", lambda: Lib())
    monkeypatch.setattr(ck, "_call", lambda fn, *a: fn())
    monkeypatch.setattr(ck, "_stream_handle", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    for n in ("empty", "empty_like"):
        def alloc(*a, _make=getattr(torch, n), **kw):
            inside.append(current[-1])
            return _make(*a, **kw)
        monkeypatch.setattr(torch, n, alloc)
    ck._bytes.cache_clear()
    try:
        run(stream=side)
    finally:
        ck._bytes.cache_clear()
    assert inside and all(s is side for s in inside)
    assert len(launched) == 1 and launched[0][1] is side


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_memory_used_again_on_the_callers_stream(name):
    """The stream is held up while the caller's stream takes and fills memory of every size that
    the call could have given back: the results are those of a call without a stream."""
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator(device="cuda").manual_seed(5)
    def z(shape, dt):
        return (0.3 * torch.randn(shape, generator=gen, device="cuda")).to(dt)
    run = calls(ck, z)[name]
    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = run(stream=side)
    for _ in range(3):
        for n in (256, 1024, 4096, 16384, 1 << 16, 1 << 18):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for a, b in zip(want if isinstance(want, tuple) else (want,),
                    got if isinstance(got, tuple) else (got,)):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.gpu
def test_workspaces_of_calls_on_two_streams():
    """Calls on a held-up stream, each of which gives the workspace of the one before it back."""
    import gated_delta_rule_ckda_gb300 as ck
    gen = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    x = [r(1, 4, 2000, 64).bfloat16() for _ in range(4)]
    g = -0.05 * r(1, 4, 2000).abs()
    rows, w = r(3000, 1000), r(1000)
    y, mean, rstd = ck.layernorm_fwd(rows, w)
    run = lambda **s: [*ck.linear_fwd(*x[:3], g, **s), *ck.linear_bwd(*x[:3], g, x[3], **s),
                       *ck.layernorm_bwd(y, rows, mean, rstd, w, **s)]
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    got = [run(stream=side) for _ in range(2)]
    for n in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24):
        for _ in range(4):
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    for outs in got:
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
