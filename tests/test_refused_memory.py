"""Memory that no kernel may be given is refused by the binding, on the host: tensors that are
not on a GPU, and a workspace on another device than they are or not in one run.  No call here
reaches the library's launches."""
import pytest
import torch

from test_streams import NAMES, calls

# (the inputs lie on the CPU, so "another device" is the meta device)
WITH_WORKSPACE = ["linear_fwd", "linear_bwd", "layernorm_bwd", "fwd", "fwd_raw", "bwd"]


@pytest.fixture
def run(monkeypatch):
    import gated_delta_rule_ckda_gb300 as ck

    class Lib:
        def __getattr__(self, fn):
            def called(*a):
                assert fn.endswith("_bytes"), f"{fn} was launched"
                return 1024
            called.argtypes = ()
            return called
    monkeypatch.setattr(ck, "lib", lambda: Lib())
    ck._bytes.cache_clear()
    yield calls(ck, lambda shape, dt: torch.zeros(shape, dtype=dt))
    ck._bytes.cache_clear()


@pytest.mark.parametrize("name", NAMES)
def test_tensors_in_host_memory(run, name):
    with pytest.raises(ValueError, match="on cpu, expected CUDA"):
        run[name]()


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspace_elsewhere(run, name):
    with pytest.raises(ValueError, match="workspace: on meta"):
        run[name](workspace=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
    with pytest.raises(ValueError, match="workspace: must be contiguous"):
        run[name](workspace=torch.empty(1 << 20, dtype=torch.uint8)[::2])


def test_outputs_of_the_older_calls(run):
    import gated_delta_rule_ckda_gb300 as ck
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    step = [z(1, 2, 128) for _ in range(4)] + [z(1, 2), torch.zeros(1, 2, 128, 128)]
    with pytest.raises(ValueError, match="o: shape"):
        ck.decode_step_raw(*step, o=z(1, 2, 64))
    rule = [z(1, 2, 8, 64), z(1, 2, 8, 64), z(1, 2, 8, 128), z(1, 2, 8, 64), z(1, 2, 8)]
    for bad in (dict(o=z(1, 2, 8, 64)), dict(hT=torch.zeros(1, 2, 64, 64)),
                dict(h0=torch.zeros(2, 2, 64, 128))):
        with pytest.raises(ValueError, match="shape"):
            ck.fwd_noalloc(*rule, **bad)
