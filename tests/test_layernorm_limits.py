"""The widest rows that layer norm takes: the kernels count columns in 32 bits, in steps of 1024
and 32 past a row's end.  On the host: nothing here reaches the GPU."""
import ctypes

import pytest

vp = ctypes.c_void_p
UNS = 2


@pytest.fixture(scope="module")
def L():
    from gated_delta_rule_ckda_gb300 import build
    build.build()
    import gated_delta_rule_ckda_gb300 as ck
    return ck.lib()


@pytest.mark.parametrize("width", [(1 << 30) + 1, (1 << 31) - 1025, (1 << 31) - 1])
def test_rows_wider_than_the_counters(L, width):
    assert L.ckda_layernorm_fwd(*[vp(256)] * 6, 1, width, 1, 0, 1e-5, None) == UNS
    assert L.ckda_layernorm_bwd(*[vp(256)] * 8, 1, width, 1, 0, vp(256), 1 << 62, None) == UNS


def test_counters_hold_up_to_the_limit():
    """A thread's column goes up to a step past the row's end, a block's up to 31 past."""
    width = 1 << 30
    assert width + 1024 < 1 << 31 and (width + 31) // 32 * 32 < 1 << 31
