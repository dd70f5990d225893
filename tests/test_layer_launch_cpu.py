"""The library's host side over a runtime of our own: a launch that fails ends the call, and
device properties are those of the device."""
import ctypes

import pytest

from kda_gated_delta_gb300 import binding
from tests import fake_runtime

FAKE = 1 << 20


@pytest.fixture
def L(tmp_path):
    return fake_runtime.load(tmp_path)


def params(H=4, P=64, N=128, G=1, io=1):
    return binding.SsmParams(H, P, N, G, io, 0, io, 20.0)


def prefill(L, p, n, T, fail=-1):
    """(status, launches tried) of a call whose launch number `fail` fails."""
    L.fake_reset(fail)
    i64, P = ctypes.c_int64, ctypes.c_void_p
    rc = L.kda_ssm_prefill(ctypes.byref(p), P(FAKE), i64(p.num_heads * p.head_dim), P(FAKE), i64(p.num_heads), P(FAKE), i64(p.num_groups * p.state_dim),
                           P(FAKE), i64(p.num_groups * p.state_dim), P(FAKE), None, None, P(FAKE), n, i64(T), P(FAKE), i64(8), P(FAKE), P(FAKE), P(FAKE),
                           ctypes.c_size_t(1 << 40), None)
    return rc, L.fake_launches()


# one long prompt in segments; many short ones beside a longer one; packed prompts; fp32 in segments and whole
@pytest.mark.parametrize("p,n,T,launches", [(params(), 1, 20000, 4), (params(), 40, 600, 3), (params(), 4, 2000, 2), (params(io=0), 1, 20000, 4),
                                            (params(io=0), 3, 500, 1)], ids=["segments", "short", "chunks", "fp32 segments", "fp32"])
def test_a_failed_launch_ends_the_call(L, p, n, T, launches):
    assert prefill(L, p, n, T) == (0, launches)
    for k in range(launches):
        assert prefill(L, p, n, T, fail=k) == (-5, k + 1)


def test_number_of_sms(L):
    """A query that fails leaves no number behind, and each device has its own."""
    size = L.kda_ssm_prefill_workspace_size
    size.restype = ctypes.c_size_t
    p, n, T = params(H=1), 1, ctypes.c_int64(1 << 20)

    def need(dev, sms, silent=0):
        L.fake_device(dev, sms)
        L.fake_silent(silent)
        return size(ctypes.byref(p), n, T)

    other = need(3, 40)
    assert need(1, 152, silent=100) == need(2, 148) != need(4, 152)
    assert need(1, 152) == need(4, 152)
    assert need(3, 40) == other != need(1, 152)


def test_a_check_makes_one_copy(L):
    """However many translation units have an error word."""
    L.fake_reset(-1)
    code = ctypes.c_int32(7)
    assert L.kda_check_device_errors(None, ctypes.byref(code)) == 0 and code.value == 0
    assert L.fake_copies() == 1
    L.fake_reset(0)
    assert L.kda_check_device_errors(None, ctypes.byref(code)) == -5 and code.value == 0 and L.fake_copies() == 0
