"""The bounded wait of a whole warp (csrc/chunk_common.cuh: short_wait): it returns at once when the phase is complete, gives up
after about the library's half second when nothing arrives (it counts tries, whose length is the hardware's: from half of
that to four times it), and early when another role has given up. The library's kernels are never
made to time out: tests/native/short_wait_probe.cu compiles the wait into a one-warp kernel of its own."""
import ctypes

import pytest
import torch

import paged_kv_cache_83_gb300 as pa
from tests.native import build_wait_probe

pytestmark = pytest.mark.gpu

LIMIT_NS = 500_000_000


@pytest.fixture(scope="module")
def probe():
    lib = ctypes.CDLL(str(build_wait_probe("short_wait_probe")))
    lib.pa_test_short_wait_probe.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    lib.pa_test_short_wait_probe.restype = ctypes.c_int
    return lib


def _run(probe, arrive, abort=False):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    elapsed = torch.zeros(1, dtype=torch.int64, device="cuda")
    assert probe.pa_test_short_wait_probe(err.data_ptr(), int(arrive), int(abort), elapsed.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    return int(err), int(elapsed)


def test_a_phase_that_is_complete(probe):
    err, ns = _run(probe, arrive=True)
    assert err == 0 and ns < LIMIT_NS // 10


def test_nothing_arrives(probe):
    err, ns = _run(probe, arrive=False)
    assert err == pa.PA_DEVERR_TIMEOUT and LIMIT_NS // 2 <= ns < 4 * LIMIT_NS
    assert _run(probe, arrive=True)[0] == 0  # the context is as usable as before


def test_another_role_gave_up(probe):
    err, ns = _run(probe, arrive=False, abort=True)
    assert err == pa.PA_DEVERR_TIMEOUT and ns < LIMIT_NS // 2
