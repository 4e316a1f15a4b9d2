"""Waits inside a kernel that run out: after the limit the threads go on, the
kernel ends, and the host reads a status once; the context stays usable."""
import ctypes
import os
import subprocess
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
OK, TIMEOUT = 0, 8


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from linear_recurrence_scan_gb300 import build
    so = tmp_path_factory.mktemp("waits") / "libwaits.so"
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-shared", os.path.join(HERE, "wait_limit.cu"), "-o", str(so)],
                   check=True, timeout=300)
    return ctypes.CDLL(str(so))


# kind of wait_limit.cu -> the threads' answers, the warps', the status (None: not asked)
CASES = {0: (0, 0, TIMEOUT), 1: (1, 1, OK), 2: (1, 1, TIMEOUT), 3: (0, 0, TIMEOUT), 4: (None, 0, TIMEOUT)}


@pytest.mark.parametrize("kind", CASES)
def test_waits(lib, kind):
    threads, warps = (torch.full((64,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    again = ctypes.c_int(-1)
    torch.cuda.synchronize()
    start = time.time()
    status = lib.run_waits(kind, ctypes.c_void_p(threads.data_ptr()), ctypes.c_void_p(warps.data_ptr()), ctypes.byref(again), None)
    assert time.time() - start < 2
    each, together, want = CASES[kind]
    assert (status, again.value) == (want, OK)
    asked = slice(32, 64) if kind == 3 else slice(0, 64)
    if each is None:
        each = (torch.arange(64, device="cuda") + 1) % 2   # the phase has come for even lanes
    assert (threads[asked] == each).all() and (warps[asked] == together).all()
    if kind == 3:
        assert (threads[:32] == 7).all() and (warps[:32] == 7).all()
    assert torch.ones(1000, device="cuda").sum().item() == 1000
