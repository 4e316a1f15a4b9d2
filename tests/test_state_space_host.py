"""The state-space layer's host side without a GPU: workspace queries of
empty calls, refusals."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scan_gb300 import _native, build
    build.build()
    return _native.lib()


EMPTY = """
from linear_recurrence_scan_gb300 import _native, state_space as ss
lib = _native.lib()
for N, T, D in ((0, 600, 64), (2, 600, 0), (0, 600, 0), (2, 0, 64), (0, 100000, 4096), (1, 100000, 0)):
    for dtype in (0, 1):
        a = ss._SCAN_ARGS.pack(N, T, D, 16, dtype, 1, *[256, T * D, D] * 3, *[256, T * 16, 16] * 2, 256, 0, 0, 0, 0, 0)
        c = ss._CONV_ARGS.pack(N, T, D, 4, dtype, 1, 256, T * D, D, 256, 0, 0, 0, 0)
        sizes = [lib.rlscan_selective_scan_workspace_bytes(a), lib.rlscan_selective_scan_backward_workspace_bytes(a),
                 lib.rlscan_causal_conv_backward_workspace_bytes(c), lib.rlscan_add_rms_norm_backward_workspace_bytes(N * T, D)]
        assert not any(sizes) or T == 0, (N, T, D, sizes)   # without tokens A's gradient is still a sum of parts
print("done")
"""


def test_empty_calls_need_no_workspace(lib):
    """No rows or no channels: the queries answer 0 (in a child: an integer division by zero ends the process)."""
    r = subprocess.run([sys.executable, "-c", EMPTY], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, (r.returncode, r.stderr[-2000:])


def test_forward_mode_is_refused():
    """Dual tensors are refused before anything else is looked at; others pass inside a dual level."""
    import torch
    import torch.autograd.forward_ad as fwd
    import linear_recurrence_scan_gb300 as rl
    x, bc, A, w = torch.zeros(2, 4, 8), torch.zeros(2, 4, 3), torch.zeros(8, 3), torch.zeros(8, 4)
    state, marks = torch.zeros(2, 8, 3), torch.zeros(2, 1, 8, 3)
    calls = [lambda f: rl.selective_scan(f(x), x, A, bc, bc), lambda f: rl.selective_scan(x, x, A, f(bc), bc),
             lambda f: rl.selective_scan(x, x, A, bc, bc, initial_state=f(state)),
             lambda f: rl.selective_scan_backward(x, x, x, f(A), bc, bc, marks),
             lambda f: rl.selective_scan_step(state, x[:, 0], f(x[:, 0]), A, bc[:, 0], bc[:, 0]),
             lambda f: rl.causal_conv(x, f(w)), lambda f: rl.causal_conv_backward(f(x), x, w),
             lambda f: rl.causal_conv_step(torch.zeros(2, 3, 8), f(x[:, 0]), w),
             lambda f: rl.add_rms_norm(f(x), A[:, 0]), lambda f: rl.add_rms_norm_backward(x, f(x), A[:, 0])]
    with fwd.dual_level():
        for call in calls:
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(lambda t: fwd.make_dual(t, torch.ones_like(t)))
            with pytest.raises(ValueError, match="CUDA"):
                call(lambda t: t)


PER_DEVICE = """
#include <cstdio>
#include "per_device.cuh"
using rlscan::seq::PerDevice;
int main()
{
    static PerDevice limits;
    int asked[3] = {0, 0, 0}, current = 0, answer = 0;
    auto find = [&] { ++asked[current]; return answer; };
    if (limits.get(0, find) != 0 || limits.get(0, find) != 0 || asked[0] != 2) return 1;   // a failure is not kept
    answer = 100;
    if (limits.get(0, find) != 100 || limits.get(0, find) != 100 || asked[0] != 3) return 2;
    current = 1;
    answer = 200;   // another device is asked itself, and the first keeps its own
    if (limits.get(1, find) != 200 || asked[1] != 1 || limits.get(0, find) != 100 || asked[0] != 3) return 3;
    current = 2;    // devices that are not numbered here are asked every time
    const int others[3] = {-1, PerDevice::kDevices, PerDevice::kDevices};
    for (int d : others)
        if (limits.get(d, find) != 200) return 4;
    if (asked[2] != 3) return 5;
    std::puts("done");
}
"""


def test_limits_are_kept_for_each_device(tmp_path):
    """What a launch finds out once (shared memory raised, SMs, resident blocks) it finds out on each device."""
    src, exe = tmp_path / "per_device.cpp", tmp_path / "per_device"
    src.write_text(PER_DEVICE)
    include = os.path.join(ROOT, "linear_recurrence_scan_gb300", "csrc_sequence")
    subprocess.run(["g++", "-std=c++17", "-I", include, str(src), "-o", str(exe)], check=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "done" in r.stdout, r.returncode
