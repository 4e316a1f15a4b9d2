"""The token policy's operators without a GPU: refusals of the C entry points
before anything is enqueued, workspace queries, refusals of the functions."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, CONFLICT, VALUE, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scan_gb300 import _native, build
    build.build()
    return _native.lib()


def gated(N=2, T=5, D=8, dtype=0, x=256, log_decay=512, token=8):
    from linear_recurrence_scan_gb300 import token_policy as tp
    return tp._GATED_ARGS.pack(N, T, D, dtype, *[x, T * token, token] * 3, log_decay, 0, 0, 0)


def projection(M=4, D=8, F=16, act=0, x=256, w=512, stride=8):
    from linear_recurrence_scan_gb300 import token_policy as tp
    return tp._PROJECTION_ARGS.pack(M, D, F, act, x, stride, w, stride, w + 4096, stride)


def distill(N=2, T=3, V=10, K=4, dtype=0, teacher=0, token=8, z=256, tau=1.0):
    from linear_recurrence_scan_gb300 import token_policy as tp
    return tp._DISTILL_ARGS.pack(N, T, V, K, dtype, teacher, token, z, T * V, V, 512, 1024, 0, tau)


def test_gated_scan_refusals(lib):
    f = lib.rlscan_gated_scan
    assert f(None, 4096, None, None, None) == NULL
    assert f(gated(N=-1), 4096, None, None, None) == SHAPE
    assert f(gated(N=1 << 40, T=1 << 20), 4096, None, None, None) == SHAPE
    assert f(gated(dtype=2), 4096, None, None, None) == VALUE
    assert f(gated(x=0), 4096, None, None, None) == NULL
    assert f(gated(log_decay=0), 4096, None, None, None) == NULL
    assert f(gated(), None, None, None, None) == NULL
    assert f(gated(), 256, None, None, None) == CONFLICT        # y is x
    assert f(gated(), 4096, 4096, None, None) == CONFLICT       # one buffer for two outputs
    for empty in (gated(N=0), gated(D=0)):
        assert f(empty, None, None, None, None) == 0
    g = lib.rlscan_gated_scan_backward
    from linear_recurrence_scan_gb300 import token_policy as tp
    from linear_recurrence_scan_gb300.state_space import _ARRAY3
    grads = tp._GATED_GRADS.pack(8192, 12288, 16384, 0, 0)
    gy = _ARRAY3.pack(20480, 40, 8)
    assert g(gated(), None, None, 24576, grads, None, 0, None) == NULL
    assert g(gated(), gy, None, None, grads, None, 0, None) == NULL
    assert g(gated(), gy, None, 24576, tp._GATED_GRADS.pack(8192, 8192, 16384, 0, 0), None, 0, None) == CONFLICT
    assert g(gated(), gy, None, 24576, tp._GATED_GRADS.pack(8192, 12288, 16384, 28672, 0), None, 0, None) == WORKSPACE
    s = lib.rlscan_gated_scan_step
    assert s(gated(), 4096, 2, None, 8192, None) == SHAPE           # several tokens
    assert s(gated(T=1), 4096, 1, None, 8192, None) == SHAPE        # two sequences, one slot
    assert s(gated(T=1), 4096, 2, None, 4096, None) == CONFLICT
    assert s(gated(T=1), None, 2, None, 8192, None) == NULL


def test_projection_refusals(lib):
    f = lib.rlscan_gated_projection
    assert f(None, 4096, None, 0, None) == NULL
    assert f(projection(M=-1), 4096, None, 0, None) == SHAPE
    assert f(projection(F=1 << 31), 4096, None, 0, None) == SHAPE
    assert f(projection(act=2), 4096, None, 0, None) == VALUE
    assert f(projection(x=0), 4096, None, 0, None) == NULL
    assert f(projection(), 256, None, 0, None) == CONFLICT
    assert f(projection(M=0), None, None, 0, None) == 0
    odd = projection(M=40, D=9, F=16, stride=9)   # rows that tensor maps do not take are copied first
    assert lib.rlscan_gated_projection_workspace_bytes(odd) >= 2 * (40 + 2 * 16) * 16
    assert f(odd, 65536, None, 0, None) == WORKSPACE
    assert lib.rlscan_gated_projection_workspace_bytes(projection(M=40)) == 0
    b = lib.rlscan_gated_projection_backward
    assert b(projection(), 8192, 16, None, 16384, None, None, 0, None) == NULL     # one weight's gradient alone
    assert b(projection(), 8192, 16, 8192, None, None, None, 0, None) == CONFLICT
    assert b(projection(), 8192, 16, 12288, 16384, 16384, None, 0, None) == CONFLICT
    assert lib.rlscan_gated_projection_backward_workspace_bytes(projection(M=0)) == 0


def test_distill_refusals(lib):
    f = lib.rlscan_distill_loss
    assert f(None, 4096, None, None) == NULL
    for bad in (distill(K=0), distill(K=257), distill(dtype=2), distill(teacher=3), distill(token=2), distill(tau=0.0),
                distill(tau=-1.0), distill(tau=float("nan")), distill(tau=float("inf"))):
        assert f(bad, 4096, None, None) == VALUE
    assert f(distill(V=1 << 31), 4096, None, None) == SHAPE
    assert f(distill(V=0), 4096, None, None) == SHAPE
    assert f(distill(z=0), 4096, None, None) == NULL
    assert f(distill(), None, None, None) == NULL
    assert f(distill(), 256, None, None) == CONFLICT
    assert f(distill(), 4096, 4096, None) == CONFLICT
    assert f(distill(N=0), None, None, None) == 0
    assert lib.rlscan_distill_loss_backward(distill(), 4096, 8192, 256, None) == CONFLICT
    assert lib.rlscan_distill_loss_backward(distill(), None, 8192, 12288, None) == NULL
    assert lib.rlscan_distill_loss_and_grad(distill(), 4096, 8192, None, 12288, None) == NULL
    assert lib.rlscan_distill_loss_and_grad(distill(), 4096, 4096, 8192, 12288, None) == CONFLICT


QUERIES = """
from linear_recurrence_scan_gb300 import _native, token_policy as tp
lib = _native.lib()
for N, T, D in ((0, 600, 64), (2, 600, 0), (0, 600, 0), (2, 0, 64), (0, 100000, 4096), (1, 100000, 0)):
    for dtype in (0, 1):
        a = tp._GATED_ARGS.pack(N, T, D, dtype, *[256, T * D, D] * 3, 256, 0, 0, 0)
        assert lib.rlscan_gated_scan_backward_workspace_bytes(a) == (0 if N * D == 0 else 4 * N * D), (N, T, D)
    p = tp._PROJECTION_ARGS.pack(N * T, D, 7, 0, 256, D, 512, D, 1024, D)
    assert not lib.rlscan_gated_projection_workspace_bytes(p) or N * T * D, (N, T, D)
    assert not lib.rlscan_gated_projection_backward_workspace_bytes(p) or N * T * D, (N, T, D)
print("done")
"""


def test_queries_of_empty_calls(lib):
    """In a child: an integer division by zero ends the process."""
    r = subprocess.run([sys.executable, "-c", QUERIES], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, (r.returncode, r.stderr[-2000:])


def test_argument_structs_match_the_header(lib, tmp_path):
    """The packed arguments have the sizes that C gives the header's structs."""
    from linear_recurrence_scan_gb300 import token_policy as tp
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include <stdio.h>\n#include "rlscan.h"\nint main(void) { printf("%zu %zu %zu %zu\\n", '
                   'sizeof(rlscan_gated_scan_args), sizeof(rlscan_gated_scan_grads), sizeof(rlscan_gated_projection_args), '
                   'sizeof(rlscan_distill_args)); return 0; }\n')
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True, timeout=60)
    sizes = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split()]
    assert sizes == [tp._GATED_ARGS.size, tp._GATED_GRADS.size, tp._PROJECTION_ARGS.size, tp._DISTILL_ARGS.size]
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_refusals_of_the_functions():
    """CPU tensors and dual tensors, before anything else."""
    import torch
    import torch.autograd.forward_ad as fwd
    import linear_recurrence_scan_gb300 as rl
    x, d, marks, state = torch.zeros(2, 4, 8), torch.zeros(8), torch.zeros(2, 1, 8), torch.zeros(2, 8)
    b = x.bfloat16()
    w = torch.zeros(6, 8, dtype=torch.bfloat16)
    z, th, tok, gl = torch.zeros(2, 4, 9), torch.zeros(2, 4, 3), torch.zeros(2, 4, 3, dtype=torch.long), torch.zeros(2, 4)
    calls = [lambda f: rl.gated_scan(f(x), x, x, d), lambda f: rl.gated_scan(x, x, x, f(d)),
             lambda f: rl.gated_scan(x, x, x, d, initial_state=f(state)),
             lambda f: rl.gated_scan_backward(x, f(x), x, x, d, marks),
             lambda f: rl.gated_scan_step(state, x[:, 0], f(x[:, 0]), x[:, 0], d),
             lambda f: rl.gated_projection(f(b), w, w), lambda f: rl.gated_projection(b, w, f(w)),
             lambda f: rl.gated_projection_backward(f(b[..., :6]), b, w, w),
             lambda f: rl.distill_loss(f(z), th, tok), lambda f: rl.distill_loss_backward(f(gl), z, th, tok, torch.zeros(2, 4, 2)),
             lambda f: rl.distill_loss_and_grad(gl, f(z), th, tok)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call(lambda t: t)
    with fwd.dual_level():
        for call in calls:
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(lambda t: fwd.make_dual(t, torch.ones_like(t)))
    with pytest.raises(ValueError, match="detach"):
        rl.distill_loss(z, th.clone().requires_grad_(), tok)
