"""The gated recurrence on the GPU against its float64 oracle: sizes where
steps, warps, pairs and clusters end, both types, strides and alignments,
episode flags, padding, empty rows, idle slots, closed gates, streams, graphs.
The bounds are derived in token_policy_cases.py."""
import numpy as np
import pytest
import torch

from oracle import token_policy as ref
from state_space_cases import DEV, U, close, np64, strided, to_dev
from token_policy_cases import gated_factor, gated_grad_factor, gated_inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


def check(N, T, D, dtype, kind, seed=0, strongest=5.0, a=None):
    """Forward and gradients of one case against the oracle, twice for the same bits."""
    made, init, resets, lengths, rng = gated_inputs(N, T, D, dtype, seed + N + 10 * T + 100 * D, kind, strongest=strongest)
    a = made if a is None else a
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gf = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32))
    r64 = {k: np64(v) for k, v in a.items()}
    args = dict(initial_state=np64(init), resets=None if resets is None else resets.numpy(),
                lengths=None if lengths is None else lengths.numpy())
    dev = {k: v.to(DEV) for k, v in a.items()}
    on = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    y, final, marks = L().gated_scan(**dev, initial_state=to_dev(init), **on, return_checkpoints=True)
    ry, rf, rs = ref.gated_scan(**r64, **args)
    my, mf, ms = ref.gated_scan(**r64, **args, bound=True)
    close(y, ry, my, gated_factor(T), "y")
    close(final, rf, mf, gated_factor(T), "final state")
    close(marks, rs[:, 0:T:32], ms[:, 0:T:32], gated_factor(T), "checkpoints")
    run = lambda: L().gated_scan_backward(gy.to(DEV), **dev, checkpoints=marks, **on, grad_final_state=to_dev(gf))  # noqa: E731
    g = run()
    want = ref.gated_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf))
    mag = ref.gated_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf), bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], gated_grad_factor(T, N * T if k == "log_decay" else 0), "gradient of " + k)
    for p, q in zip((y, final, marks, *g),
                    (*L().gated_scan(**dev, initial_state=to_dev(init), **on, return_checkpoints=True), *run())):
        assert torch.equal(p, q)
    plain = L().gated_scan(**dev, initial_state=to_dev(init), **on)
    assert len(plain) == 2 and torch.equal(plain[0], y) and torch.equal(plain[1], final)


# single values, a warp's tokens, a step's end, one and several channels, blocks of 64 channels, clusters of 2 to 8 blocks
SIZES = [(1, 1, 1), (2, 3, 2), (1, 7, 33), (2, 8, 64), (3, 9, 65), (1, 63, 40), (2, 64, 130), (2, 65, 5), (1, 127, 96),
         (2, 128, 31), (1, 129, 64), (2, 256, 66), (3, 300, 48), (1, 513, 130), (2, 700, 17)]


@pytest.mark.parametrize("kind", ["none", "packed", "ragged", "dense", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", SIZES)
def test_forward_and_gradients(N, T, D, dtype, kind):
    check(N, T, D, dtype, kind)


@pytest.mark.parametrize("kind", ["packed", "ragged"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", [(5, 150, 4100), (20, 130, 1027), (2, 200, 9800), (2, 400, 2560)])
def test_many_channels(N, T, D, dtype, kind):
    """Blocks that walk a row alone, and clusters of two and four."""
    check(N, T, D, dtype, kind)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_long_rows(dtype):
    check(1, 4000, 70, dtype, "both", strongest=0.5)
    check(2, 3001, 64, dtype, "none", strongest=0.01)
