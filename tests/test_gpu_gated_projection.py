"""The gated feed-forward block's projections on the GPU against float64:
sizes where tiles, stages and 16-byte rows end, both activations, strides,
alignments.  The bounds are derived in token_policy_cases.py."""
import numpy as np
import pytest
import torch

from state_space_cases import DEV, close
from token_policy_cases import projection_inputs, projection_oracle

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


def check(M, D, F, act="silu", seed=0, place=lambda t: t.to(DEV)):
    x, wg, wu, gh, _ = projection_inputs(M, D, F, seed + M + D + F)
    want = projection_oracle(x, wg, wu, gh, act)
    dev = [place(t) for t in (x, wg, wu)]
    h = L().gated_projection(*dev, act)
    close(h, *want["h"], 1.0, "h")
    run = lambda: L().gated_projection_backward(place(gh), *dev, act)  # noqa: E731
    g = run()
    for k in ("x", "gate_weight", "up_weight"):
        close(getattr(g, k), *want[k], 1.0, "gradient of " + k)
    for p, q in zip((h, *g), (L().gated_projection(*dev, act), *run())):
        assert torch.equal(p, q)
    L().workspace_status()


SIZES = [(3, 64, 64), (1, 8, 8), (128, 64, 128), (129, 72, 136), (256, 128, 256), (257, 200, 520), (300, 640, 320),
         (700, 512, 1000), (64, 2048, 768), (2, 256, 4096), (1000, 64, 72)]
ODD = [(1, 1, 1), (5, 7, 9), (40, 1111, 333), (260, 65, 131), (33, 130, 262)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_forward_and_gradients(M, D, F, act):
    check(M, D, F, act)


@pytest.mark.parametrize("M,D,F", ODD)
def test_odd_sizes(M, D, F):
    check(M, D, F)
    check(M, D, F, "gelu")


def test_more_tiles_than_pairs():
    check(2100, 128, 3000)
