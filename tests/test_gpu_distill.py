"""The distillation loss on the GPU against its float64 oracle: vocabularies
where warps, blocks, clusters and 16-byte units end, both types, strides,
alignments, masked rows, empty and repeated teacher tokens, infinities, NaN.
The bounds are derived in token_policy_cases.py."""
import numpy as np
import pytest
import torch

from oracle import token_policy as ref
from state_space_cases import DEV, close, np64, to_dev
from token_policy_cases import distill_factor, distill_inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


def check(logits, teacher, tokens, mask, grad_loss, tau=1.0, on_gpu=None):
    """All three calls against the oracle, the two ways to the gradient against each other."""
    V, K = logits.shape[2], teacher.shape[2]
    dev = logits.to(DEV) if on_gpu is None else on_gpu
    args = (teacher.to(DEV), tokens.to(DEV))
    m = to_dev(mask)
    loss, norm = L().distill_loss(dev, *args, tau, m, return_normalizers=True)
    grad = L().distill_loss_backward(grad_loss.to(DEV), dev, *args, norm, tau, m)
    both_loss, both_grad = L().distill_loss_and_grad(grad_loss.to(DEV), dev, *args, tau, m)
    rl, rg, ml, mg = ref.distill_loss(np64(logits), np64(teacher), tokens.numpy(), tau,
                                      None if mask is None else mask.numpy() != 0, np64(grad_loss))
    z, th = np64(logits), np64(teacher)
    z, th = z[np.isfinite(z) & (np.abs(z) < 1e30)], th[np.isfinite(th)]
    f = distill_factor(V, K, max(np.ptp(z) if z.size else 0, np.ptp(th) if th.size else 0) / tau)
    close(loss, rl, ml, f, "loss")
    close(both_loss, rl, ml, f, "loss with its gradient")
    close(grad, rg, mg, f, "gradient")
    close(both_grad, rg, mg, f, "gradient with its loss")
    assert grad.shape == logits.shape and grad.dtype == logits.dtype and grad.is_contiguous()
    again = L().distill_loss_and_grad(grad_loss.to(DEV), dev, *args, tau, m)
    assert torch.equal(again[0], both_loss) and torch.equal(again[1], both_grad)
    return loss, both_grad


# vocabularies: within a warp's registers, a small block's, a block's, a cluster's; one unit more or less
SIZES = [(1, 1, 1, 1), (2, 3, 2, 2), (1, 5, 7, 3), (2, 2, 31, 5), (3, 3, 64, 8), (1, 4, 1000, 33), (1, 3, 1023, 64),
         (2, 2, 2047, 32), (1, 2, 2049, 256), (1, 2, 4100, 31), (1, 3, 8191, 16), (1, 2, 8200, 64), (1, 2, 32761, 32),
         (1, 2, 33000, 100), (1, 1, 50257, 32), (1, 1, 131075, 20), (2, 1, 262143, 8)]


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,V,K", SIZES)
def test_loss_and_gradient(N, T, V, K, dtype, tau):
    logits, teacher, tokens, mask, grad, _ = distill_inputs(N, T, V, K, dtype, V + K)
    check(logits, teacher, tokens, mask if N * T > 2 else None, grad, tau)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,V,K", [(2, 400, 9000, 4), (1, 7000, 300, 6), (3, 900, 5000, 3), (1, 650, 36001, 3), (1, 330, 140000, 2)])
def test_many_rows(N, T, V, K, dtype):
    """More rows than blocks: every block takes several, in one part each and in several."""
    logits, teacher, tokens, mask, grad, _ = distill_inputs(N, T, V, K, dtype, 3)
    check(logits, teacher, tokens, mask, grad)


def test_rows_longer_than_a_cluster_holds():
    """The loss and its gradient in two calls, over rounds of a block."""
    for dtype, V in ((F32, 140001), (BF16, 270001)):
        logits, teacher, tokens, mask, grad, _ = distill_inputs(1, 2, V, 5, dtype, 9)
        check(logits, teacher, tokens, None, grad)


@pytest.mark.parametrize("token_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("teacher_dtype", [F32, BF16], ids=["f32", "bf16"])
def test_teacher_types(teacher_dtype, token_dtype):
    logits, teacher, tokens, mask, grad, _ = distill_inputs(2, 9, 300, 12, BF16, 4, teacher_dtype, token_dtype)
    check(logits, teacher, tokens, mask.bool(), grad)
