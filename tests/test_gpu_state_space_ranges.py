"""The state-space layer on the GPU where the ordinary cases of
test_gpu_state_space.py do not lead: states that decay within a token."""
import numpy as np
import pytest
import torch

from oracle import state_space as ref
from state_space_cases import DEV, close, np64, scan_grad_factor, scan_inputs, to_dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


# time steps of 0.3 to 3.6 against rates up to 16, or of 0.1 to 0.35 against rates up to 128: exponents down to -57
@pytest.mark.parametrize("kind", ["none", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D,S,bias", [(2, 70, 40, 16, 2.0), (1, 400, 24, 16, 0.5), (2, 33, 12, 128, -1.5),
                                          (2, 40, 8, 3, 2.0)])
def test_scan_gradients_of_states_that_decay_at_once(N, T, D, S, bias, dtype, kind):
    """exp(dt A) h_{t-1} to its own size, however small beside dt x B."""
    a, init, resets, lengths, rng = scan_inputs(N, T, D, S, dtype, 31 * T + S, kind)
    a["delta"] = (a["delta"] * 0.7).clamp(-1.5, 1.5)
    a["delta_bias"] = torch.full((D,), bias)
    rates = torch.arange(1, S + 1).float()
    a["A"] = -(rates * (16 / 3 if S == 3 else 1)).repeat(D, 1)
    if S == 128:
        a["delta"] = a["delta"] * 0.4   # dt <= 0.35
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gf = torch.from_numpy(rng.standard_normal((N, D, S)).astype(np.float32))
    r64 = {k: np64(v) for k, v in a.items()}
    dev = {k: v.to(DEV) for k, v in a.items()}
    flags = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    args = dict(initial_state=np64(init), **{k: None if f is None else f.numpy()
                                             for k, f in (("resets", resets), ("lengths", lengths))})
    y, final, marks = L().selective_scan(**dev, initial_state=to_dev(init), **flags, return_checkpoints=True)
    g = L().selective_scan_backward(gy.to(DEV), dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks, dev["D"],
                                    dev["z"], dev["delta_bias"], **flags, grad_final_state=to_dev(gf))
    want = ref.selective_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf))
    mag = ref.selective_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf), bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], scan_grad_factor(T, max(D, N * T)), "gradient of " + k)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scan_gradient_of_a_first_token_has_no_decay(dtype):
    """Nothing stands before the first token of a row or of an episode: A's gradient is 0 to the bit."""
    N, T, D, S = 2, 40, 24, 16
    a, _, _, _, rng = scan_inputs(N, T, D, S, dtype, 32)
    dev = {k: v.to(DEV) for k, v in a.items()}
    for t, resets in ((1, None), (T, torch.ones(N, T, dtype=torch.uint8, device=DEV))):
        d = {k: (v[:, :t] if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
        y, final, marks = L().selective_scan(**d, resets=resets, return_checkpoints=True)
        g = L().selective_scan_backward(d["x"], d["x"], d["delta"], d["A"], d["B"], d["C"], marks, d["D"], d["z"],
                                        d["delta_bias"], resets=resets)
        assert g.x.any() and not g.A.any()
