"""The state-space layer on the GPU where the ordinary cases of
test_gpu_state_space.py do not lead: states that decay within a token, and
calls large enough for the variants that the largest workloads take."""
import numpy as np
import pytest
import torch

from oracle import state_space as ref
from state_space_cases import (DEV, U, close, conv_factor, norm_factor, np64, scan_factor, scan_grad_factor, scan_inputs,
                               to_dev)

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


# ---------------------------------------------------------------------------
# as many rows, tokens and channels as the wide variants take

def channels_of(D):
    """some of D channels: both ends, and every place in a vector of eight"""
    return sorted({0, 1, 2, 3, D // 2, D // 2 + 5, D // 3, D - 9, D - 4, D - 3, D - 2, D - 1})


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D,K,kind", [(4, 4099, 4096, 4, "both"), (2, 4100, 1024, 4, "none"), (3, 1031, 4100, 2, "both"),
                                          (3, 1031, 4098, 8, "both")])
def test_conv_of_long_runs(N, T, D, K, kind, dtype):
    """Four and two channels a thread in runs of up to 64 and 128 tokens; every channel by itself, so some are compared."""
    g = torch.Generator(device=DEV)
    g.manual_seed(N + T + D + K)

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(to)

    x, w, b = normal(N, T, D), normal(D, K, scale=0.5, to=F32), normal(D, to=F32)
    init, gy, gf = normal(N, K - 1, D), normal(N, T, D), normal(N, K - 1, D)
    resets = lengths = None
    if kind == "both":
        resets = (torch.rand(N, T, generator=g, device=DEV) < 1 / 50).to(torch.uint8)
        lengths = torch.tensor([T, T - 70, 513, 2][:N], dtype=torch.int32, device=DEV)
    flags = dict(resets=resets, lengths=lengths)
    y, final = L().causal_conv(x, w, b, initial_state=init, **flags)
    grads = L().causal_conv_backward(gy, x, w, b, initial_state=init, **flags, grad_final_state=gf)
    at = channels_of(D)
    args = (np64(x[..., at]), np64(w[at]), np64(b[at]), "silu", np64(init[..., at]),
            *(None if f is None else f.cpu().numpy() for f in (resets, lengths)))
    ry, rf, _, _ = ref.causal_conv(*args)
    _, _, mag, _ = ref.causal_conv(*args, bound=True)
    close(y[..., at], ry, mag, conv_factor(K), "y")
    assert np.array_equal(np64(final[..., at]), rf)
    want = ref.causal_conv_backward(np64(gy[..., at]), *args, grad_final=np64(gf[..., at]))
    mag = ref.causal_conv_backward(np64(gy[..., at]), *args, grad_final=np64(gf[..., at]), bound=True)
    for k in want:
        got = getattr(grads, k)[at] if k in ("weight", "bias") else getattr(grads, k)[..., at]
        close(got, want[k], mag[k], conv_factor(K, N * T), "gradient of " + k)


def near(got, want, tol, what):
    """|got - want| within tol, and a rounding to bfloat16 where got has that type (all on the GPU, in 64 bits)"""
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * want.abs()
    off = ~((got.double() - want).abs() <= tol + 1e-30)
    assert not off.any(), f"{what}: {int(off.sum())} of {off.numel()} off, first at {off.nonzero()[0].tolist()}"


@pytest.mark.parametrize("rtype", [None, F32, BF16], ids=["plain", "res32", "res16"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(5003, 2560), (5003, 2561), (9001, 200), (9001, 131), (1501, 9000), (701, 20001)])
def test_norm_of_many_rows(M, D, dtype, rtype):
    """Blocks and warps that take several rows, wide, narrow, odd and long, their sums over rows, and the 8-bit output."""
    if dtype == F32 and rtype == BF16:
        return
    g = torch.Generator(device=DEV)
    g.manual_seed(M + D)

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(to)

    eps = 1e-5
    x, w, gy = normal(M, D), 1 + normal(D, scale=0.3, to=F32), normal(M, D)
    r = None if rtype is None else normal(M, D, scale=2.0, to=rtype)
    out = L().add_rms_norm(x, w, r, eps=eps)
    q = L().add_rms_norm(x, w, r, eps=eps, out_dtype=torch.float8_e4m3fn)
    x64, w64 = x.double(), w.double()
    h64 = x64 if r is None else x64 + r.double()
    hmag = x64.abs() if r is None else x64.abs() + r.double().abs()
    inv = 1 / (h64.square().mean(-1, keepdim=True) + eps).sqrt()
    want = h64 * inv * w64
    slack = norm_factor(D) * (want.abs() + hmag * w64.abs() * inv)
    near(out.y, want, slack, "y")
    if r is not None:
        near(out.residual, h64, 2 * U * hmag, "sum")
        assert torch.equal(out.residual, q.residual)
    pad = torch.nn.functional.pad
    blocks, parts = (pad(t.abs(), (0, -D % 128)).view(M, -1, 128).amax(-1) for t in (want, slack))
    near(q.scales, blocks / 448, parts / 448 + 4 * U * blocks / 448, "scales")
    each = q.scales.double().repeat_interleave(128, -1)[:, :D]
    near(q.y.float() * each.float(), want, 1.001 * (2.0 ** -4 * want.abs() + 2.0 ** -10 * each) + slack, "8-bit y")
    h = x if r is None else out.residual
    gr = None if r is None else normal(M, D, to=rtype)
    grads = L().add_rms_norm_backward(gy, h, w, gr, eps=eps)
    h64, gy64 = h.double(), gy.double()
    inv = 1 / (h64.square().mean(-1, keepdim=True) + eps).sqrt()
    n, gn = h64 * inv, gy64 * w64
    more, size = (0, 0) if gr is None else (gr.double(), gr.double().abs())
    want = inv * (gn - n * (gn * n).mean(-1, keepdim=True)) + more
    mag = inv * (gn.abs() + n.abs() * (gn * n).abs().mean(-1, keepdim=True)) + size
    near(grads.x, want, 2 * norm_factor(D) * mag, "gradient of x")
    near(grads.residual, want, 2 * norm_factor(D) * mag, "gradient of the residual")
    near(grads.weight, (gy64 * n).sum(0), (2 * norm_factor(D) + M * U) * (gy64 * n).abs().sum(0), "gradient of weight")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,D,S", [(257, 1024, 16), (255, 1001, 16), (257, 1024, 8), (130, 1024, 13), (258, 515, 32),
                                   (514, 2048, 3), (66, 512, 128)])
def test_scan_step_of_many_sequences(N, D, S, dtype):
    """Several sequences a lane, idle ones among them, the last lanes' without a sequence."""
    a, _, _, _, rng = scan_inputs(N, 1, D, S, dtype, 50 + N + D, step=True)
    P = N + 5
    state = torch.from_numpy(rng.standard_normal((P, D, S)).astype(np.float32))
    slots = torch.from_numpy(rng.permutation(P)[:N].astype(np.int32))
    slots[::7], slots[3::50] = -1, P
    st = state.to(DEV)
    y = L().selective_scan_step(st, **{k: v.to(DEV) for k, v in a.items()}, slots=to_dev(slots))
    r64 = {k: (np64(v)[:, None] if k in ("x", "delta", "z", "B", "C") else np64(v)) for k, v in a.items()}
    at = slots.numpy()
    idle = (at < 0) | (at >= P)
    old = np64(state)[np.where(idle, 0, at)]
    ry, rf, _, _ = ref.selective_scan(**r64, initial_state=old)
    my, mf, _, _ = ref.selective_scan(**r64, initial_state=old, bound=True)
    ry[idle] = 0
    close(y, ry[:, 0], my[:, 0], scan_factor(1), "y")
    want, mag = np64(state), np.abs(np64(state))
    want[at[~idle]], mag[at[~idle]] = rf[~idle], mf[~idle]
    close(st, want, mag, scan_factor(1), "state")
    untouched = np.setdiff1d(np.arange(P), at)
    assert np.array_equal(st.cpu().numpy()[untouched], state.numpy()[untouched])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scan_of_many_whole_rows(dtype):
    """More than a block an SM, rows of several tiles and unlike lengths, episodes inside."""
    N, T, D, S = 24, 90, 1280, 16
    a, init, _, _, rng = scan_inputs(N, T, D, S, dtype, 60)
    resets = torch.from_numpy((rng.random((N, T)) < 0.02).astype(np.uint8))
    lengths = torch.from_numpy(rng.integers(1, T + 1, N).astype(np.int32))
    lengths[3], lengths[5] = T, 0
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    r64 = {k: np64(v) for k, v in a.items()}
    dev = {k: v.to(DEV) for k, v in a.items()}
    flags = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    args = dict(initial_state=np64(init), resets=resets.numpy(), lengths=lengths.numpy())
    y, final, marks = L().selective_scan(**dev, initial_state=to_dev(init), **flags, return_checkpoints=True)
    ry, rf, _, _ = ref.selective_scan(**r64, **args)
    my, mf, _, _ = ref.selective_scan(**r64, **args, bound=True)
    close(y, ry, my, scan_factor(T), "y")
    close(final, rf, mf, scan_factor(T), "final state")
    g = L().selective_scan_backward(gy.to(DEV), dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks, dev["D"],
                                    dev["z"], dev["delta_bias"], **flags)
    want = ref.selective_scan_backward(np64(gy), **r64, **args)
    mag = ref.selective_scan_backward(np64(gy), **r64, **args, bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], scan_grad_factor(T, max(D, N * T)), "gradient of " + k)
