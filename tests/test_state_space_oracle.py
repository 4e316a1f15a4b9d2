"""The state-space layer's oracle: its gradients against central differences
of its own forward pass, closed forms, and the Python layer's refusals that
need no GPU."""
import numpy as np
import pytest
import torch

from oracle import state_space as ref


def differences(f, a, eps=1e-6):
    """d f / d a by central differences (error of order eps^2 and 1e-16 / eps)"""
    g = np.zeros_like(a)
    flat, out = a.reshape(-1), g.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + eps
        hi = f()
        flat[i] = keep - eps
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * eps)
    return g


KINDS = ["none", "packed", "ragged"]


def _flags(kind, N, T):
    resets = lengths = None
    if kind == "packed":
        resets = np.zeros((N, T), np.uint8)
        resets[0, 2] = resets[1, 0] = resets[1, T - 1] = 1
    if kind == "ragged":
        lengths = np.array([T - 2, 0])
    return resets, lengths


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_are_the_differences(kind, softplus):
    rng = np.random.default_rng(1)
    N, T, W, S = 2, 5, 2, 3
    a = dict(x=rng.standard_normal((N, T, W)), delta=rng.uniform(0.1, 1, (N, T, W)),
             A=-rng.uniform(0.2, 2, (W, S)), B=rng.standard_normal((N, T, S)), C=rng.standard_normal((N, T, S)),
             D=rng.standard_normal(W), z=rng.standard_normal((N, T, W)), delta_bias=rng.uniform(-1, 1, W),
             initial_state=rng.standard_normal((N, W, S)))
    resets, lengths = _flags(kind, N, T)
    gy, gf = rng.standard_normal((N, T, W)), rng.standard_normal((N, W, S))

    def loss():
        y, final, _, _ = ref.selective_scan(delta_softplus=softplus, resets=resets, lengths=lengths, **a)
        return (y * gy).sum() + (final * gf).sum()

    g = ref.selective_scan_backward(gy, delta_softplus=softplus, resets=resets, lengths=lengths, grad_final=gf, **a)
    for k in a:
        assert np.allclose(g[k], differences(loss, a[k]), rtol=1e-6, atol=1e-7), k


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("K", [1, 3, 4])
def test_conv_gradients_are_the_differences(kind, activation, K):
    rng = np.random.default_rng(2)
    N, T, W = 2, 4, 2
    a = dict(x=rng.standard_normal((N, T, W)), weight=rng.standard_normal((W, K)), bias=rng.standard_normal(W),
             initial_state=rng.standard_normal((N, K - 1, W)))
    resets, lengths = _flags(kind, N, T)
    gy, gf = rng.standard_normal((N, T, W)), rng.standard_normal((N, K - 1, W))

    def loss():
        y, final, _, _ = ref.causal_conv(activation=activation, resets=resets, lengths=lengths, **a)
        return (y * gy).sum() + (final * gf).sum()

    g = ref.causal_conv_backward(gy, activation=activation, resets=resets, lengths=lengths, grad_final=gf, **a)
    for k in a:
        assert np.allclose(g[k], differences(loss, a[k]), rtol=1e-6, atol=1e-7), k


def test_norm_gradients_are_the_differences():
    rng = np.random.default_rng(3)
    a = dict(x=rng.standard_normal((3, 5)), weight=rng.standard_normal(5))
    residual = rng.standard_normal((3, 5))
    gy, gr = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss():
        y, h = ref.add_rms_norm(a["x"], a["weight"], residual)
        return (y * gy).sum() + (h * gr).sum()

    g = ref.add_rms_norm_backward(gy, a["x"] + residual, a["weight"], gr)
    for k in a:
        assert np.allclose(g[k], differences(loss, a[k]), rtol=1e-6, atol=1e-7), k


def test_scan_closed_form_and_resets():
    """Constant decay a and input b from 0: h_t = b (1 - a^(t+1)) / (1 - a); a reset starts it again."""
    T = 12
    one = np.ones((1, T, 1))
    A = np.full((1, 1), np.log(0.75))
    y, final, _, _ = ref.selective_scan(2 * one, one, A, one, one, delta_softplus=False)
    want = 2 * (1 - 0.75 ** np.arange(1, T + 1)) / 0.25
    assert np.allclose(y[0, :, 0], want, rtol=1e-13)
    resets = np.zeros((1, T), np.uint8)
    resets[0, 7] = 1
    y, final, _, _ = ref.selective_scan(2 * one, one, A, one, one, delta_softplus=False, resets=resets)
    assert np.allclose(y[0, 7:, 0], want[:T - 7], rtol=1e-13) and np.allclose(y[0, :7, 0], want[:7], rtol=1e-13)


def test_splitting_a_prompt_changes_nothing():
    rng = np.random.default_rng(4)
    N, T, W, S, K = 2, 9, 3, 4, 4
    x, d, z = (rng.standard_normal((N, T, W)) for _ in range(3))
    B, C = (rng.standard_normal((N, T, S)) for _ in range(2))
    A = -rng.uniform(0.2, 2, (W, S))
    y, final, _, _ = ref.selective_scan(x, d, A, B, C, z=z)
    y1, f1, _, _ = ref.selective_scan(x[:, :5], d[:, :5], A, B[:, :5], C[:, :5], z=z[:, :5])
    y2, f2, _, _ = ref.selective_scan(x[:, 5:], d[:, 5:], A, B[:, 5:], C[:, 5:], z=z[:, 5:], initial_state=f1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, rtol=1e-12) and np.allclose(f2, final, rtol=1e-12)
    w = rng.standard_normal((W, K))
    y, final, _, _ = ref.causal_conv(x, w)
    y1, f1, _, _ = ref.causal_conv(x[:, :2], w)
    y2, f2, _, _ = ref.causal_conv(x[:, 2:], w, initial_state=f1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, rtol=1e-12) and np.allclose(f2, final, rtol=1e-12)


def test_python_layer_refuses_cpu_tensors_and_bad_options():
    import linear_recurrence_scan_gb300 as rl
    x, bc, A = torch.zeros(2, 4, 8), torch.zeros(2, 4, 3), torch.zeros(8, 3)
    with pytest.raises(ValueError, match="CUDA"):
        rl.selective_scan(x, x, A, bc, bc)
    with pytest.raises(ValueError, match="dimensions"):
        rl.selective_scan(x[0], x[0], A, bc[0], bc[0])
    with pytest.raises(TypeError, match="Tensor"):
        rl.selective_scan(None, x, A, bc, bc)
    with pytest.raises(ValueError, match="CUDA"):
        rl.selective_scan_step(torch.zeros(2, 8, 3), x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        rl.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        rl.causal_conv_step(torch.zeros(2, 3, 8), x[:, 0], torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        rl.add_rms_norm(x, torch.ones(8))
    with pytest.raises(ValueError, match="2 dimensions"):
        rl.add_rms_norm(torch.zeros(8), torch.ones(8))


# ---------------------------------------------------------------------------
# the C entry points refuse before any CUDA call (addresses that nothing reads)

@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scan_gb300 import _native, build
    build.build()
    return _native.lib()


def _scan(**kw):
    from linear_recurrence_scan_gb300 import state_space as ss
    a = dict(N=2, T=3, D=8, S=4, dtype=0, softplus=1, x=256, delta=512, z=0, B=768, C=1024, A=1280)
    a.update(kw)
    return ss._SCAN_ARGS.pack(a["N"], a["T"], a["D"], a["S"], a["dtype"], a["softplus"], a["x"], 24, 8, a["delta"], 24,
                              8, a["z"], 24, 8, a["B"], 12, 4, a["C"], 12, 4, a["A"], 0, 0, 0, 0, 0)


def test_c_entry_points_validate(lib):
    from linear_recurrence_scan_gb300 import state_space as ss

    def fwd(y=4096, final=None, **kw):
        return lib.rlscan_selective_scan(_scan(**kw), y, final, None, None, 0, None)

    assert lib.rlscan_selective_scan(None, 1, None, None, None, 0, None) == 1
    assert fwd(N=-1) == 2 and fwd(T=-1) == 2 and fwd(D=-1) == 2
    assert fwd(S=0) == 4 and fwd(S=129) == 4 and fwd(dtype=2) == 4 and fwd(softplus=2) == 4
    assert fwd(N=0) == 0 and fwd(D=0) == 0
    assert fwd(x=0) == 1 and fwd(A=0) == 1 and fwd(y=None) == 1
    assert fwd(y=256) == 3 and fwd(final=1280) == 3
    assert fwd(N=1 << 40, T=1 << 20) == 2

    def step(state=8192, P=2, slots=None, y=4096, **kw):
        return lib.rlscan_selective_scan_step(_scan(T=kw.pop("T", 1), **kw), state, P, slots, y, None)

    assert step(T=2) == 2 and step(P=1) == 2 and step(P=-1, slots=64) == 2
    assert step(state=None) == 1 and step(y=None) == 1
    assert step(y=8192) == 3 and step(state=256) == 3
    assert step(N=0, P=0) == 0

    gy = ss._ARRAY3.pack(2048, 24, 8)

    def grads(x=4096, z=0, skip=0, bias=0):
        return ss._SCAN_GRADS.pack(x, 0, z, 0, 0, 0, skip, bias, 0)

    def bwd(g=None, marks=8192, ws=None, n=0, **kw):
        return lib.rlscan_selective_scan_backward(_scan(**kw), gy, None, marks, g or grads(), ws, n, None)

    need = lib.rlscan_selective_scan_backward_workspace_bytes(_scan())
    assert need > 0
    assert bwd(S=0) == 4 and bwd(marks=None) == 1 and bwd(g=grads(x=0)) == 1
    assert bwd(g=grads(z=64)) == 3 and bwd(g=grads(skip=64)) == 3 and bwd(g=grads(bias=64)) == 3
    assert bwd(g=grads(x=2048)) == 3 and bwd(g=grads(x=8192)) == 3
    assert bwd() == 5 and bwd(ws=16384 + 8, n=need) == 5 and bwd(ws=16384, n=need - 1) == 5

    def conv_args(**kw):
        a = dict(N=2, T=3, D=8, K=4, dtype=0, silu=1, x=256, w=512)
        a.update(kw)
        return ss._CONV_ARGS.pack(a["N"], a["T"], a["D"], a["K"], a["dtype"], a["silu"], a["x"], 24, 8, a["w"], 0, 0, 0, 0)

    def conv(y=4096, final=None, **kw):
        return lib.rlscan_causal_conv(conv_args(**kw), y, final, None)

    assert conv(K=0) == 4 and conv(K=9) == 4 and conv(dtype=2) == 4 and conv(silu=3) == 4 and conv(T=-1) == 2
    assert conv(x=0) == 1 and conv(w=0) == 1 and conv(y=None) == 1 and conv(y=256) == 3 and conv(final=512) == 3
    assert conv(N=0) == 0
    assert lib.rlscan_causal_conv_step(conv_args(), 8192, 2, None, 4096, None) == 2      # T is 1 for a step
    assert lib.rlscan_causal_conv_step(conv_args(T=1), None, 2, None, 4096, None) == 1
    assert lib.rlscan_causal_conv_step(conv_args(T=1), 8192, 1, None, 4096, None) == 2
    assert lib.rlscan_causal_conv_backward(conv_args(), gy, None, 4096, 8192, None, None, None, 0, None) == 5
    assert lib.rlscan_causal_conv_backward(conv_args(), gy, None, 2048, None, None, None, None, 0, None) == 3
    assert lib.rlscan_causal_conv_backward(conv_args(), gy, None, None, None, None, None, None, 0, None) == 1

    def norm(x=256, r=0, w=512, M=2, D=8, eps=1e-6, dt=0, rt=0, y=4096, s=None, ro=None):
        return lib.rlscan_add_rms_norm(x, 8, r, 8, w, M, D, eps, dt, rt, y, s, ro, None)

    assert norm(M=-1) == 2 and norm(dt=2) == 4 and norm(eps=-1.0) == 4 and norm(eps=float("nan")) == 4
    assert norm(r=64, dt=0, rt=1, ro=8192) == 4 and norm(r=64) == 1 and norm(x=0) == 1
    assert norm(y=256) == 3 and norm(r=64, ro=4096) == 3 and norm(s=4096) == 3 and norm(M=0) == 0

    def norm_bwd(gy=256, h=512, w=768, gx=4096, gh=None, gw=None, dt=0, ht=0, ws=None, n=0):
        return lib.rlscan_add_rms_norm_backward(gy, 8, h, 8, None, 0, w, 2, 8, 1e-6, dt, ht, gx, gh, gw, ws, n, None)

    assert norm_bwd(gx=None) == 1 and norm_bwd(gx=512) == 3 and norm_bwd(gh=4096) == 3 and norm_bwd(ht=1) == 4
    assert norm_bwd(gw=8192) == 5
