"""The token policy's float64 oracle: gradients against central differences,
closed forms, brute force, identities (no GPU)."""
import math

import numpy as np
import pytest

from oracle import token_policy as ref


def gated(N, T, D, seed=0, kind="none"):
    rng = np.random.default_rng(seed)
    a = dict(x=rng.standard_normal((N, T, D)), gate=rng.standard_normal((N, T, D)), input_gate=rng.standard_normal((N, T, D)),
             log_decay=-rng.uniform(0.05, 2, D))
    more = dict(initial_state=rng.standard_normal((N, D)))
    if kind in ("packed", "both"):
        more["resets"] = (rng.random((N, T)) < 0.3).astype(np.uint8)
    if kind in ("ragged", "both"):
        more["lengths"] = rng.integers(0, T + 1, N)
    return a, more, rng


def test_gated_scan_is_the_sum_over_earlier_tokens():
    """h_t = prod a h_{-1} + sum_s (prod_{s < u <= t} a_u) b_s, summed directly."""
    a, more, _ = gated(2, 6, 3)
    y, final, _ = ref.gated_scan(**a, **more)
    sig = lambda v: 1 / (1 + np.exp(-v))  # noqa: E731
    r, i = sig(a["gate"]), sig(a["input_gate"])
    decay = np.exp(a["log_decay"] * r)
    b = np.sqrt(1 - decay ** 2) * i * a["x"]
    for t in range(6):
        want = more["initial_state"] * decay[:, :t + 1].prod(1)
        for s in range(t + 1):
            want = want + b[:, s] * decay[:, s + 1:t + 1].prod(1)
        np.testing.assert_allclose(y[:, t], want, rtol=1e-12)
    np.testing.assert_array_equal(final, y[:, -1])


def test_gated_scan_keeps_the_variance():
    """A constant gate on unit noise: states keep unit variance, which is what the root is for."""
    rng = np.random.default_rng(1)
    T, D = 400, 4000
    y, _, _ = ref.gated_scan(rng.standard_normal((1, T, D)), np.zeros((1, T, D)), np.full((1, T, D), 40.0), np.full(D, -0.2))
    assert abs(y[0, -1].var() - 1) < 0.1


def test_gated_scan_resets_and_lengths():
    """Packed episodes are their own rows; padding changes nothing."""
    a, _, _ = gated(1, 9, 4, 3)
    resets = np.zeros((1, 9), np.uint8)
    resets[0, 4] = 1
    y, final, _ = ref.gated_scan(**a, resets=resets)
    part = lambda s: {k: (v if k == "log_decay" else v[:, s]) for k, v in a.items()}  # noqa: E731
    first, second = ref.gated_scan(**part(slice(0, 4)))[0], ref.gated_scan(**part(slice(4, 9)))
    np.testing.assert_array_equal(y, np.concatenate([first, second[0]], 1))
    np.testing.assert_array_equal(final, second[1])
    cut = ref.gated_scan(**a, lengths=[5])
    np.testing.assert_array_equal(cut[0][:, :5], ref.gated_scan(**part(slice(0, 5)))[0])
    assert not cut[0][:, 5:].any()
    np.testing.assert_array_equal(cut[1], ref.gated_scan(**part(slice(0, 5)))[1])


@pytest.mark.parametrize("kind", ["none", "packed", "ragged", "both"])
def test_gated_scan_gradients_against_differences(kind):
    a, more, rng = gated(2, 7, 3, 5, kind)
    gy, gf = rng.standard_normal(a["x"].shape), rng.standard_normal(more["initial_state"].shape)
    grads = ref.gated_scan_backward(gy, **a, **more, grad_final=gf)

    def loss(**change):
        y, final, _ = ref.gated_scan(**{**a, **more, **change})
        return (y * gy).sum() + (final * gf).sum()

    for k, v in {**a, "initial_state": more["initial_state"]}.items():
        for at in [tuple(rng.integers(0, n) for n in v.shape) for _ in range(8)]:
            e = 1e-6
            up, down = v.copy(), v.copy()
            up[at] += e
            down[at] -= e
            want = (loss(**{k: up}) - loss(**{k: down})) / (2 * e)
            assert math.isclose(grads[k][at], want, rel_tol=1e-6, abs_tol=1e-7), (k, at)


def distilled(seed=0, N=2, T=3, V=11, K=5):
    rng = np.random.default_rng(seed)
    tokens = rng.integers(-1, V + 1, (N, T, K))
    tokens[..., 0] = rng.integers(0, V, (N, T))
    tokens[0, 0, 1] = tokens[0, 0, 0]   # twice
    return rng.standard_normal((N, T, V)), rng.standard_normal((N, T, K)), tokens, rng


@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
def test_distill_gradients_against_differences(tau):
    z, th, tokens, rng = distilled()
    w = rng.standard_normal(z.shape[:2])
    mask = np.ones(z.shape[:2], bool)
    mask[1, 1] = False
    _, grad, _, _ = ref.distill_loss(z, th, tokens, tau, mask, w)
    for at in [tuple(rng.integers(0, n) for n in z.shape) for _ in range(40)]:
        e = 1e-6
        up, down = z.copy(), z.copy()
        up[at] += e
        down[at] -= e
        want = ((ref.distill_loss(up, th, tokens, tau, mask)[0] - ref.distill_loss(down, th, tokens, tau, mask)[0]) * w).sum() / (2 * e)
        assert math.isclose(grad[at], want, rel_tol=1e-6, abs_tol=1e-8)


def test_distill_closed_forms():
    """A teacher that is the student over the whole vocabulary: no loss, no gradient.  One token: the
    cross entropy.  A token twice: its probability once.  Nothing left: 0."""
    rng = np.random.default_rng(2)
    z = rng.standard_normal((1, 1, 6))
    every = np.arange(6)[None, None]
    loss, grad, _, _ = ref.distill_loss(z, z, every, 1.0, None, np.ones((1, 1)))
    assert abs(loss[0, 0]) < 1e-14 and np.abs(grad).max() < 1e-14
    loss, grad, _, _ = ref.distill_loss(z, np.zeros((1, 1, 1)), np.full((1, 1, 1), 2), 1.0, None, np.ones((1, 1)))
    p = np.exp(z[0, 0]) / np.exp(z[0, 0]).sum()
    assert math.isclose(loss[0, 0], -math.log(p[2]), rel_tol=1e-12)
    np.testing.assert_allclose(grad[0, 0], p - np.eye(6)[2], atol=1e-14)
    twice = ref.distill_loss(z, np.zeros((1, 1, 2)), np.full((1, 1, 2), 2), 1.0, None, np.ones((1, 1)))
    np.testing.assert_allclose(twice[1], grad, atol=1e-14)
    assert math.isclose(twice[0][0, 0], -math.log(p[2]) - math.log(2), rel_tol=1e-12)
    none = ref.distill_loss(z, np.zeros((1, 1, 2)), np.full((1, 1, 2), -1), 1.0, None, np.ones((1, 1)))
    assert none[0][0, 0] == 0 and not none[1].any()


def test_projection_oracle_gradients_against_differences():
    """The bounds' oracle of the feed-forward block (tests/token_policy_cases.py)."""
    import torch
    from token_policy_cases import projection_inputs, projection_oracle
    x, wg, wu, gh, rng = projection_inputs(3, 5, 4, 0)

    def h(args, act):
        a, b, c = (t.double().numpy() if isinstance(t, torch.Tensor) else t for t in args)
        z = a @ b.T
        g = 1 / (1 + np.exp(-z)) if act == "silu" else 0.5 * (1 + np.vectorize(math.erf)(z / math.sqrt(2)))
        return z * g * (a @ c.T)

    for act in ("silu", "gelu"):
        want = projection_oracle(x, wg, wu, gh, act)
        np.testing.assert_allclose(want["h"][0], h((x, wg, wu), act), rtol=1e-12)
        for i, k in enumerate(("x", "gate_weight", "up_weight")):
            args = [t.double().numpy() for t in (x, wg, wu)]
            for at in [tuple(rng.integers(0, n) for n in args[i].shape) for _ in range(6)]:
                d = []
                for e in (1e-6, -1e-6):
                    moved = [v.copy() for v in args]
                    moved[i][at] += e
                    d.append((h(moved, act) * gh.double().numpy()).sum())
                assert math.isclose(want[k][0][at], (d[0] - d[1]) / 2e-6, rel_tol=1e-5, abs_tol=1e-7), (act, k, at)
