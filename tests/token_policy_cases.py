"""Inputs and error bounds the tests of the token policy's operators share.

u = 2^-24 is the float32 rounding unit; every bound is a factor times the
formula on absolute values (``bound=True`` of the oracle).

* gated scan, gate values within 4 of 0.  exp(-v) is right to (|v| + 2) u, so
  a sigmoid to (|v| + 2) u e / (1 + e) + 2 u <= 14 u, the exponent L =
  log_decay r to 15 u and a = exp(L) to (15 |L| + 5) u.  1 - a^2 is its series
  to 25 u, or beyond |2 L| = 1/4, where a^2 <= 0.78, to 2 (15 |L| + 5) u a^2 /
  (1 - a^2) <= 55 u; its root to 30 u, and root i x to 50 u.  A contribution
  that has decayed by exp(-X) over n steps is right to (15 X + 6 n) u of
  itself, and past X = 25 it no longer counts: gated(T) = (430 + 6 T) u.
  A gradient multiplies two such sums; a^2 / root adds 2 (15 |L| + 5) + 32 u
  (|L| <= 5 here: 192 u), 1 - r, whose r is right to 3 u where it is near 1,
  another 3 u / (1 - r) <= 165 u and its factors 20 u; a sum over `terms`
  tokens in float32 adds as many u: (2 (430 + 6 T) + 400 + terms) u.
* distillation.  With X the largest difference of two logits (the student's
  or the teacher's) over the temperature, an exponent is right to 2 X u and an
  exponential to (2 X + 4) u, a softmax to twice that and its sum's rounding:
  a thread adds at most V / 32 values one after the other, in four sums at
  once, lanes and warps another 60.  Products and logarithms add 20 u, sums
  over the K tokens K u: (4 X + 100 + V / 32 + K) u of the terms' magnitude.
* an output in bfloat16 is rounded by at most 2^-9 of itself (2^-8 where the
  two sides lie on different sides of a binade).
"""
import numpy as np
import torch

from state_space_cases import U, flags


def gated_factor(T):
    return (430 + 6 * T) * U


def gated_grad_factor(T, terms=0):
    return (2 * (430 + 6 * T) + 400 + terms) * U


def gated_inputs(N, T, D, dtype, seed, kind="none", step=False, strongest=5.0):
    """x, both gates, log_decay between -strongest and -1e-4; initial state, resets, lengths, the generator"""
    rng = np.random.default_rng(seed)
    lead = (N,) if step else (N, T)

    def normal(*shape, scale=1.0, to=dtype):
        return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(to)

    a = dict(x=normal(*lead, D), gate=normal(*lead, D, scale=1.3).clamp(-4, 4),
             input_gate=normal(*lead, D, scale=1.3).clamp(-4, 4),
             log_decay=-torch.from_numpy(np.exp(rng.uniform(np.log(1e-4), np.log(strongest), D)).astype(np.float32)))
    resets, lengths = flags(kind, N, T, rng)
    return a, normal(N, D, to=torch.float32), resets, lengths, rng


def distill_factor(V, K, spread):
    return (4 * spread + 100 + V / 32 + K) * U


def distill_inputs(N, T, V, K, dtype, seed, teacher_dtype=torch.float32, token_dtype=torch.int64):
    """logits, the teacher's logits and tokens (some empty, some twice), a mask, grad_loss, the generator"""
    rng = np.random.default_rng(seed)
    tokens = rng.integers(0, V, (N, T, K))
    tokens[rng.random((N, T, K)) < 0.1] = -1
    tokens[rng.random((N, T, K)) < 0.03] = V
    tokens[..., 0] = rng.integers(0, V, (N, T))
    logits = torch.from_numpy((2 * rng.standard_normal((N, T, V))).astype(np.float32)).to(dtype)
    teacher = torch.from_numpy((2 * rng.standard_normal((N, T, K))).astype(np.float32)).to(teacher_dtype)
    mask = torch.from_numpy((rng.random((N, T)) < 0.8).astype(np.uint8))
    grad = torch.from_numpy(rng.standard_normal((N, T)).astype(np.float32))
    return logits, teacher, torch.from_numpy(tokens).to(token_dtype), mask, grad, rng


def projection_inputs(M, D, F, seed, scale=1.0):
    """x, both weights, grad_h in bfloat16, the generator"""
    rng = np.random.default_rng(seed)

    def normal(*shape, s=1.0):
        return torch.from_numpy((rng.standard_normal(shape) * s).astype(np.float32)).to(torch.bfloat16)

    return normal(M, D, s=scale), normal(F, D, s=D ** -0.5), normal(F, D, s=D ** -0.5), normal(M, F), rng


def projection_oracle(x, wg, wu, gh, act):
    """name -> (value, bound in front of the last rounding), float64.

    A sum of n products in the tensor cores is right to 2 n u of its terms'
    magnitude (each of n additions is off by less than a step, 2 u); an
    activation and its slope move by at most 1.13 and 0.8 of z's error and are
    right to 40 u of themselves (a sigmoid to (2 |z| + 6) u, |z| <= 17); gz and
    gu are rounded by 2^-8 of themselves for the products that follow."""
    x, wg, wu, gh = (np.asarray(t.float().numpy(), np.float64) for t in (x, wg, wu, gh))
    n = lambda k: 2 * (k + 8) * U  # noqa: E731
    z, u = x @ wg.T, x @ wu.T
    ez, eu = (n(x.shape[1]) * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
    if act == "silu":
        g = 1 / (1 + np.exp(-z))
        a, s = z * g, g * (1 + z * (1 - g))
    else:
        from scipy.special import ndtr
        g = ndtr(z)
        a, s = z * g, g + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    ea = 1.13 * ez + 40 * U * np.abs(a)
    es = 0.8 * ez + 40 * U * (1 + np.abs(z) * 0)
    h, gz, gu = a * u, gh * u * s, gh * a
    r = 2.0 ** -8
    egz = np.abs(gh) * (np.abs(s) * eu + np.abs(u) * es) + r * np.abs(gz) + 1e-30
    egu = np.abs(gh) * ea + r * np.abs(gu) + 1e-30
    F, M = wg.shape[0], x.shape[0]
    return dict(
        h=(h, np.abs(u) * ea + np.abs(a) * eu + 4 * U * np.abs(h)),
        x=(gz @ wg + gu @ wu, egz @ np.abs(wg) + egu @ np.abs(wu) + n(2 * F) * (np.abs(gz) @ np.abs(wg) + np.abs(gu) @ np.abs(wu))),
        gate_weight=(gz.T @ x, egz.T @ np.abs(x) + n(M) * (np.abs(gz).T @ np.abs(x))),
        up_weight=(gu.T @ x, egu.T @ np.abs(x) + n(M) * (np.abs(gu).T @ np.abs(x))))
