"""Inputs and error bounds the state-space layer's tests share.

u = 2^-24 is the float32 rounding unit.  Every bound is a factor times the
same formula on absolute values (``bound=True`` of the oracle), the measure
of the terms a float32 evaluation adds up:

* selective scan.  dt: the sum in front of softplus is off by u |pre|, the
  exponential's argument by another u |pre| and the functions by a few u;
  the tests keep |pre| <= 9, so dt is right to 26 u.  A step's decay
  exp(dt A) is then right to 26 u |dt A| + 5 u, and a contribution that has
  decayed by exp(-X) over n steps to (26 X + 5 n) u of itself; past X = 25 it
  no longer counts.  With 30 u of its own: scan(T) = (680 + 5 T) u.
  A gradient is a product of two such sums, summed over up to `terms`
  channels or tokens in float32: (3 (680 + 5 T) + terms) u.
* convolution.  K products and sums, a sigmoid right to 2 |pre| u + 6 u with
  |pre| <= 20, and their gradients: 64 (1 + K) u, plus u for each summed term.
* norm.  Sums of D squares in at least 32 partial sums: (D / 32 + 64) u.
* an output in bfloat16 is rounded by at most 2^-9 of itself (2^-8 where the
  two sides lie on different sides of a binade).
"""
import numpy as np
import torch

U = 2.0 ** -24
DEV = "cuda:0"


def scan_factor(T):
    return (680 + 5 * T) * U


def scan_grad_factor(T, terms):
    return (3 * (680 + 5 * T) + terms) * U


def conv_factor(K, terms=0):
    return (64 * (1 + K) + terms) * U


def norm_factor(D):
    return (D / 32 + 64) * U


def close(got, ref, mag, factor, what, sel=None):
    """|got - ref| within factor * mag, and a rounding to bfloat16 where got has that type."""
    g = got.detach().double().cpu().numpy()
    ref, mag = np.asarray(ref, np.float64), np.asarray(mag, np.float64)
    tol = factor * mag + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    assert g.shape == ref.shape, f"{what}: shape {g.shape} != {ref.shape}"
    err = np.abs(g - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: "
                           f"{g[bad][0]!r} for {ref[bad][0]!r}, allowed {tol[bad][0]:.3g}")


def np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def flags(kind, N, T, rng):
    """resets and lengths of a kind: none, packed, dense (every token), ragged (with an empty and a full row)"""
    resets = lengths = None
    if kind in ("packed", "both"):
        resets = torch.from_numpy((rng.random((N, T)) < 0.15).astype(np.uint8))
    if kind == "dense":
        resets = torch.ones(N, T, dtype=torch.uint8)
    if kind in ("ragged", "both"):
        lengths = torch.from_numpy(rng.integers(0, T + 1, N).astype(np.int32))
        lengths[0] = 0
        lengths[-1] = T
    return resets, lengths


def strided(t, pad, offset=0):
    """the same values in a wider array whose last dimension has `pad` more elements, `offset` of them in front"""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad), float("nan"), dtype=t.dtype)
    wide[..., offset:offset + t.shape[-1]] = t
    return wide.to(DEV)[..., offset:offset + t.shape[-1]]


def scan_inputs(N, T, D, S, dtype, seed, kind="none", step=False):
    rng = np.random.default_rng(seed)
    lead = (N,) if step else (N, T)

    def normal(*shape, scale=1.0, to=dtype):
        return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(to)

    f32 = torch.float32
    a = dict(x=normal(*lead, D), delta=normal(*lead, D, scale=0.7).clamp(-3, 3),
             A=-torch.from_numpy(rng.uniform(0.2, 1.0, (D, S)).astype(np.float32)) * torch.arange(1, S + 1).float(),
             B=normal(*lead, S), C=normal(*lead, S), D=normal(D, to=f32), z=normal(*lead, D, scale=1.5),
             delta_bias=torch.from_numpy(rng.uniform(-6, 1, D).astype(np.float32)))
    resets, lengths = flags(kind, N, T, rng)
    return a, normal(N, D, S, to=f32), resets, lengths, rng


def to_dev(t):
    return None if t is None else t.to(DEV)
