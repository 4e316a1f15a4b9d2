"""The state-space layer's operators in float64, one token after the other
(numpy; test infrastructure, never on the product path).

Each function follows the formulas of include/rlscan.h.  ``bound=True`` runs
the same formulas on absolute values: every sum then adds the magnitudes of
its terms, which is what a float32 evaluation's rounding errors are
proportional to.
"""
import numpy as np


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def _f64(*ts):
    return [None if t is None else np.asarray(t, np.float64) for t in ts]


def _lengths(lengths, N, T):
    return np.full(N, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True, initial_state=None,
                   resets=None, lengths=None, bound=False):
    """(y, final_state, pre-gate y, states [N,T+1,D,S] with the state before token t at t)"""
    x, delta, A, B, C, D, z, delta_bias, h = _f64(x, delta, A, B, C, D, z, delta_bias, initial_state)
    N, T, W = x.shape
    S = A.shape[1]
    m = np.abs if bound else (lambda v: v)
    dt = delta + (0 if delta_bias is None else delta_bias)
    dt = _softplus(dt) if delta_softplus else dt
    lens = _lengths(lengths, N, T)
    h = np.zeros((N, W, S)) if h is None else m(h).copy()
    states = np.zeros((N, T + 1, W, S))
    pre = np.zeros((N, T, W))
    for n in range(N):
        for t in range(T):
            states[n, t] = h[n]
            if t >= lens[n]:
                continue
            before = h[n] if resets is None or not resets[n, t] else np.zeros((W, S))
            h[n] = np.exp(dt[n, t][:, None] * A) * before + m(dt[n, t] * x[n, t])[:, None] * m(B[n, t])[None, :]
            pre[n, t] = (h[n] * m(C[n, t])[None, :]).sum(1) + (0 if D is None else m(D) * m(x[n, t]))
        states[n, T] = h[n]
    y = pre if z is None else pre * m(np.where(np.arange(T)[None, :, None] < lens[:, None, None],
                                               z * _sigmoid(z), 0.0))
    return np.where(np.arange(T)[None, :, None] < lens[:, None, None], y, 0.0), h, pre, states


def selective_scan_backward(gy, x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=True,
                            initial_state=None, resets=None, lengths=None, grad_final=None, bound=False):
    _, _, ypre, states = selective_scan(x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, resets,
                                        lengths, bound)
    gy, x, delta, A, B, C, D, z, delta_bias, gf = _f64(gy, x, delta, A, B, C, D, z, delta_bias, grad_final)
    N, T, W = x.shape
    S = A.shape[1]
    m = np.abs if bound else (lambda v: v)
    pre = delta + (0 if delta_bias is None else delta_bias)
    dt = _softplus(pre) if delta_softplus else pre
    slope = _sigmoid(pre) if delta_softplus else np.ones_like(pre)
    lens = _lengths(lengths, N, T)
    out = dict(x=np.zeros_like(x), delta=np.zeros_like(x), A=np.zeros_like(A), B=np.zeros_like(B),
               C=np.zeros_like(C), D=np.zeros(W), z=np.zeros_like(x), delta_bias=np.zeros(W),
               initial_state=np.zeros((N, W, S)))
    for n in range(N):
        G = np.zeros((W, S)) if gf is None else m(gf[n]).copy()
        for t in range(lens[n] - 1, -1, -1):
            g = m(gy[n, t])
            if z is not None:
                sg = _sigmoid(z[n, t])
                out["z"][n, t] = g * ypre[n, t] * sg * (1 + m(z[n, t]) * (1 - sg))
                g = g * m(z[n, t] * sg)
            a = np.exp(dt[n, t][:, None] * A)
            h, before = states[n, t + 1], states[n, t]
            reset = resets is not None and bool(resets[n, t])
            G = G + g[:, None] * m(C[n, t])[None, :]
            out["C"][n, t] = (g[:, None] * h).sum(0)
            dtx = m(dt[n, t] * x[n, t])
            out["B"][n, t] = (G * dtx[:, None]).sum(0)
            u = (G * m(B[n, t])[None, :]).sum(1)
            q = np.zeros_like(G) if reset else G * a * before
            if bound:  # the decay's own error, 26 units of |dt A|, does not fade where every term has decayed
                q = q * (1 + np.abs(dt[n, t][:, None] * A) / 26)
            out["A"] += q * m(dt[n, t])[:, None]
            gdt = ((q * m(A)).sum(1) + u * m(x[n, t])) * slope[n, t]
            out["delta"][n, t] = gdt
            out["delta_bias"] += gdt
            out["x"][n, t] = u * m(dt[n, t]) + (0 if D is None else g * m(D))
            out["D"] += g * m(x[n, t])
            G = np.zeros_like(G) if reset else G * a
        out["initial_state"][n] = G
    return out


def causal_conv(x, weight, bias=None, activation="silu", initial_state=None, resets=None, lengths=None, bound=False):
    """(y, final_state, the sums before the activation, [N,T,K,D] tap inputs)"""
    x, weight, bias, init = _f64(x, weight, bias, initial_state)
    N, T, W = x.shape
    K = weight.shape[1]
    m = np.abs if bound else (lambda v: v)
    lens = _lengths(lengths, N, T)
    y, pre = np.zeros((N, T, W)), np.zeros((N, T, W))
    taps = np.zeros((N, T, K, W))
    final = np.zeros((N, K - 1, W))
    for n in range(N):
        window = [np.zeros(W) if init is None else init[n, k] for k in range(K - 1)]
        for t in range(lens[n]):
            if resets is not None and resets[n, t]:
                window = [np.zeros(W)] * (K - 1)
            window = window + [x[n, t]]
            taps[n, t] = np.stack(window)
            pre[n, t] = sum(m(window[k] * weight[:, k]) for k in range(K)) + (0 if bias is None else m(bias))
            window = window[1:]
        for k in range(K - 1):
            final[n, k] = window[k]
    live = np.arange(T)[None, :, None] < lens[:, None, None]
    y = np.where(live, pre * _sigmoid(pre) if activation else pre, 0.0)
    return y, final, pre, taps


def causal_conv_backward(gy, x, weight, bias=None, activation="silu", initial_state=None, resets=None, lengths=None,
                         grad_final=None, bound=False):
    _, _, pre, taps = causal_conv(x, weight, bias, activation, initial_state, resets, lengths)
    premag = causal_conv(x, weight, bias, activation, initial_state, resets, lengths, True)[2] if bound else None
    gy, x, weight, gf = _f64(gy, x, weight, grad_final)
    N, T, W = x.shape
    K = weight.shape[1]
    m = np.abs if bound else (lambda v: v)
    lens = _lengths(lengths, N, T)
    gx = np.zeros((N, T + K - 1, W))   # positions from the initial state's first on
    gw, gb = np.zeros_like(weight), np.zeros(W)
    for n in range(N):
        since = K
        for t in range(lens[n]):
            since = 0 if resets is not None and resets[n, t] else since
            sg = _sigmoid(pre[n, t])
            slope = sg * (1 + m(pre[n, t]) * (1 - sg)) if activation else 1.0
            if bound and activation:  # what an error of the sum in front of it does, too
                slope = 1.1 * (1 + premag[n, t])
            g = m(gy[n, t]) * slope
            gb += g
            for k in range(K):
                if K - 1 - k <= since:
                    gx[n, t + k] += m(weight[:, k]) * g
                    gw[:, k] += g * m(taps[n, t, k])
            since = min(since + 1, K)
        if gf is not None:
            for k in range(K - 1):
                if resets is None or not np.any(resets[n, max(lens[n] - (K - 1) + k + 1, 0):lens[n]]):
                    gx[n, lens[n] + k] += m(gf[n, k])
    return dict(x=gx[:, K - 1:], weight=gw, bias=gb, initial_state=gx[:, :K - 1])


def add_rms_norm(x, weight, residual=None, eps=1e-6):
    x, weight, residual = _f64(x, weight, residual)
    h = x if residual is None else x + residual
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight, h


def block_scales(y, block=128, top=448.0, floor=2.0 ** -100):
    """[..., ceil(D/block)] scales of an 8-bit y"""
    D = y.shape[-1]
    parts = [np.abs(y[..., b:b + block]).max(-1) for b in range(0, D, block)]
    return np.maximum(np.stack(parts, -1), floor) / top


def add_rms_norm_backward(gy, h, weight, grad_residual=None, eps=1e-6):
    gy, h, weight, gr = _f64(gy, h, weight, grad_residual)
    D = h.shape[-1]
    r = 1 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, gn = h * r, gy * weight
    gh = r * (gn - n * (gn * n).sum(-1, keepdims=True) / D)
    if gr is not None:
        gh = gh + gr
    return dict(x=gh, weight=(gy * n).reshape(-1, D).sum(0))
