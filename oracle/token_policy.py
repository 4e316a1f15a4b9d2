"""The token policy's gated recurrence in float64, one token after the other
(numpy; test infrastructure, never on the product path).

The functions follow the formulas of include/rlscan.h.  ``bound=True`` runs
the same formulas on absolute values: every sum then adds the magnitudes of
its terms, which is what a float32 evaluation's rounding errors are
proportional to.
"""
import numpy as np

from .state_space import _f64, _lengths, _sigmoid


def _gates(gate, input_gate, log_decay):
    r, i = _sigmoid(gate), _sigmoid(input_gate)
    L = log_decay * r
    return r, i, np.exp(L), np.sqrt(-np.expm1(2 * L))


def gated_scan(x, gate, input_gate, log_decay, initial_state=None, resets=None, lengths=None, bound=False):
    """(y, final_state, states [N,T+1,D] with the state before token t at t)"""
    x, gate, input_gate, log_decay, h = _f64(x, gate, input_gate, log_decay, initial_state)
    N, T, D = x.shape
    m = np.abs if bound else (lambda v: v)
    _, i, a, root = _gates(gate, input_gate, log_decay)
    b = m(root * i * x)
    lens = _lengths(lengths, N, T)
    h = np.zeros((N, D)) if h is None else m(h).copy()
    states, y = np.zeros((N, T + 1, D)), np.zeros((N, T, D))
    for t in range(T):
        states[:, t] = h
        on = (t < lens)[:, None]
        start = h if resets is None else np.where(np.asarray(resets)[:, t, None] != 0, 0.0, h)
        h = np.where(on, a[:, t] * start + b[:, t], h)
        y[:, t] = np.where(on, h, 0.0)
    states[:, T] = h
    return y, h, states


def gated_scan_backward(gy, x, gate, input_gate, log_decay, initial_state=None, resets=None, lengths=None,
                        grad_final=None, bound=False):
    _, _, states = gated_scan(x, gate, input_gate, log_decay, initial_state, resets, lengths, bound)
    gy, x, gate, input_gate, log_decay, G = _f64(gy, x, gate, input_gate, log_decay, grad_final)
    N, T, D = x.shape
    m = np.abs if bound else (lambda v: v)
    minus = 1.0 if bound else -1.0
    r, i, a, root = _gates(gate, input_gate, log_decay)
    lens = _lengths(lengths, N, T)
    G = np.zeros((N, D)) if G is None else m(G).copy()
    out = dict(x=np.zeros_like(x), gate=np.zeros_like(x), input_gate=np.zeros_like(x), log_decay=np.zeros(D))
    for t in range(T - 1, -1, -1):
        on = (t < lens)[:, None]
        cut = np.zeros((N, 1), bool) if resets is None else np.asarray(resets)[:, t, None] != 0
        total = G + m(gy[:, t])
        out["x"][:, t] = np.where(on, total * root[:, t] * i[:, t], 0)
        out["input_gate"][:, t] = np.where(on, total * root[:, t] * m(x[:, t]) * i[:, t] * (1 - i[:, t]), 0)
        dL = total * (a[:, t] * np.where(cut, 0.0, states[:, t]) + minus * i[:, t] * m(x[:, t]) * a[:, t] ** 2 / root[:, t])
        out["gate"][:, t] = np.where(on, dL * m(log_decay) * r[:, t] * (1 - r[:, t]), 0)
        out["log_decay"] += np.where(on, dL * r[:, t], 0).sum(0)
        G = np.where(on, np.where(cut, 0.0, a[:, t] * total), G)
    out["initial_state"] = G
    return out


def distill_loss(logits, teacher_logits, teacher_tokens, temperature=1.0, mask=None, grad_loss=None):
    """(loss [N,T], gradient [N,T,V] or None, the terms' magnitude for each of both)"""
    logits, teacher = _f64(logits, teacher_logits)
    N, T, V = logits.shape
    K = teacher.shape[2]
    loss, mag = np.zeros((N, T)), np.zeros((N, T))
    grad = gmag = None
    if grad_loss is not None:
        grad, gmag = np.zeros((N, T, V)), np.zeros((N, T, V))
    for n in range(N):
        for t in range(T):
            if mask is not None and not mask[n, t]:
                continue
            ok = (teacher_tokens[n, t] >= 0) & (teacher_tokens[n, t] < V)
            with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
                th = np.where(ok, teacher[n, t], -np.inf) / temperature
                if (th == -np.inf).all():
                    continue
                lq = th - th.max()
                lq = lq - np.log(np.exp(lq).sum())
                q = np.exp(lq)
                z = (logits[n, t] - logits[n, t].max()) / temperature
                e = np.exp(z)
                p = e / e.sum()
                for k in range(K):
                    if q[k] != 0:
                        zk = z[teacher_tokens[n, t, k]]
                        loss[n, t] += q[k] * (lq[k] - zk + np.log(e.sum()))
                        mag[n, t] += q[k] * (abs(lq[k]) + abs(zk) + np.log(e.sum()) + 1)
                if grad is not None:
                    w = grad_loss[n, t] / temperature
                    grad[n, t], gmag[n, t] = p * w, p * abs(w)
                    for k in range(K):
                        if ok[k]:
                            grad[n, t, teacher_tokens[n, t, k]] -= q[k] * w
                            gmag[n, t, teacher_tokens[n, t, k]] += q[k] * abs(w)
    return loss, grad, mag, gmag
