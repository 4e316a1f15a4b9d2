"""The state-space layer on the GPU against its float64 oracle: sizes where
tiles, lanes and vectors end, both types, strides and alignments, episode
flags, padding, empty rows, idle slots, states that do not fit 32-bit offsets.
The bounds are derived in state_space_cases.py."""
import numpy as np
import pytest
import torch

from oracle import state_space as ref
from state_space_cases import (DEV, U, close, conv_factor, flags, norm_factor, np64, scan_factor, scan_grad_factor,
                               scan_inputs, strided, to_dev)

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


# N, T, D, S: single values, one lane to a whole warp a channel, tails of every tile, more than one segment
SCAN_SIZES = [(1, 1, 1, 1), (2, 5, 33, 16), (1, 17, 128, 16), (3, 64, 40, 8), (2, 33, 7, 12), (1, 130, 65, 16),
              (2, 50, 24, 32), (1, 40, 12, 128), (1, 20, 3, 3), (2, 16, 64, 64), (1, 15, 260, 5), (4, 37, 16, 16)]


@pytest.mark.parametrize("kind", ["none", "packed", "ragged", "dense", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D,S", SCAN_SIZES)
def test_scan_forward_and_gradients(N, T, D, S, dtype, kind):
    a, init, resets, lengths, rng = scan_inputs(N, T, D, S, dtype, N + 10 * T + 100 * D + S, kind)
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gf = torch.from_numpy(rng.standard_normal((N, D, S)).astype(np.float32))
    r64 = {k: np64(v) for k, v in a.items()}
    rs, ln = (None if f is None else f.numpy() for f in (resets, lengths))
    dev = {k: v.to(DEV) for k, v in a.items()}
    y, final, marks = L().selective_scan(**dev, initial_state=to_dev(init), resets=to_dev(resets),
                                         lengths=to_dev(lengths), return_checkpoints=True)
    args = dict(initial_state=np64(init), resets=rs, lengths=ln)
    ry, rf, _, _ = ref.selective_scan(**r64, **args)
    my, mf, _, _ = ref.selective_scan(**r64, **args, bound=True)
    close(y, ry, my, scan_factor(T), "y")
    close(final, rf, mf, scan_factor(T), "final state")
    g = L().selective_scan_backward(gy.to(DEV), dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks, dev["D"],
                                    dev["z"], dev["delta_bias"], resets=to_dev(resets), lengths=to_dev(lengths),
                                    grad_final_state=to_dev(gf))
    want = ref.selective_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf))
    mag = ref.selective_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf), bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], scan_grad_factor(T, max(D, N * T)), "gradient of " + k)
    # the same bits again
    again = L().selective_scan_backward(gy.to(DEV), dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks,
                                        dev["D"], dev["z"], dev["delta_bias"], resets=to_dev(resets),
                                        lengths=to_dev(lengths), grad_final_state=to_dev(gf))
    for p, q in zip(g, again):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D,S", [(40, 21, 520, 16), (64, 18, 700, 16), (33, 9, 1300, 8), (65, 7, 400, 16)])
def test_scan_rows_in_the_order_of_their_lengths(N, T, D, S, dtype):
    """More blocks than SMs, up to and over two an SM: rows change places, equal and empty ones too."""
    test_scan_forward_and_gradients(N, T, D, S, dtype, "ragged")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(700, 64), (2100, 24), (1030, 7)])
def test_scan_long_rows(T, D, dtype):
    """Few channels and many tokens: rows that are split along the tokens."""
    N, S = 2, 16
    a, init, resets, lengths, rng = scan_inputs(N, T, D, S, dtype, T, "none")
    resets = torch.from_numpy((rng.random((N, T)) < 0.004).astype(np.uint8))
    resets[0] = 0
    lengths = torch.tensor([T, T - T // 3], dtype=torch.int32)
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gf = torch.from_numpy(rng.standard_normal((N, D, S)).astype(np.float32))
    r64 = {k: np64(v) for k, v in a.items()}
    dev = {k: v.to(DEV) for k, v in a.items()}
    args = dict(initial_state=np64(init), resets=resets.numpy(), lengths=lengths.numpy())
    y, final, marks = L().selective_scan(**dev, initial_state=to_dev(init), resets=to_dev(resets),
                                         lengths=to_dev(lengths), return_checkpoints=True)
    ry, rf, _, _ = ref.selective_scan(**r64, **args)
    my, mf, _, _ = ref.selective_scan(**r64, **args, bound=True)
    close(y, ry, my, scan_factor(T), "y")
    close(final, rf, mf, scan_factor(T), "final state")
    plain, pf = L().selective_scan(**dev, initial_state=to_dev(init), resets=to_dev(resets), lengths=to_dev(lengths))
    close(plain, ry, my, scan_factor(T), "y without checkpoints")
    close(pf, rf, mf, scan_factor(T), "final state without checkpoints")
    g = L().selective_scan_backward(gy.to(DEV), dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks, dev["D"],
                                    dev["z"], dev["delta_bias"], resets=to_dev(resets), lengths=to_dev(lengths),
                                    grad_final_state=to_dev(gf))
    want = ref.selective_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf))
    mag = ref.selective_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf), bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], scan_grad_factor(T, max(D, N * T)), "gradient of " + k)


@pytest.mark.parametrize("with_d", [True, False])
@pytest.mark.parametrize("with_z", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_optional_arguments(with_d, with_z, with_bias, softplus):
    N, T, D, S = 2, 35, 48, 16
    a, _, _, _, rng = scan_inputs(N, T, D, S, F32, 5)
    if not softplus:
        a["delta"] = a["delta"].abs() * 0.1
        a["delta_bias"] = a["delta_bias"].abs() * 0.01
    for k, on in (("D", with_d), ("z", with_z), ("delta_bias", with_bias)):
        a[k] = a[k] if on else None
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32))
    r64 = {k: np64(v) for k, v in a.items()}
    dev = {k: to_dev(v) for k, v in a.items()}
    y, final, marks = L().selective_scan(**dev, delta_softplus=softplus, return_checkpoints=True)
    ry, rf, _, _ = ref.selective_scan(**r64, delta_softplus=softplus)
    my, mf, _, _ = ref.selective_scan(**r64, delta_softplus=softplus, bound=True)
    close(y, ry, my, scan_factor(T), "y")
    close(final, rf, mf, scan_factor(T), "final state")
    g = L().selective_scan_backward(gy.to(DEV), dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks, dev["D"],
                                    dev["z"], dev["delta_bias"], softplus)
    want = ref.selective_scan_backward(np64(gy), **r64, delta_softplus=softplus)
    mag = ref.selective_scan_backward(np64(gy), **r64, delta_softplus=softplus, bound=True)
    for k in want:
        if k in a and a[k] is None:
            assert getattr(g, k) is None
        else:
            close(getattr(g, k), want[k], mag[k], scan_grad_factor(T, N * T), "gradient of " + k)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(64, 0), (16, 16), (1, 1), (3, 0), (8, 4)])
def test_scan_strides_and_alignments(pad, offset, dtype):
    """Slices of wider arrays (NaN around them) give the dense arrays' bits."""
    N, T, D, S = 2, 45, 96, 16
    a, init, resets, _, rng = scan_inputs(N, T, D, S, dtype, 6, "packed")
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    dense = {k: v.to(DEV) for k, v in a.items()}
    views = dict(dense)
    for k in ("x", "delta", "z", "B", "C"):
        views[k] = strided(a[k], pad, offset)
    outs = []
    for d, g in ((dense, gy.to(DEV)), (views, strided(gy, pad, offset))):
        y, final, marks = L().selective_scan(**d, initial_state=to_dev(init), resets=to_dev(resets),
                                             return_checkpoints=True)
        grads = L().selective_scan_backward(g, d["x"], d["delta"], d["A"], d["B"], d["C"], marks, d["D"], d["z"],
                                            d["delta_bias"], resets=to_dev(resets))
        outs.append((y, final, *grads))
    for p, q in zip(*outs):
        assert torch.equal(p, q)


def test_scan_broadcast_inputs():
    """Strides of 0: one row of B and C for all rows, one token's delta for all tokens."""
    N, T, D, S = 3, 40, 32, 16
    a, _, _, _, _ = scan_inputs(N, T, D, S, F32, 7)
    dev = {k: v.to(DEV) for k, v in a.items()}
    dev["B"], dev["C"] = dev["B"][:1].expand(N, T, S), dev["C"][:1].expand(N, T, S)
    dev["delta"] = dev["delta"][:, :1].expand(N, T, D)
    y, final = L().selective_scan(**dev)
    y2, final2 = L().selective_scan(**{k: v.contiguous() for k, v in dev.items()})
    assert torch.equal(y, y2) and torch.equal(final, final2)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scan_masked_places_may_hold_anything(dtype):
    """Padding holds NaN and infinities; an episode's infinities end at a reset."""
    N, T, D, S = 2, 50, 40, 16
    a, init, _, _, rng = scan_inputs(N, T, D, S, dtype, 8)
    lengths = torch.tensor([20, 0], dtype=torch.int32)
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    clean = {k: v.to(DEV) for k, v in a.items()}
    dirty = dict(clean)
    for k in ("x", "delta", "z", "B", "C"):
        v = a[k].clone()
        v[0, 20:] = float("nan")
        v[1] = float("inf")
        v[1, ::2] = torch.finfo(dtype).min
        dirty[k] = v.to(DEV)
    bad_gy = gy.clone()
    bad_gy[0, 20:] = float("inf")
    bad_gy[1] = float("nan")
    outs = []
    for d, g in ((clean, gy), (dirty, bad_gy)):
        y, final, marks = L().selective_scan(**d, initial_state=to_dev(init), lengths=to_dev(lengths),
                                             return_checkpoints=True)
        grads = L().selective_scan_backward(g.to(DEV), d["x"], d["delta"], d["A"], d["B"], d["C"], marks, d["D"],
                                            d["z"], d["delta_bias"], lengths=to_dev(lengths))
        outs.append((y, final, *grads))
    for p, q in zip(*outs):
        assert torch.equal(p, q)
    assert not outs[1][0][0, 20:].any() and not outs[1][0][1].any()
    assert torch.equal(outs[1][1][1], init[1].to(DEV))   # an empty row hands its state through
    # the episode before a reset overflows; what follows is as if it began there
    v = a["x"].clone()
    v[:, 10] = float("inf")
    resets = torch.zeros(N, T, dtype=torch.uint8)
    resets[:, 11] = 1
    y, final = L().selective_scan(**{**clean, "x": v.to(DEV)}, resets=to_dev(resets))
    tail = {k: (t[:, 11:] if k in ("x", "delta", "z", "B", "C") else t) for k, t in clean.items()}
    y2, final2 = L().selective_scan(**tail)
    assert not torch.isfinite(y[:, 10].float()).all() and torch.isfinite(y[:, 11:].float()).all()
    mag = np.abs(np64(y2)) + 1
    close(y[:, 11:].contiguous(), np64(y2), mag, 50 * scan_factor(T), "after the reset")
    close(final, np64(final2), np.abs(np64(final2)) + 1, scan_factor(T), "final state after the reset")


@pytest.mark.parametrize("T,n", [(20, 17), (64, 33), (250, 1)])
def test_scan_padding_leaves_the_state(T, n):
    """A padded row's states and outputs are the shorter call's, bit for bit."""
    a, init, _, _, _ = scan_inputs(1, T, 48, 16, F32, 22)
    dev = {k: v.to(DEV) for k, v in a.items()}
    lengths = torch.tensor([n], dtype=torch.int32).to(DEV)
    y, final = L().selective_scan(**dev, initial_state=to_dev(init), lengths=lengths)
    head = {k: (t[:, :n] if k in ("x", "delta", "z", "B", "C") else t) for k, t in dev.items()}
    y2, final2 = L().selective_scan(**head, initial_state=to_dev(init))
    assert torch.equal(y[:, :n], y2) and torch.equal(final, final2) and not y[:, n:].any()


def test_scan_no_tokens_and_no_rows():
    a, init, _, _, _ = scan_inputs(2, 1, 8, 4, F32, 9)
    none = {k: (v[:, :0] if k in ("x", "delta", "z", "B", "C") else v).to(DEV) for k, v in a.items()}
    y, final, marks = L().selective_scan(**none, initial_state=to_dev(init), return_checkpoints=True)
    assert y.shape == (2, 0, 8) and torch.equal(final.cpu(), init) and marks.shape[1] == 0
    g = L().selective_scan_backward(none["x"], none["x"], none["delta"], none["A"], none["B"], none["C"], marks,
                                    none["D"], none["z"], none["delta_bias"], grad_final_state=final)
    assert torch.equal(g.initial_state, final) and not g.A.any() and not g.D.any() and not g.delta_bias.any()
    rows = {k: (v[:0] if k in ("x", "delta", "z", "B", "C") else v).to(DEV) for k, v in a.items()}
    y, final, marks = L().selective_scan(**rows, return_checkpoints=True)
    assert y.shape == (0, 1, 8) and final.shape == (0, 8, 4)
    g = L().selective_scan_backward(rows["x"], rows["x"], rows["delta"], rows["A"], rows["B"], rows["C"], marks,
                                    rows["D"], rows["z"], rows["delta_bias"])
    assert not g.A.any() and not g.D.any() and not g.delta_bias.any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,D,S", [(1, 1, 1), (1, 1536, 16), (3, 33, 16), (5, 40, 8), (2, 7, 12), (2, 24, 32),
                                   (2, 12, 128), (4, 130, 3), (3, 17, 64), (65, 64, 16)])
@pytest.mark.parametrize("slotted", [True, False])
def test_scan_step(N, D, S, dtype, slotted):
    a, _, _, _, rng = scan_inputs(N, 1, D, S, dtype, 10 + N + D, step=True)
    P = N + 3
    state = torch.from_numpy(rng.standard_normal((P, D, S)).astype(np.float32))
    slots = torch.from_numpy(rng.permutation(P)[:N].astype(np.int32)) if slotted else None
    if slotted and N > 1:
        slots[0], slots[N // 2] = -1, P + 5   # idle
    st = state.to(DEV)
    y = L().selective_scan_step(st, **{k: v.to(DEV) for k, v in a.items()}, slots=to_dev(slots))
    r64 = {k: (np64(v)[:, None] if k in ("x", "delta", "z", "B", "C") else np64(v)) for k, v in a.items()}
    at = np.arange(N) if slots is None else slots.numpy()
    idle = (at < 0) | (at >= P)
    old = np64(state)[np.where(idle, 0, at)]
    ry, rf, _, _ = ref.selective_scan(**r64, initial_state=old)
    my, mf, _, _ = ref.selective_scan(**r64, initial_state=old, bound=True)
    ry[idle] = 0
    close(y, ry[:, 0], my[:, 0], scan_factor(1), "y")
    want, mag = np64(state), np.abs(np64(state))
    for n in range(N):
        if not idle[n]:
            want[at[n]], mag[at[n]] = rf[n], mf[n]
    close(st, want, mag, scan_factor(1), "state")
    untouched = np.setdiff1d(np.arange(P), at)
    assert np.array_equal(st.cpu().numpy()[untouched], state.numpy()[untouched])


def test_step_by_step_is_the_prompt():
    """T tokens one at a time (convolution and scan) against the two prompt calls."""
    N, T, D, S, K = 3, 12, 64, 16, 4
    a, init, _, _, rng = scan_inputs(N, T, D, S, F32, 11)
    w = torch.from_numpy(rng.standard_normal((D, K)).astype(np.float32)).to(DEV)
    dev = {k: v.to(DEV) for k, v in a.items()}
    x, conv_final = L().causal_conv(dev["x"], w)
    y, final = L().selective_scan(**{**dev, "x": x}, initial_state=to_dev(init))
    window, state = torch.zeros(N, K - 1, D, device=DEV), init.to(DEV)
    for t in range(T):
        at = {k: (v[:, t] if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
        xt = L().causal_conv_step(window, dev["x"][:, t], w)
        yt = L().selective_scan_step(state, **{**at, "x": xt})
        close(xt, np64(x[:, t]), np.abs(np64(x[:, t])) + 1, conv_factor(K), "convolution")
        close(yt, np64(y[:, t]), np.abs(np64(y[:, t])) + 10, scan_factor(T), "scan")
    assert torch.equal(window, conv_final)
    close(state, np64(final), np.abs(np64(final)) + 1, scan_factor(T), "state")


CONV_SIZES = [(1, 1, 1, 4), (2, 5, 33, 4), (1, 64, 128, 4), (3, 40, 7, 3), (2, 100, 65, 2), (1, 33, 40, 1), (2, 3, 24, 8),
              (1, 150, 12, 5), (2, 70, 256, 4), (4, 31, 130, 4)]


@pytest.mark.parametrize("kind", ["none", "packed", "ragged", "dense", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D,K", CONV_SIZES)
def test_conv_forward_and_gradients(N, T, D, K, dtype, kind):
    rng = np.random.default_rng(N + 10 * T + 100 * D + K)

    def normal(*shape, to=dtype):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(to)

    x, w, b = normal(N, T, D), normal(D, K, to=F32), normal(D, to=F32)
    init, gy, gf = normal(N, K - 1, D), normal(N, T, D), normal(N, K - 1, D)
    resets, lengths = flags(kind, N, T, rng)
    extra = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    rextra = dict(resets=None if resets is None else resets.numpy(), lengths=None if lengths is None else lengths.numpy())
    for activation, state, bias in (("silu", init, b), (None, None, None)):
        y, final = L().causal_conv(x.to(DEV), w.to(DEV), to_dev(bias), activation, to_dev(state), **extra)
        args = (np64(x), np64(w), np64(bias), activation, np64(state))
        ry, rf, _, _ = ref.causal_conv(*args, **rextra)
        _, _, mag, _ = ref.causal_conv(*args, **rextra, bound=True)
        close(y, ry, mag, conv_factor(K), "y")
        assert np.array_equal(np64(final), rf)
        g = L().causal_conv_backward(gy.to(DEV), x.to(DEV), w.to(DEV), to_dev(bias), activation, to_dev(state), **extra,
                                     grad_final_state=gf.to(DEV))
        want = ref.causal_conv_backward(np64(gy), *args, **rextra, grad_final=np64(gf))
        mag = ref.causal_conv_backward(np64(gy), *args, **rextra, grad_final=np64(gf), bound=True)
        for k in want:
            if k == "bias" and bias is None:
                assert g.bias is None
            else:
                close(getattr(g, k), want[k], mag[k], conv_factor(K, N * T), "gradient of " + k)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(64, 0), (16, 16), (1, 1), (3, 0), (8, 4)])
def test_conv_strides_and_alignments(pad, offset, dtype):
    rng = np.random.default_rng(12)
    N, T, D, K = 2, 90, 96, 4
    x = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    w = torch.from_numpy(rng.standard_normal((D, K)).astype(np.float32)).to(DEV)
    outs = []
    for xv, gv in ((x.to(DEV), gy.to(DEV)), (strided(x, pad, offset), strided(gy, pad, offset))):
        y, final = L().causal_conv(xv, w)
        outs.append((y, final, *[t for t in L().causal_conv_backward(gv, xv, w) if t is not None]))
    for p, q in zip(*outs):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_conv_masked_places_may_hold_anything(dtype):
    rng = np.random.default_rng(13)
    N, T, D, K = 2, 70, 40, 4
    x = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    w = torch.from_numpy(rng.standard_normal((D, K)).astype(np.float32)).to(DEV)
    lengths = torch.tensor([33, 0], dtype=torch.int32).to(DEV)
    outs = []
    for bad in (0.0, float("nan")):
        xv, gv = x.clone(), gy.clone()
        for v in (xv, gv):
            v[0, 33:] = bad
            v[1] = bad
        y, final = L().causal_conv(xv.to(DEV), w, lengths=lengths)
        outs.append((y, final, *[t for t in L().causal_conv_backward(gv.to(DEV), xv.to(DEV), w, lengths=lengths)
                                 if t is not None]))
    for p, q in zip(*outs):
        assert torch.equal(p, q)
    xv = x.clone()
    xv[:, 9] = float("inf")
    resets = torch.zeros(N, T, dtype=torch.bool)
    resets[:, 10] = True
    y, _ = L().causal_conv(xv.to(DEV), w, resets=resets.to(DEV))
    y2, _ = L().causal_conv(x[:, 10:].to(DEV), w)
    assert torch.equal(y[:, 10:], y2)


def test_conv_no_tokens():
    w, init = torch.ones(8, 4, device=DEV), torch.randn(2, 3, 8, device=DEV)
    x = torch.zeros(2, 0, 8, device=DEV)
    y, final = L().causal_conv(x, w, initial_state=init)
    assert y.shape == (2, 0, 8) and torch.equal(final, init)
    g = L().causal_conv_backward(x, x, w, initial_state=init, grad_final_state=init)
    assert torch.equal(g.initial_state, init) and not g.weight.any()
    g = L().causal_conv_backward(x[:0], x[:0], w)
    assert not g.weight.any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,D,K", [(1, 1, 4), (3, 33, 4), (5, 256, 3), (2, 130, 2), (2, 24, 1), (2, 40, 8), (64, 64, 4)])
def test_conv_step(N, D, K, dtype):
    rng = np.random.default_rng(14 + N + D + K)

    def normal(*shape, to=dtype):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(to)

    P = N + 2
    state, x, w, b = normal(P, K - 1, D), normal(N, D), normal(D, K, to=F32), normal(D, to=F32)
    slots = torch.from_numpy(rng.permutation(P)[:N].astype(np.int32))
    if N > 1:
        slots[0], slots[N // 2] = -1, P
    st = state.to(DEV)
    y = L().causal_conv_step(st, x.to(DEV), w.to(DEV), b.to(DEV), slots=slots.to(DEV))
    at = slots.numpy()
    idle = (at < 0) | (at >= P)
    old = np64(state)[np.where(idle, 0, at)]
    ry, rf, _, _ = ref.causal_conv(np64(x)[:, None], np64(w), np64(b), initial_state=old)
    _, _, mag, _ = ref.causal_conv(np64(x)[:, None], np64(w), np64(b), initial_state=old, bound=True)
    ry[idle] = 0
    close(y, ry[:, 0], mag[:, 0], conv_factor(K), "y")
    want = np64(state)
    want[at[~idle]] = rf[~idle]
    assert np.array_equal(np64(st), want)


NORM_SIZES = [(1, 1), (3, 33), (5, 128), (2, 129), (4, 1000), (130, 64), (7, 2560), (2, 4096), (1, 9000), (3, 20000)]


@pytest.mark.parametrize("rtype", [None, F32, BF16], ids=["plain", "res32", "res16"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", NORM_SIZES)
def test_norm_forward_and_gradients(M, D, dtype, rtype):
    if dtype == F32 and rtype == BF16:
        return
    rng = np.random.default_rng(M + 10 * D)

    def normal(*shape, to=dtype):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(to)

    x, w, gy = normal(M, D), 1 + 0.3 * normal(D, to=F32), normal(M, D)
    r = None if rtype is None else 2 * normal(M, D, to=rtype)
    out = L().add_rms_norm(x.to(DEV), w.to(DEV), to_dev(r), eps=1e-5)
    ry, rh = ref.add_rms_norm(np64(x), np64(w), np64(r), 1e-5)
    hmag = np.abs(np64(x)) + (0 if r is None else np.abs(np64(r)))
    # an error of u (|x| + |r|) in h is one of that share in y
    scale = np.abs(ry) + hmag * np.abs(np64(w)) / np.sqrt((rh * rh).mean(-1, keepdims=True) + 1e-5)
    close(out.y, ry, scale, norm_factor(D), "y")
    assert out.scales is None
    if r is None:
        assert out.residual is None
    else:
        assert out.residual.dtype == rtype
        close(out.residual, rh, hmag, 2 * U, "sum")
    h = x.to(DEV) if r is None else out.residual
    gr = None if r is None else normal(M, D, to=rtype)
    g = L().add_rms_norm_backward(gy.to(DEV), h, w.to(DEV), to_dev(gr), eps=1e-5)
    h64, w64, gy64 = np64(h), np64(w), np64(gy)
    want = ref.add_rms_norm_backward(gy64, h64, w64, np64(gr), 1e-5)
    inv = 1 / np.sqrt((h64 * h64).mean(-1, keepdims=True) + 1e-5)
    n, gn = np.abs(h64 * inv), np.abs(gy64 * w64)
    mag = inv * (gn + n * (gn * n).mean(-1, keepdims=True)) + (0 if gr is None else np.abs(np64(gr)))
    close(g.x, want["x"], mag, 2 * norm_factor(D), "gradient of x")
    close(g.residual, want["x"], mag, 2 * norm_factor(D), "gradient of the residual")
    close(g.weight, want["weight"], np.abs(gy64 * h64 * inv).sum(0), 2 * norm_factor(D) + M * U, "gradient of weight")


@pytest.mark.parametrize("rtype", [None, F32, BF16], ids=["plain", "res32", "res16"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("M,D", NORM_SIZES)
def test_norm_eight_bits(M, D, dtype, rtype):
    """Scales to the norm's bound; a stored value to half a step of e4m3:
    2^-4 of itself, or 2^-10 of its scale where it is subnormal."""
    if dtype == F32 and rtype == BF16:
        return
    rng = np.random.default_rng(M + 10 * D + 1)
    x = torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).to(dtype)
    x[M // 2, : min(D, 128)] = 0     # a block of zeros
    w = torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32))
    r = None if rtype is None else torch.from_numpy(rng.standard_normal((M, D)).astype(np.float32)).to(rtype)
    if r is not None:
        r[M // 2, : min(D, 128)] = 0
    out = L().add_rms_norm(x.to(DEV), w.to(DEV), to_dev(r), out_dtype=torch.float8_e4m3fn)
    ry, rh = ref.add_rms_norm(np64(x), np64(w), np64(r))
    rs = ref.block_scales(ry)
    assert out.y.dtype == torch.float8_e4m3fn and out.scales.shape == rs.shape
    hmag = np.abs(np64(x)) + (0 if r is None else np.abs(np64(r)))
    slack = norm_factor(D) * (np.abs(ry) + hmag * np.abs(np64(w)) / np.sqrt((rh * rh).mean(-1, keepdims=True) + 1e-6))
    top = np.stack([slack[:, b:b + 128].max(-1) for b in range(0, D, 128)], -1) / 448
    close(out.scales, rs, np.abs(rs) + top / U, 4 * U, "scales")
    each = np.repeat(np64(out.scales), 128, -1)[:, :D]
    got = np64(out.y.float()) * each
    tol = 2.0 ** -4 * np.abs(ry) * 1.001 + 2.0 ** -10 * each * 1.001 + slack
    assert (np.abs(got - ry) <= tol).all()
    assert not got[M // 2, : min(D, 128)].any() and np.isfinite(np64(out.scales)).all()


def test_norm_eight_bits_of_a_block_that_is_not_finite():
    x = torch.randn(2, 300, device=DEV)
    x[1, 5] = float("inf")
    out = L().add_rms_norm(x, torch.ones(300, device=DEV), out_dtype=torch.float8_e4m3fn)
    assert torch.isfinite(out.scales[0]).all() and torch.isnan(out.scales[1, 0])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(64, 0), (16, 16), (1, 1), (3, 0)])
def test_norm_strides_and_leading_dimensions(pad, offset, dtype):
    rng = np.random.default_rng(15)
    x, r, gy, gr = (torch.from_numpy(rng.standard_normal((2, 3, 260)).astype(np.float32)).to(dtype) for _ in range(4))
    w = torch.from_numpy(rng.standard_normal(260).astype(np.float32)).to(DEV)
    outs = []
    for f in (lambda t: t.to(DEV), lambda t: strided(t, pad, offset)):
        o = L().add_rms_norm(f(x), w, f(r))
        q = L().add_rms_norm(f(x), w, f(r), out_dtype=torch.float8_e4m3fn)
        h = strided(o.residual.cpu(), pad, offset)
        outs.append((o.y, o.residual, q.y.view(torch.uint8), q.scales, *L().add_rms_norm_backward(f(gy), h, w, f(gr))))
        assert o.y.shape == (2, 3, 260) and q.scales.shape == (2, 3, 3)
    for p, q in zip(*outs):
        assert torch.equal(p, q)


def test_norm_no_rows():
    w = torch.ones(40, device=DEV)
    x = torch.zeros(0, 40, device=DEV)
    assert L().add_rms_norm(x, w, x).y.shape == (0, 40)
    assert not L().add_rms_norm_backward(x, x, w).weight.any()


def test_state_pool_past_32_bit_offsets():
    """Slots whose states lie beyond 2^32 bytes and 2^31 elements."""
    D, S, K = 4096, 16, 4
    P = 33000   # 2.2e9 state values
    state = torch.empty(P, D, S, device=DEV)
    window = torch.empty(P * 6, K - 1, D, dtype=BF16, device=DEV)   # 2.4e9 values
    slots = torch.tensor([P - 1, 3, P - 7], dtype=torch.int32, device=DEV)
    a, _, _, _, rng = scan_inputs(3, 1, D, S, BF16, 16, step=True)
    dev = {k: v.to(DEV) for k, v in a.items()}
    init = torch.from_numpy(rng.standard_normal((3, D, S)).astype(np.float32)).to(DEV)
    state[slots.long()] = init
    y = L().selective_scan_step(state, **dev, slots=slots)
    small = init.clone()
    y2 = L().selective_scan_step(small, **dev)
    assert torch.equal(y, y2) and torch.equal(state[slots.long()], small)
    del state
    wslots = slots.clone()
    wslots[0] = P * 6 - 1
    wi = torch.randn(3, K - 1, D, device=DEV).to(BF16)
    window[wslots.long()] = wi
    w = torch.randn(D, K, device=DEV)
    y = L().causal_conv_step(window, dev["x"], w, slots=wslots)
    y2 = L().causal_conv_step(wi, dev["x"], w)
    assert torch.equal(y, y2) and torch.equal(window[wslots.long()], wi)


def test_rows_past_32_bit_offsets():
    """Row strides that put the last row beyond 2^32 elements."""
    N, T, D, S = 3, 20, 32, 16
    far = 2_200_000_000
    a, _, _, _, _ = scan_inputs(N, T, D, S, BF16, 17)
    dev = {k: v.to(DEV) for k, v in a.items()}
    store = torch.empty(2 * far + T * D, dtype=BF16, device=DEV)
    wide = store.as_strided((N, T, D), (far, D, 1))
    wide.copy_(dev["x"])
    w = torch.randn(D, 4, device=DEV)
    for p, q in zip(L().selective_scan(**{**dev, "x": wide}), L().selective_scan(**dev)):
        assert torch.equal(p, q)
    for p, q in zip(L().causal_conv(wide, w), L().causal_conv(dev["x"], w)):
        assert torch.equal(p, q)
    for p, q in zip(L().causal_conv_backward(wide, wide, w), L().causal_conv_backward(dev["x"], dev["x"], w)):
        assert p is None or torch.equal(p, q)
    weight = torch.randn(D, device=DEV)
    rows = store.as_strided((N, D), (far, 1))
    assert torch.equal(L().add_rms_norm(rows, weight).y, L().add_rms_norm(dev["x"][:, 0], weight).y)


def test_autograd_is_the_backward_calls():
    """A layer's loss through torch.autograd against the explicit gradients."""
    N, T, D, S, K = 2, 30, 32, 16, 4
    a, init, resets, _, rng = scan_inputs(N, T, D, S, F32, 18, "packed")
    w = torch.from_numpy(rng.standard_normal((D, K)).astype(np.float32))
    nw = torch.ones(D)
    resets = to_dev(resets)
    leaves = {k: v.to(DEV).requires_grad_() for k, v in {**a, "w": w, "nw": nw, "init": init}.items()}
    n = L().add_rms_norm(leaves["x"], leaves["nw"], leaves["x"])
    c, cf = L().causal_conv(n.y, leaves["w"], resets=resets)
    y, final = L().selective_scan(c, *(leaves[k] for k in ("delta", "A", "B", "C", "D", "z", "delta_bias")),
                                  initial_state=leaves["init"], resets=resets)
    (y.square().sum() + final.sum() + n.residual.sum() + cf.sum()).backward()
    d = {k: v.detach() for k, v in leaves.items()}
    n2 = L().add_rms_norm(d["x"], d["nw"], d["x"])
    c2, cf2 = L().causal_conv(n2.y, d["w"], resets=resets)
    args = [d[k] for k in ("delta", "A", "B", "C")]
    opts = [d[k] for k in ("D", "z", "delta_bias")]
    y2, final2, marks = L().selective_scan(c2, *args, *opts, initial_state=d["init"], resets=resets,
                                           return_checkpoints=True)
    assert torch.equal(y2, y) and torch.equal(final2, final)
    g = L().selective_scan_backward(2 * y2, c2, *args, marks, *opts, resets=resets,
                                    grad_final_state=torch.ones_like(final2))
    gc = L().causal_conv_backward(g.x, n2.y, d["w"], resets=resets, grad_final_state=torch.ones_like(cf2))
    gn = L().add_rms_norm_backward(gc.x, n2.residual, d["nw"], torch.ones_like(n2.residual))
    for k in ("delta", "A", "B", "C", "D", "z", "delta_bias"):
        assert torch.equal(leaves[k].grad, getattr(g, k)), k
    assert torch.equal(leaves["init"].grad, g.initial_state) and torch.equal(leaves["w"].grad, gc.weight)
    assert torch.equal(leaves["nw"].grad, gn.weight) and torch.equal(leaves["x"].grad, gn.x + gn.residual)


def test_another_stream_and_a_captured_graph():
    N, T, D, S = 2, 300, 64, 16
    a, init, _, _, _ = scan_inputs(N, T, D, S, BF16, 19)
    dev = {k: v.to(DEV) for k, v in a.items()}
    w = torch.randn(D, 4, device=DEV)
    nw = torch.ones(D, device=DEV)
    want = L().selective_scan(**dev), L().causal_conv(dev["x"], w), L().add_rms_norm(dev["x"], nw, dev["z"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            got = L().selective_scan(**dev), L().causal_conv(dev["x"], w), L().add_rms_norm(dev["x"], nw, dev["z"])
    s.synchronize()
    for p, q in zip(want, got):
        for u, v in zip(p, q):
            assert u is None or torch.equal(u, v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, final, marks = L().selective_scan(**dev, return_checkpoints=True)
        grads = L().selective_scan_backward(y, dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks, dev["D"],
                                            dev["z"], dev["delta_bias"])
    b, _, _, _, _ = scan_inputs(N, T, D, S, BF16, 20)
    for k in dev:
        dev[k].copy_(b[k])
    g.replay()
    torch.cuda.synchronize()
    y2, final2, marks2 = L().selective_scan(**dev, return_checkpoints=True)
    grads2 = L().selective_scan_backward(y2, dev["x"], dev["delta"], dev["A"], dev["B"], dev["C"], marks2, dev["D"],
                                         dev["z"], dev["delta_bias"])
    for u, v in zip((y, final, marks, *grads), (y2, final2, marks2, *grads2)):
        assert u is None or torch.equal(u, v)


def test_refusals():
    N, T, D, S, K = 2, 6, 16, 4, 4
    a, init, _, _, _ = scan_inputs(N, T, D, S, F32, 21)
    dev = {k: v.to(DEV) for k, v in a.items()}
    scan = L().selective_scan
    w, x = torch.ones(D, K, device=DEV), dev["x"]
    for bad, err in ((dict(x=x.half()), TypeError), (dict(x=x[0]), ValueError), (dict(delta=x.bfloat16()), TypeError),
                     (dict(B=dev["B"][:, :, :2]), ValueError), (dict(A=dev["A"].bfloat16()), TypeError),
                     (dict(A=torch.zeros(D, 129, device=DEV)), ValueError), (dict(z=x.cpu()), ValueError),
                     (dict(D=torch.ones(D + 1, device=DEV)), ValueError),
                     (dict(resets=torch.zeros(N, T, device=DEV)), TypeError),
                     (dict(lengths=torch.ones(N, dtype=torch.int64, device=DEV)), TypeError),
                     (dict(initial_state=init.to(DEV)[:1]), ValueError)):
        with pytest.raises(err):
            scan(**{**dev, **bad})
    with pytest.raises(ValueError, match="checkpoints"):
        L().selective_scan_backward(x, x, dev["delta"], dev["A"], dev["B"], dev["C"], None)
    step = {k: (v[:, 0] if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
    with pytest.raises(ValueError, match="slots"):
        L().selective_scan_step(torch.zeros(1, D, S, device=DEV), **step)
    with pytest.raises(ValueError, match="contiguous"):
        L().selective_scan_step(torch.zeros(N, S, D, device=DEV).transpose(1, 2), **step)
    with pytest.raises(TypeError):
        L().selective_scan_step(torch.zeros(N, D, S, device=DEV).bfloat16(), **step)
    with pytest.raises(ValueError, match="activation"):
        L().causal_conv(x, w, activation="relu")
    with pytest.raises(ValueError, match="taps"):
        L().causal_conv(x, torch.ones(D, 9, device=DEV))
    with pytest.raises(TypeError):
        L().causal_conv(x, w.bfloat16())
    with pytest.raises(TypeError):
        L().causal_conv_step(torch.zeros(N, K - 1, D, device=DEV).bfloat16(), x[:, 0], w)
    nw = torch.ones(D, device=DEV)
    with pytest.raises(ValueError, match="out_dtype"):
        L().add_rms_norm(x, nw, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="eps"):
        L().add_rms_norm(x, nw, eps=-1.0)
    with pytest.raises(TypeError, match="residual"):
        L().add_rms_norm(x, nw, x.bfloat16())
    with pytest.raises(ValueError):
        L().add_rms_norm(x, nw[:-1])


def test_the_native_call_layer_is_the_python_way(monkeypatch):
    """Calls in the usual form go through the native layer; the Python way gives the same bits."""
    from linear_recurrence_scan_gb300 import state_space as ss
    fast = ss._load_fast()
    assert fast is not ss._NoFastCall
    N, T, D, S, K = 2, 40, 32, 16, 4
    a, init, resets, _, _ = scan_inputs(N, T, D, S, BF16, 23, "packed")
    dev = {k: v.to(DEV) for k, v in a.items()}
    step = {k: (v[:, 0] if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
    w, nw = torch.randn(D, K, device=DEV), torch.randn(D, device=DEV)
    lengths = torch.tensor([T, 7], dtype=torch.int32, device=DEV)
    slots = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    rows = dev["x"].view(-1, D)
    window = torch.randn(N, K - 1, D, device=DEV).to(BF16)

    def calls():
        state, win = init.to(DEV), window.clone()
        n = L().add_rms_norm(rows, nw, rows)
        q = L().add_rms_norm(rows, nw, rows.float(), out_dtype=torch.float8_e4m3fn)
        return [*L().selective_scan(**dev), *L().selective_scan(**dev, initial_state=init.to(DEV),
                                                                resets=to_dev(resets), lengths=lengths),
                L().selective_scan_step(state, **step, slots=slots), state,
                *L().causal_conv(dev["x"], w, nw, None, window, to_dev(resets).bool(), lengths),
                L().causal_conv_step(win, step["x"], w, nw, slots=slots), win, n.y, n.residual, q.y.view(torch.uint8),
                q.scales, q.residual]

    got = calls()
    assert fast.selective_scan_step(init.to(DEV), *(step[k] for k in ("x", "delta", "A", "B", "C", "D", "z",
                                                                      "delta_bias")), True, None) is not None
    assert fast.add_rms_norm(rows, nw, None, 1e-6, None) is not None
    # what is not in the usual form is left to Python
    assert fast.add_rms_norm(rows, nw.bfloat16(), None, 1e-6, None) is None
    assert fast.add_rms_norm(rows, nw.clone().requires_grad_(), None, 1e-6, None) is None
    assert fast.causal_conv(dev["x"].cpu(), w, None, "silu", None, None, None) is None
    with torch.no_grad():
        assert fast.add_rms_norm(rows, torch.nn.Parameter(nw), None, 1e-6, None) is not None
    monkeypatch.setattr(ss, "_fast", ss._NoFastCall)
    for p, q in zip(got, calls()):
        assert torch.equal(p, q)


@pytest.mark.parametrize("gap", [0, 3])
def test_scan_rows_of_two_byte_alignment(gap):
    """Odd rows of bfloat16, large enough to be copied into aligned rows first, against the same values in aligned ones."""
    N, T, D, S = 2, 333, 601, 12
    a, init, resets, _, rng = scan_inputs(N, T, D, S, BF16, 24, "packed")
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(BF16)
    even = {k: (strided(v, 8 - v.shape[-1] % 8) if k in ("x", "delta", "z", "B", "C") else v.to(DEV))
            for k, v in a.items()}
    odd = {k: (strided(v, gap) if gap and k in ("x", "delta", "z", "B", "C") else v.to(DEV)) for k, v in a.items()}
    outs = []
    for d, g in ((even, strided(gy, 8 - D % 8)), (odd, gy.to(DEV))):
        y, final, marks = L().selective_scan(**d, initial_state=to_dev(init), resets=to_dev(resets),
                                             return_checkpoints=True)
        grads = L().selective_scan_backward(g, d["x"], d["delta"], d["A"], d["B"], d["C"], marks, d["D"], d["z"],
                                            d["delta_bias"], resets=to_dev(resets))
        outs.append((y, final, *grads))
    for p, q in zip(*outs):
        assert torch.equal(p, q)
