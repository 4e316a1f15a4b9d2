"""The gated recurrence on the GPU against its float64 oracle: sizes where
steps, warps, pairs and clusters end, both types, strides and alignments,
episode flags, padding, empty rows, idle slots, closed gates, streams, graphs.
The bounds are derived in token_policy_cases.py."""
import numpy as np
import pytest
import torch

from oracle import token_policy as ref
from state_space_cases import DEV, U, close, np64, strided, to_dev
from token_policy_cases import gated_factor, gated_grad_factor, gated_inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


def check(N, T, D, dtype, kind, seed=0, strongest=5.0, a=None):
    """Forward and gradients of one case against the oracle, twice for the same bits."""
    made, init, resets, lengths, rng = gated_inputs(N, T, D, dtype, seed + N + 10 * T + 100 * D, kind, strongest=strongest)
    a = made if a is None else a
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gf = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32))
    r64 = {k: np64(v) for k, v in a.items()}
    args = dict(initial_state=np64(init), resets=None if resets is None else resets.numpy(),
                lengths=None if lengths is None else lengths.numpy())
    dev = {k: v.to(DEV) for k, v in a.items()}
    on = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    y, final, marks = L().gated_scan(**dev, initial_state=to_dev(init), **on, return_checkpoints=True)
    ry, rf, rs = ref.gated_scan(**r64, **args)
    my, mf, ms = ref.gated_scan(**r64, **args, bound=True)
    close(y, ry, my, gated_factor(T), "y")
    close(final, rf, mf, gated_factor(T), "final state")
    close(marks, rs[:, 0:T:32], ms[:, 0:T:32], gated_factor(T), "checkpoints")
    run = lambda: L().gated_scan_backward(gy.to(DEV), **dev, checkpoints=marks, **on, grad_final_state=to_dev(gf))  # noqa: E731
    g = run()
    want = ref.gated_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf))
    mag = ref.gated_scan_backward(np64(gy), **r64, **args, grad_final=np64(gf), bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], gated_grad_factor(T, N * T if k == "log_decay" else 0), "gradient of " + k)
    for p, q in zip((y, final, marks, *g),
                    (*L().gated_scan(**dev, initial_state=to_dev(init), **on, return_checkpoints=True), *run())):
        assert torch.equal(p, q)
    plain = L().gated_scan(**dev, initial_state=to_dev(init), **on)
    assert len(plain) == 2 and torch.equal(plain[0], y) and torch.equal(plain[1], final)


# single values, a warp's tokens, a step's end, one and several channels, blocks of 64 channels, clusters of 2 to 8 blocks
SIZES = [(1, 1, 1), (2, 3, 2), (1, 7, 33), (2, 8, 64), (3, 9, 65), (1, 63, 40), (2, 64, 130), (2, 65, 5), (1, 127, 96),
         (2, 128, 31), (1, 129, 64), (2, 256, 66), (3, 300, 48), (1, 513, 130), (2, 700, 17)]


@pytest.mark.parametrize("kind", ["none", "packed", "ragged", "dense", "both"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", SIZES)
def test_forward_and_gradients(N, T, D, dtype, kind):
    check(N, T, D, dtype, kind)


@pytest.mark.parametrize("kind", ["packed", "ragged"])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", [(5, 150, 4100), (20, 130, 1027), (2, 200, 9800), (2, 400, 2560)])
def test_many_channels(N, T, D, dtype, kind):
    """Blocks that walk a row alone, and clusters of two and four."""
    check(N, T, D, dtype, kind)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_long_rows(dtype):
    check(1, 4000, 70, dtype, "both", strongest=0.5)
    check(2, 3001, 64, dtype, "none", strongest=0.01)


def dense_run(a, init, resets, lengths, gy, gf):
    dev = {k: v.to(DEV) for k, v in a.items()}
    on = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    y, final, marks = L().gated_scan(**dev, initial_state=to_dev(init), **on, return_checkpoints=True)
    return y, final, marks, L().gated_scan_backward(gy.to(DEV), **dev, checkpoints=marks, **on, grad_final_state=to_dev(gf))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(64, 0), (16, 16), (8, 4), (2, 2), (1, 1), (3, 0)])
@pytest.mark.parametrize("T,D", [(70, 96), (300, 130), (40, 64)])
def test_strides_and_alignments(T, D, pad, offset, dtype):
    """Slices of wider arrays (NaN around them) against the oracle, by tensor maps, pairs and values."""
    N = 2
    a, init, resets, lengths, rng = gated_inputs(N, T, D, dtype, 3, "both")
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    r64 = {k: np64(v) for k, v in a.items()}
    args = dict(initial_state=np64(init), resets=resets.numpy(), lengths=lengths.numpy())
    dev = {k: (v.to(DEV) if k == "log_decay" else strided(v, pad, offset)) for k, v in a.items()}
    on = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    y, final, marks = L().gated_scan(**dev, initial_state=to_dev(init), **on, return_checkpoints=True)
    close(y, ref.gated_scan(**r64, **args)[0], ref.gated_scan(**r64, **args, bound=True)[0], gated_factor(T), "y")
    g = L().gated_scan_backward(strided(gy, pad, offset), **dev, checkpoints=marks, **on)
    want = ref.gated_scan_backward(np64(gy), **r64, **args)
    mag = ref.gated_scan_backward(np64(gy), **r64, **args, bound=True)
    for k in want:
        close(getattr(g, k), want[k], mag[k], gated_grad_factor(T, N * T if k == "log_decay" else 0), "gradient of " + k)


def test_broadcast_and_transposed_inputs():
    """A stride of 0 over rows or tokens, time-major arrays, an element stride that is not 1."""
    N, T, D = 3, 70, 64
    a, init, _, _, _ = gated_inputs(N, T, D, BF16, 8)
    dev = {k: v.to(DEV) for k, v in a.items()}
    row, token = dev["gate"][:1].expand(N, T, D), dev["input_gate"][:, :1].expand(N, T, D)
    got = L().gated_scan(dev["x"], row, token, dev["log_decay"])
    want = L().gated_scan(dev["x"], row.contiguous(), token.contiguous(), dev["log_decay"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    time_major = dev["x"].transpose(0, 1).contiguous().transpose(0, 1)
    channel_major = dev["gate"].transpose(1, 2).contiguous().transpose(1, 2)
    got = L().gated_scan(time_major, channel_major, dev["input_gate"], dev["log_decay"])
    want = L().gated_scan(**dev)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 66, 65])
def test_padding_is_not_looked_at(D, dtype):
    """NaN and infinity behind the rows' last tokens and in front of resets."""
    N, T = 3, 150
    a, init, _, _, rng = gated_inputs(N, T, D, dtype, 4)
    lengths = torch.tensor([0, 77, 150], dtype=torch.int32)
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(dtype)
    gf = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32))
    clean = dense_run(a, init, None, lengths, gy, gf)
    dirty = {k: v.clone() for k, v in a.items()}
    bad = gy.clone()
    for n in range(N):
        for k in ("x", "gate", "input_gate"):
            dirty[k][n, int(lengths[n]):] = float("nan") if n else float("inf")
        bad[n, int(lengths[n]):] = float("nan")
    got = dense_run(dirty, init, None, lengths, bad, gf)
    for p, q in zip((*clean[:3], *clean[3]), (*got[:3], *got[3])):
        assert torch.equal(p, q)
    assert torch.equal(clean[1][0], init[0].to(DEV)) and torch.equal(clean[3].initial_state[0], gf[0].to(DEV))
    # an infinite state does not reach past a reset
    resets = torch.zeros(N, T, dtype=torch.uint8)
    resets[:, 40] = 1
    inf = init.clone()
    inf[:] = float("inf")
    y = L().gated_scan(**{k: v.to(DEV) for k, v in a.items()}, initial_state=inf.to(DEV), resets=resets.to(DEV))[0]
    assert torch.isinf(y[:, :40]).all() and torch.isfinite(y[:, 40:]).all()


def test_closed_and_open_gates():
    """Gates of +-100: decays of 1 and of exp(log_decay), no NaN, gradients finite."""
    N, T, D = 1, 70, 64
    for gate in (-100.0, 100.0):
        for dtype in (F32, BF16):
            x = torch.randn(N, T, D, device=DEV).to(dtype)
            g = torch.full_like(x, gate)
            ld = torch.full((D,), -0.5, device=DEV)
            init = torch.randn(N, D, device=DEV)
            y, final, marks = L().gated_scan(x, g, g, ld, initial_state=init, return_checkpoints=True)
            grads = L().gated_scan_backward(torch.ones_like(x), x, g, g, ld, marks)
            assert all(torch.isfinite(t).all() for t in (y, final, *grads))
            if gate < 0:   # the state is kept, the input has no root
                assert torch.equal(final, init)
                assert torch.equal(grads.initial_state, torch.full_like(init, T))


def test_strong_decays():
    """States that are gone after one token, and rates that hardly decay."""
    check(2, 130, 66, F32, "packed", strongest=5.0)
    a, _, _, _, _ = gated_inputs(2, 200, 64, F32, 1)
    a["log_decay"] = -torch.logspace(-6, 0.7, 64)
    check(2, 200, 64, F32, "none", a=a)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,D,P", [(1, 1, 1), (3, 64, 3), (7, 65, 9), (40, 130, 64), (5, 1537, 5)])
def test_step(N, D, P, dtype):
    a, _, _, _, rng = gated_inputs(N, 1, D, dtype, N + D, step=True)
    state = torch.from_numpy(rng.standard_normal((P, D)).astype(np.float32))
    slots = torch.from_numpy(rng.permutation(P)[:N].astype(np.int32))
    if N > 2:
        slots[1], slots[2] = -1, P   # idle sequences
    dev = {k: v.to(DEV) for k, v in a.items()}
    got = state.to(DEV)
    y = L().gated_scan_step(got, **dev, slots=slots.to(DEV))
    busy = [n for n in range(N) if 0 <= slots[n] < P]
    want, mag = np64(state), np.abs(np64(state))
    r64 = {k: np64(v) for k, v in a.items()}
    seq = {k: (v if k == "log_decay" else v[:, None]) for k, v in r64.items()}
    at = np.clip(slots.numpy(), 0, P - 1)
    h = ref.gated_scan(**seq, initial_state=np64(state)[at])[1]
    hm = ref.gated_scan(**seq, initial_state=np64(state)[at], bound=True)[1]
    for n in busy:
        want[slots[n]], mag[slots[n]] = h[n], hm[n]
    close(got, want, mag, gated_factor(1), "state")
    ry, rm = np.zeros((N, D)), np.zeros((N, D))
    ry[busy], rm[busy] = h[busy], hm[busy]
    close(y, ry, rm, gated_factor(1), "y")
    idle = sorted(set(range(P)) - {int(slots[n]) for n in busy})
    assert torch.equal(got[idle], state.to(DEV)[idle])
    if P >= N:
        one, two = state.to(DEV), state.to(DEV)
        assert torch.equal(L().gated_scan_step(one, **dev), L().gated_scan_step(two, **dev, slots=torch.arange(N, dtype=torch.int32, device=DEV)))
        assert torch.equal(one, two)


def test_steps_continue_a_prompt():
    """A prompt, then tokens one by one, as one longer prompt."""
    N, T, D = 4, 90, 192
    a, init, _, _, _ = gated_inputs(N, T, D, F32, 2)
    dev = {k: v.to(DEV) for k, v in a.items()}
    whole = L().gated_scan(**dev, initial_state=init.to(DEV))
    part = {k: (v if k == "log_decay" else v[:, :70]) for k, v in dev.items()}
    y, state = L().gated_scan(**part, initial_state=init.to(DEV))
    ys = [y]
    for t in range(70, T):
        ys.append(L().gated_scan_step(state, *(dev[k][:, t] for k in ("x", "gate", "input_gate")), dev["log_decay"])[:, None])
    torch.testing.assert_close(torch.cat(ys, 1), whole[0], rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(state, whole[1], rtol=1e-5, atol=1e-5)


def test_empty_sizes():
    for N, T, D in ((0, 5, 8), (2, 0, 8), (2, 5, 0), (0, 0, 0)):
        x = torch.zeros(N, T, D, device=DEV)
        ld, init = -torch.ones(D, device=DEV), torch.ones(N, D, device=DEV)
        y, final, marks = L().gated_scan(x, x, x, ld, initial_state=init, return_checkpoints=True)
        assert y.shape == (N, T, D) and (T > 0 or torch.equal(final, init))
        g = L().gated_scan_backward(x, x, x, x, ld, marks, grad_final_state=2 * init)
        assert g.log_decay.shape == (D,) and not g.log_decay.any()
        if T == 0 and D > 0:
            assert torch.equal(g.initial_state, 2 * init)
    assert L().gated_scan_step(torch.zeros(3, 8, device=DEV), *[torch.zeros(0, 8, device=DEV)] * 3, -torch.ones(8, device=DEV)).shape == (0, 8)


@pytest.mark.parametrize("D", [128, 65])
def test_autograd(D):
    N, T = 2, 100
    a, init, resets, lengths, rng = gated_inputs(N, T, D, F32, 6, "both")
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32))
    gf = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32))
    plain = dense_run(a, init, resets, lengths, gy, gf)
    leaves = {k: v.to(DEV).requires_grad_() for k, v in a.items()}
    h0 = init.to(DEV).requires_grad_()
    y, final = L().gated_scan(**leaves, initial_state=h0, resets=resets.to(DEV).bool(), lengths=to_dev(lengths))
    assert torch.equal(y, plain[0]) and torch.equal(final, plain[1])
    grads = torch.autograd.grad([y, final], [*leaves.values(), h0], [gy.to(DEV), gf.to(DEV)], retain_graph=True)
    g = plain[3]
    for p, q in zip(grads, (g.x, g.gate, g.input_gate, g.log_decay, g.initial_state)):
        assert torch.equal(p, q)
    only = torch.autograd.grad(final.sum(), leaves["x"], retain_graph=True)[0]   # y without a gradient
    assert torch.isfinite(only).all()
    (twice,) = torch.autograd.grad(y.sum(), leaves["x"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        torch.autograd.grad(twice.sum(), leaves["gate"])
    state = torch.zeros(N, D, device=DEV)
    kept = (state * h0).sum()
    L().gated_scan_step(state, *(a[k][:, 0].to(DEV) for k in ("x", "gate", "input_gate")), a["log_decay"].to(DEV))
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        kept.backward()


def test_streams_and_graphs():
    """Another stream than the default one; a captured and replayed forward, backward and step, on new inputs."""
    N, T, D = 2, 300, 192
    a, init, resets, lengths, rng = gated_inputs(N, T, D, BF16, 7, "both")
    gy = torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)).to(BF16)
    gf = torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32))
    want = dense_run(a, init, resets, lengths, gy, gf)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = dense_run(a, init, resets, lengths, gy, gf)
    side.synchronize()
    for p, q in zip((*want[:3], *want[3]), (*got[:3], *got[3])):
        assert torch.equal(p, q)
    dev = {k: v.to(DEV) for k, v in a.items()}
    on = dict(resets=to_dev(resets), lengths=to_dev(lengths))
    h0, gy, gf = init.to(DEV), gy.to(DEV), gf.to(DEV)
    state = init.to(DEV)
    one = [dev[k][:, 0] for k in ("x", "gate", "input_gate")]
    with torch.cuda.stream(side):
        L().gated_scan_step(state.clone(), *one, dev["log_decay"])
    side.synchronize()
    graphs = []
    for _ in range(2):   # two graphs alive at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, final, marks = L().gated_scan(**dev, initial_state=h0, **on, return_checkpoints=True)
            g = L().gated_scan_backward(gy, **dev, checkpoints=marks, **on, grad_final_state=gf)
            s = L().gated_scan_step(state, *one, dev["log_decay"])
        graphs.append((graph, y, final, marks, g, s))
    fresh, init2, _, _, rng = gated_inputs(N, T, D, BF16, 70, "both")
    for k in ("x", "gate", "input_gate", "log_decay"):
        dev[k].copy_(fresh[k])
    state.copy_(h0)
    for graph, *_ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    want = dense_run(fresh, init, resets, lengths, gy.cpu(), gf.cpu())
    for _, y, final, marks, g, s in graphs:
        for p, q in zip((*want[:3], *want[3]), (y, final, marks, *g)):
            assert torch.equal(p, q)
    other = h0.clone()
    for _ in range(2):
        s = L().gated_scan_step(other, *one, dev["log_decay"])
    assert torch.equal(other, state) and torch.equal(s, graphs[1][5])
    L().workspace_status()


@pytest.mark.parametrize("D", [64, 66, 63])
def test_offsets_past_32_bits(D):
    """Rows 2^31 + 2^10 elements apart in one buffer."""
    N, T, apart = 2, 40, 2 ** 31 + 2 ** 10
    a, init, _, _, _ = gated_inputs(N, T, D, BF16, 9)
    buffer = torch.zeros(apart + 8 * T * 72, dtype=BF16, device=DEV)
    views = {}
    for i, k in enumerate(("x", "gate", "input_gate")):
        views[k] = buffer.as_strided((N, T, D), (apart, 72, 1), i * 2 * T * 72)
        views[k].copy_(a[k])
    dense = {k: v.to(DEV) for k, v in a.items()}
    want = L().gated_scan(**dense, return_checkpoints=True)
    got = L().gated_scan(**views, log_decay=dense["log_decay"], return_checkpoints=True)
    for p, q in zip(want, got):
        torch.testing.assert_close(p, q, rtol=2 ** -7, atol=1e-6)
    gw = L().gated_scan_backward(dense["x"], **dense, checkpoints=want[2])
    gg = L().gated_scan_backward(views["x"], **views, log_decay=dense["log_decay"], checkpoints=want[2])
    for p, q in zip(gw, gg):
        torch.testing.assert_close(p, q, rtol=2 ** -7, atol=1e-5)


def test_refusals():
    x = torch.zeros(2, 5, 8, device=DEV)
    d = torch.zeros(8, device=DEV)
    f = L().gated_scan
    with pytest.raises(TypeError, match="gate"):
        f(x, x.bfloat16(), x, d)
    with pytest.raises(ValueError, match="input_gate shape"):
        f(x, x, x[:, :4], d)
    with pytest.raises(TypeError, match="log_decay"):
        f(x, x, x, d.double())
    with pytest.raises(TypeError, match="log_decay"):
        f(x, x, x, None)
    with pytest.raises(TypeError, match="x: expected"):
        f(x.half(), x, x, d)
    with pytest.raises(ValueError, match="3 dimensions"):
        f(x[0], x[0], x[0], d)
    with pytest.raises(ValueError, match="initial_state shape"):
        f(x, x, x, d, initial_state=torch.zeros(2, 9, device=DEV))
    with pytest.raises(TypeError, match="lengths"):
        f(x, x, x, d, lengths=torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="checkpoints"):
        L().gated_scan_backward(x, x, x, x, d, None)
    with pytest.raises(ValueError, match="checkpoints shape"):
        L().gated_scan_backward(x, x, x, x, d, torch.zeros(2, 2, 8, device=DEV))
    s = L().gated_scan_step
    one = x[:, 0]
    with pytest.raises(ValueError, match="contiguous"):
        s(torch.zeros(8, 2, device=DEV).t(), one, one, one, d)
    with pytest.raises(ValueError, match="slots"):
        s(torch.zeros(1, 8, device=DEV), one, one, one, d)
    with pytest.raises(TypeError, match="state"):
        s(torch.zeros(2, 8, dtype=BF16, device=DEV), one, one, one, d)
    with pytest.raises(ValueError, match="state"):
        s(torch.zeros(2, 1, 8, device=DEV), one, one, one, d)


@pytest.mark.parametrize("which", ["x", "y", "all"])
def test_page_locked_memory(which):
    """Page-locked host arrays, which bulk copies are not for, are read and written in place."""
    from linear_recurrence_scan_gb300 import _native, token_policy as tp
    N, T, D = 2, 100, 64
    rng = np.random.default_rng(7)
    x, gate, ig = (torch.from_numpy(rng.standard_normal((N, T, D)).astype(np.float32)) for _ in range(3))
    ld = torch.from_numpy(-rng.uniform(0.1, 2, D).astype(np.float32))
    want = L().gated_scan(x.to(DEV), gate.to(DEV), ig.to(DEV), ld.to(DEV))[0]
    at = {k: v.pin_memory() if which in (k, "all") else v.to(DEV)
          for k, v in dict(x=x, gate=gate, ig=ig, ld=ld, y=torch.empty(N, T, D)).items()}
    args = tp._GATED_ARGS.pack(N, T, D, 0, *(v for k in ("x", "gate", "ig") for v in (at[k].data_ptr(), T * D, D)),
                               at["ld"].data_ptr(), 0, 0, 0)
    stream = torch.cuda.current_stream().cuda_stream
    assert _native.lib().rlscan_gated_scan(args, at["y"].data_ptr(), None, None, stream) == 0
    torch.cuda.synchronize()
    # the same sums in another order: T products and sums of terms below 5 (|x| < 5), each rounded to 2^-24
    torch.testing.assert_close(at["y"].cpu(), want.cpu(), rtol=0, atol=5 * 3 * T * 2 ** -24)
    L().workspace_status()


def test_channels_past_32_bits():
    """More than 2^31 channels, whose blocks tensor maps cannot address: the first, the last and those around 2^31 against
    the oracle, forward, gradients and a single token."""
    D = 2 ** 31 + 136
    gen = torch.Generator(DEV).manual_seed(1)

    def normal():
        return torch.empty(1, 1, D, dtype=BF16, device=DEV).normal_(generator=gen)

    a = dict(x=normal(), gate=normal(), input_gate=normal(),
             log_decay=torch.empty(D, dtype=F32, device=DEV).uniform_(-3, -0.01, generator=gen))
    init = torch.empty(1, D, dtype=F32, device=DEV).normal_(generator=gen)
    gy = normal()
    y, final, marks = L().gated_scan(**a, initial_state=init, return_checkpoints=True)
    g = L().gated_scan_backward(gy, **a, checkpoints=marks)
    L().workspace_status()
    step = init.clone()
    ys = L().gated_scan_step(step, *(a[k][:, 0] for k in ("x", "gate", "input_gate")), a["log_decay"])
    for at in (slice(0, 300), slice(2 ** 31 - 200, 2 ** 31 + 136)):
        r64 = {k: np64(v[..., at]) for k, v in a.items()}
        h0, gy64 = np64(init[..., at]), np64(gy[..., at])
        ry, rf, _ = ref.gated_scan(**r64, initial_state=h0)
        my, mf, _ = ref.gated_scan(**r64, initial_state=h0, bound=True)
        close(y[..., at], ry, my, gated_factor(1), "y")
        close(final[..., at], rf, mf, gated_factor(1), "final state")
        close(step[..., at], rf, mf, gated_factor(1), "state of one token")
        close(ys[..., at], ry[:, 0], my[:, 0], gated_factor(1), "y of one token")
        want = ref.gated_scan_backward(gy64, **r64, initial_state=h0)
        mag = ref.gated_scan_backward(gy64, **r64, initial_state=h0, bound=True)
        for k in want:
            close(getattr(g, k)[..., at], want[k], mag[k], gated_grad_factor(1, 1), "gradient of " + k)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", [(2, 200, 64), (2, 200, 66), (2, 200, 65), (2, 200, 20480), (2, 700, 130), (1, 3000, 64)])
def test_values_that_are_not_numbers(N, T, D, dtype):
    """A NaN or an infinity stays in its row's states (and gradients' messages) up to the next reset and no further, also
    where the product of a few decays is 0 in 32 bits (here exp(-40) each)."""
    first, second, cut, last = T // 20, T // 5, 3 * T // 4, T - 5
    for strong in (True, False):
        x, gate, ig, gy = (torch.randn(N, T, D, device=DEV).clamp(-3, 3).to(dtype) for _ in range(4))
        if strong:
            gate[:] = 10
        ld = torch.full((D,), -40.0 if strong else -0.1, device=DEV)
        for bad in (float("nan"), float("inf")):
            resets = torch.zeros(N, T, dtype=torch.uint8, device=DEV)
            resets[:, first], resets[:, cut], resets[:, cut + 2], resets[:, cut - 30] = 1, 1, 1, 1
            resets[:, second - 1] = 1
            xb, gb, init = x.clone(), gy.clone(), torch.full((N, D), bad, device=DEV)
            xb[:, second], gb[:, last] = bad, bad
            y, final, marks = L().gated_scan(xb, gate, ig, ld, initial_state=init, resets=resets, return_checkpoints=True)
            want = torch.zeros(T, dtype=torch.bool, device=DEV)
            want[:first] = want[second:cut - 30] = True
            assert torch.equal(~torch.isfinite(y), want[None, :, None].expand(N, T, D))
            assert torch.isfinite(final).all()
            g = L().gated_scan_backward(gb, xb, gate, ig, ld, marks, resets=resets)
            back = torch.zeros(T, dtype=torch.bool, device=DEV)
            back[cut + 2:last + 1] = True
            assert torch.equal(~torch.isfinite(g.x), back[None, :, None].expand(N, T, D))
            assert torch.isfinite(g.initial_state).all()
            # without the resets all that follows (or, of the gradients, is in front)
            y, final, marks = L().gated_scan(xb, gate, ig, ld, return_checkpoints=True)
            want[:] = False
            want[second:] = True
            assert torch.equal(~torch.isfinite(y), want[None, :, None].expand(N, T, D))
            assert not torch.isfinite(final).any()
            g = L().gated_scan_backward(gb, xb, gate, ig, ld, marks)
            assert not torch.isfinite(g.x[:, :last + 1]).any() and torch.isfinite(g.x[:, last + 1:]).all()
            assert not torch.isfinite(g.initial_state).any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,D", [(10, 150, 4096), (11, 70, 4098), (9, 90, 4161), (19, 260, 2048)])
def test_more_chains_than_places(N, T, D, dtype):
    """640 chains of blocks and about as many, where the GPU holds 456 or 304 at once: a second round of them."""
    check(N, T, D, dtype, "both")
