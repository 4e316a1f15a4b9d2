"""The gated feed-forward block's projections on the GPU against float64:
sizes where tiles, stages and 16-byte rows end, both activations, strides,
alignments.  The bounds are derived in token_policy_cases.py."""
import numpy as np
import pytest
import torch

from state_space_cases import DEV, close
from token_policy_cases import projection_inputs, projection_oracle

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


def check(M, D, F, act="silu", seed=0, place=lambda t: t.to(DEV)):
    x, wg, wu, gh, _ = projection_inputs(M, D, F, seed + M + D + F)
    want = projection_oracle(x, wg, wu, gh, act)
    dev = [place(t) for t in (x, wg, wu)]
    h = L().gated_projection(*dev, act)
    close(h, *want["h"], 1.0, "h")
    run = lambda: L().gated_projection_backward(place(gh), *dev, act)  # noqa: E731
    g = run()
    for k in ("x", "gate_weight", "up_weight"):
        close(getattr(g, k), *want[k], 1.0, "gradient of " + k)
    for p, q in zip((h, *g), (L().gated_projection(*dev, act), *run())):
        assert torch.equal(p, q)
    L().workspace_status()


SIZES = [(3, 64, 64), (1, 8, 8), (128, 64, 128), (129, 72, 136), (256, 128, 256), (257, 200, 520), (300, 640, 320),
         (700, 512, 1000), (64, 2048, 768), (2, 256, 4096), (1000, 64, 72)]
ODD = [(1, 1, 1), (5, 7, 9), (40, 1111, 333), (260, 65, 131), (33, 130, 262)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_forward_and_gradients(M, D, F, act):
    check(M, D, F, act)


@pytest.mark.parametrize("M,D,F", ODD)
def test_odd_sizes(M, D, F):
    check(M, D, F)
    check(M, D, F, "gelu")


def test_more_tiles_than_pairs():
    check(2100, 128, 3000)


@pytest.mark.parametrize("M", [1, 7, 8, 9, 16, 17, 31, 32, 33])
@pytest.mark.parametrize("D,F", [(64, 48), (40, 17), (33, 70), (8, 300), (520, 16)])
def test_few_rows(M, D, F):
    check(M, D, F, "gelu" if M % 2 else "silu")


@pytest.mark.parametrize("M", [5, 70])
@pytest.mark.parametrize("pad,offset", [(8, 0), (16, 8), (1, 1), (3, 0), (8, 4)])
def test_strides_and_alignments(pad, offset, M):
    """Slices of wider arrays with NaN around them."""
    def place(t):
        wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
        wide[:, offset:offset + t.shape[1]] = t.to(DEV)
        return wide[:, offset:offset + t.shape[1]]
    check(M, 72, 136, place=place)


def test_halves_of_one_weight_and_leading_dimensions():
    x, wg, wu, gh, _ = projection_inputs(60, 64, 96, 5)
    both = torch.cat([wg, wu]).to(DEV)
    want = L().gated_projection(x.to(DEV), wg.to(DEV), wu.to(DEV))
    got = L().gated_projection(x.to(DEV).view(3, 20, 64), both[:96], both[96:])
    assert got.shape == (3, 20, 96) and torch.equal(got.view(60, 96), want)
    g = L().gated_projection_backward(gh.to(DEV), x.to(DEV), wg.to(DEV), wu.to(DEV))
    h = L().gated_projection_backward(gh.to(DEV).view(3, 20, 96), x.to(DEV).view(3, 20, 64), both[:96], both[96:])
    assert h.x.shape == (3, 20, 64)
    assert torch.equal(h.x.view(60, 64), g.x) and torch.equal(h.gate_weight, g.gate_weight) and torch.equal(h.up_weight, g.up_weight)
    # one row for all, a column-major weight, the same weight twice
    row = x[:1].to(DEV).expand(60, 64)
    assert torch.equal(L().gated_projection(row, both[:96], both[96:]), L().gated_projection(row.contiguous(), both[:96], both[96:]))
    turned = wg.to(DEV).t().contiguous().t()
    assert torch.equal(L().gated_projection(x.to(DEV), turned, wu.to(DEV)), want)
    assert torch.equal(L().gated_projection(x.to(DEV), wg.to(DEV), wg.to(DEV)), L().gated_projection(x.to(DEV), wg.to(DEV), wg.to(DEV).clone()))


def test_sums_in_parts():
    """Few tiles of a long K (dx of few rows, dW of few columns) join parts."""
    check(20, 256, 3000)
    check(3000, 64, 72)
    check(2500, 130, 65, "gelu")
    check(33, 70, 4001)


def test_large_values():
    """Activations far out: gates of hundreds, both signs."""
    x, wg, wu, gh, _ = projection_inputs(40, 64, 64, 3, scale=100.0)
    for act in ("silu", "gelu"):
        h = L().gated_projection(x.to(DEV), wg.to(DEV), wu.to(DEV), act)
        g = L().gated_projection_backward(gh.to(DEV), x.to(DEV), wg.to(DEV), wu.to(DEV), act)
        want = projection_oracle(x, wg, wu, gh, act)
        assert all(torch.isfinite(t).all() for t in (h, *g))
        got = h.double().cpu().numpy()
        assert (np.abs(got - want["h"][0]) <= 2.0 ** -7 * np.abs(want["h"][0]) + 0.02).all()


def test_empty_sizes():
    w = torch.ones(6, 8, dtype=BF16, device=DEV)
    x = torch.ones(0, 8, dtype=BF16, device=DEV)
    assert L().gated_projection(x, w, w).shape == (0, 6)
    g = L().gated_projection_backward(torch.ones(0, 6, dtype=BF16, device=DEV), x, w, w)
    assert g.x.shape == (0, 8) and not g.gate_weight.any() and not g.up_weight.any()
    x = torch.ones(5, 8, dtype=BF16, device=DEV)
    assert L().gated_projection(x, w[:0], w[:0]).shape == (5, 0)
    g = L().gated_projection_backward(torch.ones(5, 0, dtype=BF16, device=DEV), x, w[:0], w[:0])
    assert not g.x.any() and g.gate_weight.shape == (0, 8)


def test_autograd():
    x, wg, wu, gh, _ = (t.to(DEV) if isinstance(t, torch.Tensor) else t for t in projection_inputs(70, 64, 96, 9))
    want = L().gated_projection_backward(gh, x, wg, wu, "gelu")
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu)]
    h = L().gated_projection(*leaves, "gelu")
    assert torch.equal(h, L().gated_projection(x, wg, wu, "gelu"))
    got = torch.autograd.grad(h, leaves, gh, create_graph=True)
    for p, q in zip(got, want):
        assert torch.equal(p, q)
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        torch.autograd.grad(got[0].float().sum(), leaves[1])
    for i in range(3):   # one of them alone
        some = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, wg, wu))]
        (one,) = torch.autograd.grad(L().gated_projection(*some, "gelu"), [some[i]], gh)
        assert torch.equal(one, want[i])


def test_streams_and_graphs():
    for M in (3, 90):
        x, wg, wu, gh, _ = (t.to(DEV) if isinstance(t, torch.Tensor) else t for t in projection_inputs(M, 72, 129, M))
        want = (L().gated_projection(x, wg, wu), *L().gated_projection_backward(gh, x, wg, wu))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = (L().gated_projection(x, wg, wu), *L().gated_projection_backward(gh, x, wg, wu))
        side.synchronize()
        for p, q in zip(want, got):
            assert torch.equal(p, q)
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = (L().gated_projection(x, wg, wu), *L().gated_projection_backward(gh, x, wg, wu))
            graphs.append((graph, out))
        x.copy_(-x)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = (L().gated_projection(x, wg, wu), *L().gated_projection_backward(gh, x, wg, wu))
        for _, out in graphs:
            for p, q in zip(want, out):
                assert torch.equal(p, q)
    L().workspace_status()


def test_two_streams_at_once():
    """Projections and gated scans that share the SMs."""
    x, wg, wu, gh, _ = (t.to(DEV) if isinstance(t, torch.Tensor) else t for t in projection_inputs(1500, 512, 1000, 4))
    s = torch.randn(4, 900, 256, device=DEV).to(BF16)
    ld = -torch.rand(256, device=DEV) - 0.01
    want = (*L().gated_projection_backward(gh, x, wg, wu), *L().gated_scan(s, s, s, ld))
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(one):
            a = L().gated_projection_backward(gh, x, wg, wu)
        with torch.cuda.stream(two):
            b = L().gated_scan(s, s, s, ld)
            c = L().gated_projection_backward(gh, x, wg, wu)
    torch.cuda.synchronize()
    for p, q in zip(want, (*a, *b)):
        assert torch.equal(p, q)
    for p, q in zip(a, c):
        assert torch.equal(p, q)
    L().workspace_status()


def test_offsets_past_32_bits():
    """More than 2^31 outputs: rows of the end against the same rows alone."""
    M, D, F = 70000, 64, 33000
    torch.manual_seed(0)
    x, wg, wu = (torch.randn(n, D, device=DEV).to(BF16) for n in (M, F, F))
    h = L().gated_projection(x, wg, wu)
    tail = L().gated_projection(x[-300:], wg, wu)
    torch.testing.assert_close(h[-300:], tail, rtol=2 ** -7, atol=1e-6)
    gh = torch.zeros(M, F, dtype=BF16, device=DEV)
    gh[-300:] = torch.randn(300, F, device=DEV).to(BF16)
    g, t = L().gated_projection_backward(gh, x, wg, wu), L().gated_projection_backward(gh[-300:], x[-300:], wg, wu)
    torch.testing.assert_close(g.x[-300:], t.x, rtol=2 ** -6, atol=2.0)
    torch.testing.assert_close(g.gate_weight, t.gate_weight, rtol=2 ** -6, atol=0.5)
    assert not g.x[:-300].any()


def test_refusals():
    x, w = torch.zeros(4, 8, dtype=BF16, device=DEV), torch.zeros(6, 8, dtype=BF16, device=DEV)
    f = L().gated_projection
    with pytest.raises(TypeError, match="bfloat16"):
        f(x.float(), w, w)
    with pytest.raises(TypeError, match="gate_weight"):
        f(x, w.float(), w)
    with pytest.raises(ValueError, match="up_weight shape"):
        f(x, w, w[:5])
    with pytest.raises(ValueError, match="gate_weight shape"):
        f(x, w[:, :7], w)
    with pytest.raises(ValueError, match="activation"):
        f(x, w, w, "relu")
    with pytest.raises(ValueError, match="2 dimensions"):
        f(x[0], w, w)
    with pytest.raises(ValueError, match="values"):
        f(x[:, :0], w[:, :0], w[:, :0])
    with pytest.raises(ValueError, match="grad_h shape"):
        L().gated_projection_backward(torch.zeros(4, 5, dtype=BF16, device=DEV), x, w, w)


@pytest.mark.parametrize("M,D,F", [(8, 512, 3000), (3000, 128, 128), (300, 640, 320), (40, 111, 333)])
def test_one_gradient_alone(M, D, F):
    """The gradient of x or of the weights alone: other items, other parts of K, than both together."""
    x, wg, wu, gh, _ = projection_inputs(M, D, F, M + D)
    want = projection_oracle(x, wg, wu, gh, "silu")
    for names in (("x",), ("gate_weight", "up_weight")):
        t = dict(x=x.to(DEV), gate_weight=wg.to(DEV), up_weight=wu.to(DEV))
        for k in names:
            t[k].requires_grad_()
        L().gated_projection(**t).backward(gh.to(DEV))
        for k, v in t.items():
            assert (v.grad is not None) == (k in names)
            if k in names:
                close(v.grad, *want[k], 1.0, "gradient of " + k)
    L().workspace_status()


def test_much_work():
    """Gradients of so many steps that their products take a launch each; some rows and some features against float64."""
    M, D, F = 16384, 4096, 6144
    gen = torch.Generator(DEV).manual_seed(3)
    x, wg, wu, gh = (torch.randn(s, generator=gen, device=DEV, dtype=BF16) * f
                     for s, f in (((M, D), 1.0), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((M, F), 1.0)))
    h = L().gated_projection(x, wg, wu)
    g = L().gated_projection_backward(gh, x, wg, wu)
    rows, features = [0, 255, 256, 5000, M - 1], [0, 127, 128, 3333, F - 1]
    want = projection_oracle(x[rows].cpu(), wg.cpu(), wu.cpu(), gh[rows].cpu(), "silu")
    close(h[rows], *want["h"], 1.0, "h")
    close(g.x[rows], *want["x"], 1.0, "gradient of x")
    want = projection_oracle(x.cpu(), wg[features].cpu(), wu[features].cpu(), gh[:, features].cpu(), "silu")
    for k in ("gate_weight", "up_weight"):
        close(getattr(g, k)[features], *want[k], 1.0, "gradient of " + k)
    L().workspace_status()


@pytest.mark.parametrize("rows", [5, 700])
def test_gelu_far_from_zero(rows):
    """One value a row, weights 1: h = gelu(z) itself, to its own size.  The exponential's argument z^2 / 2 is rounded
    twice (2^-24 of itself each, times log 2 in the result, below z^2 2^-24 in all), the rest adds less than 20 steps of
    2^-24, and the result is rounded by 2^-8 of itself at most."""
    from scipy.special import ndtr
    z = torch.linspace(-12, 12, rows).to(BF16)
    z[rows // 2] = 0
    x, w = torch.zeros(rows, 8, dtype=BF16), torch.zeros(16, 8, dtype=BF16)
    x[:, 0], x[:, 1] = z, 1
    up = w.clone()
    w[:, 0], up[:, 1] = 1, 1
    h = L().gated_projection(x.to(DEV), w.to(DEV), up.to(DEV), "gelu").double().cpu().numpy()
    v = z.double().numpy()
    want = (v * ndtr(v))[:, None]
    assert (np.abs(h - want) <= np.abs(want) * (2.0 ** -8 + (v[:, None] ** 2 + 20) * 2.0 ** -24)).all()


@pytest.mark.parametrize("M,D,F", [(1, 20001, 64), (1, 50257, 128), (600, 9001, 1)])
def test_outputs_that_leave_in_different_ways(M, D, F):
    """A single row leaves by a tensor map whatever its length, rows of an odd length beside it value by value: pairs of
    blocks that take tiles of both."""
    check(M, D, F)


@pytest.mark.parametrize("M,D,F", [(64, 4096, 2048), (2000, 2048, 300), (300, 8192, 520)])
def test_outputs_of_different_alignment(M, D, F):
    """Through the C entry point: gradients on 16 bytes and off them in one call, the same bits as dense ones."""
    from linear_recurrence_scan_gb300 import _native, token_policy as tp
    from linear_recurrence_scan_gb300.api import _stream_handle
    lib = _native.lib()
    x, wg, wu, gh, _ = (t.to(DEV) if isinstance(t, torch.Tensor) else t for t in projection_inputs(M, D, F, 2))
    want = L().gated_projection_backward(gh, x, wg, wu)
    args = tp._PROJECTION_ARGS.pack(M, D, F, 0, x.data_ptr(), D, wg.data_ptr(), D, wu.data_ptr(), D)
    ws = torch.empty(lib.rlscan_gated_projection_backward_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    for offsets in ((0, 1, 0), (0, 0, 3), (5, 0, 0), (0, 7, 1), (1, 2, 3)):
        flat = [torch.full((t.numel() + 8,), 7.0, dtype=BF16, device=DEV) for t in want]
        outs = [f[o:o + t.numel()] for f, o, t in zip(flat, offsets, want)]
        assert lib.rlscan_gated_projection_backward(args, gh.data_ptr(), F, *(o.data_ptr() for o in outs), ws.data_ptr(),
                                                    ws.numel(), _stream_handle(x.device)) == 0
        for f, o, out, t in zip(flat, offsets, outs, want):
            assert torch.equal(out.view(t.shape), t)
            assert (f[:o] == 7).all() and (f[o + t.numel():] == 7).all()
    L().workspace_status()


def test_more_work_than_one_launch_takes():
    """So many steps a pair of blocks that both products of the gradients have a launch of their own: the same bits as
    each gradient alone, and some rows against float64."""
    M, D, F = 30000, 4096, 12288
    gen = torch.Generator(DEV).manual_seed(4)
    x, wg, wu, gh = (torch.randn(s, generator=gen, device=DEV, dtype=BF16) * f
                     for s, f in (((M, D), 1.0), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((M, F), 1.0)))
    g = L().gated_projection_backward(gh, x, wg, wu)
    for i, k in enumerate(("x", "gate_weight", "up_weight")):
        leaves = [t.clone().requires_grad_(j == i) for j, t in enumerate((x, wg, wu))]
        (one,) = torch.autograd.grad(L().gated_projection(*leaves), [leaves[i]], gh)
        assert torch.equal(one, getattr(g, k)), k
    rows = [0, 255, 256, 29999]
    want = projection_oracle(x[rows].cpu(), wg.cpu(), wu.cpu(), gh[rows].cpu(), "silu")
    close(g.x[rows], *want["x"], 1.0, "gradient of x")
    L().workspace_status()
