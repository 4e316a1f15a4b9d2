"""The distillation loss on the GPU against its float64 oracle: vocabularies
where warps, blocks, clusters and 16-byte units end, both types, strides,
alignments, masked rows, empty and repeated teacher tokens, infinities, NaN.
The bounds are derived in token_policy_cases.py."""
import numpy as np
import pytest
import torch

from oracle import token_policy as ref
from state_space_cases import DEV, close, np64, strided, to_dev
from token_policy_cases import distill_factor, distill_inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


def check(logits, teacher, tokens, mask, grad_loss, tau=1.0, on_gpu=None):
    """All three calls against the oracle, the two ways to the gradient against each other."""
    V, K = logits.shape[2], teacher.shape[2]
    dev = logits.to(DEV) if on_gpu is None else on_gpu
    args = (teacher.to(DEV), tokens.to(DEV))
    m = to_dev(mask)
    loss, norm = L().distill_loss(dev, *args, tau, m, return_normalizers=True)
    grad = L().distill_loss_backward(grad_loss.to(DEV), dev, *args, norm, tau, m)
    both_loss, both_grad = L().distill_loss_and_grad(grad_loss.to(DEV), dev, *args, tau, m)
    rl, rg, ml, mg = ref.distill_loss(np64(logits), np64(teacher), tokens.numpy(), tau,
                                      None if mask is None else mask.numpy() != 0, np64(grad_loss))
    z, th = np64(logits), np64(teacher)
    z, th = z[np.isfinite(z) & (np.abs(z) < 1e30)], th[np.isfinite(th)]
    f = distill_factor(V, K, max(np.ptp(z) if z.size else 0, np.ptp(th) if th.size else 0) / tau)
    close(loss, rl, ml, f, "loss")
    close(both_loss, rl, ml, f, "loss with its gradient")
    close(grad, rg, mg, f, "gradient")
    close(both_grad, rg, mg, f, "gradient with its loss")
    assert grad.shape == logits.shape and grad.dtype == logits.dtype and grad.is_contiguous()
    again = L().distill_loss_and_grad(grad_loss.to(DEV), dev, *args, tau, m)
    assert torch.equal(again[0], both_loss) and torch.equal(again[1], both_grad)
    return loss, both_grad


# vocabularies: within a warp's registers, a small block's, a block's, a cluster's; one unit more or less
SIZES = [(1, 1, 1, 1), (2, 3, 2, 2), (1, 5, 7, 3), (2, 2, 31, 5), (3, 3, 64, 8), (1, 4, 1000, 33), (1, 3, 1023, 64),
         (2, 2, 2047, 32), (1, 2, 2049, 256), (1, 2, 4100, 31), (1, 3, 8191, 16), (1, 2, 8200, 64), (1, 2, 32761, 32),
         (1, 2, 33000, 100), (1, 1, 50257, 32), (1, 1, 131075, 20), (2, 1, 262143, 8)]


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,V,K", SIZES)
def test_loss_and_gradient(N, T, V, K, dtype, tau):
    logits, teacher, tokens, mask, grad, _ = distill_inputs(N, T, V, K, dtype, V + K)
    check(logits, teacher, tokens, mask if N * T > 2 else None, grad, tau)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,T,V,K", [(2, 400, 9000, 4), (1, 7000, 300, 6), (3, 900, 5000, 3), (1, 650, 36001, 3), (1, 330, 140000, 2)])
def test_many_rows(N, T, V, K, dtype):
    """More rows than blocks: every block takes several, in one part each and in several."""
    logits, teacher, tokens, mask, grad, _ = distill_inputs(N, T, V, K, dtype, 3)
    check(logits, teacher, tokens, mask, grad)


def test_rows_longer_than_a_cluster_holds():
    """The loss and its gradient in two calls, over rounds of a block."""
    for dtype, V in ((F32, 140001), (BF16, 270001)):
        logits, teacher, tokens, mask, grad, _ = distill_inputs(1, 2, V, 5, dtype, 9)
        check(logits, teacher, tokens, None, grad)


@pytest.mark.parametrize("token_dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("teacher_dtype", [F32, BF16], ids=["f32", "bf16"])
def test_teacher_types(teacher_dtype, token_dtype):
    logits, teacher, tokens, mask, grad, _ = distill_inputs(2, 9, 300, 12, BF16, 4, teacher_dtype, token_dtype)
    check(logits, teacher, tokens, mask.bool(), grad)


def test_masked_vocabulary():
    """Logits of -infinity and of the type's lowest value: probability 0, or, where a row has nothing else, all alike."""
    for dtype in (F32, BF16):
        logits, teacher, tokens, _, grad, rng = distill_inputs(1, 4, 700, 5, dtype, 1)
        tokens = tokens.clamp(0, 99)
        low = torch.finfo(dtype).min
        logits[0, 0, 100:] = -float("inf")
        logits[0, 1, 100:] = low
        loss, g = check(logits, teacher, tokens, None, grad)
        assert not g[0, :2, 100:].any()
        for k in range(5):   # tokens twice and all rows of one value
            tokens[0, :, k] = k
        logits[0, 2] = low
        logits[0, 3] = 0
        loss, g = check(logits[:, 2:], teacher[:, 2:], tokens[:, 2:], None, grad[:, 2:])
        teacher[0, 3] = teacher[0, 2]
        a, _ = L().distill_loss_and_grad(grad.to(DEV), logits.to(DEV), teacher.to(DEV), tokens.to(DEV))
        assert torch.equal(a[0, 2], a[0, 3])
        # the teacher learns of a token that the student rules out: an infinite loss, a finite gradient
        logits[0, 0, tokens[0, 0, 0]] = -float("inf")
        a, g = L().distill_loss_and_grad(grad.to(DEV), logits.to(DEV), teacher.to(DEV), tokens.to(DEV))
        assert a[0, 0] == float("inf") and torch.isfinite(g[0, 0]).all()


@pytest.mark.parametrize("V", [50, 3000, 40000])
def test_rows_without_a_loss(V):
    """Masked rows (NaN in them), rows without a teacher's token, teachers of -infinity: loss 0, gradient 0."""
    for dtype in (F32, BF16):
        logits, teacher, tokens, mask, grad, _ = distill_inputs(2, 6, V, 4, dtype, 2)
        mask[:] = 1
        mask[0, 2] = mask[1, 5] = 0
        logits[0, 2] = float("nan")
        teacher[1, 5] = float("nan")
        tokens[0, 3] = -1
        teacher[0, 4] = -float("inf")
        teacher[0, 5, 0] = -float("inf")
        tokens[0, 5] = torch.arange(4)
        loss, g = check(logits, teacher, tokens, mask, grad)
        for n, t in ((0, 2), (1, 5), (0, 3), (0, 4)):
            assert loss[n, t] == 0 and not g[n, t].any()
        none = torch.zeros_like(mask)
        loss, g = check(logits, teacher, tokens, none, grad)
        assert not loss.any() and not g.any()


def test_values_that_are_not_numbers():
    """A NaN or +infinity stays in its row; a row of -infinity alone has no distribution."""
    logits, teacher, tokens, _, grad, _ = distill_inputs(1, 6, 900, 3, F32, 3)
    logits[0, 0, 5] = float("nan")
    logits[0, 1, 7] = float("inf")
    logits[0, 2] = -float("inf")
    teacher[0, 3, 0] = float("nan")
    teacher[0, 4, 0] = float("inf")
    for d in (F32, BF16):
        loss, norm = L().distill_loss(logits.to(DEV).to(d), teacher.to(DEV), tokens.to(DEV), return_normalizers=True)
        both, g = L().distill_loss_and_grad(grad.to(DEV), logits.to(DEV).to(d), teacher.to(DEV), tokens.to(DEV))
        for v in (loss, both):
            assert torch.isnan(v[0, :5]).all() and torch.isfinite(v[0, 5])
        assert torch.isnan(g[0, :3]).all() and torch.isfinite(g[0, 5]).all()
        assert torch.isnan(g[0, 3]).any() and torch.isnan(g[0, 4]).any()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 9, 300, 1003, 5001, 33001])
@pytest.mark.parametrize("pad,offset", [(8, 0), (5, 3), (16, 8), (1, 1)])
def test_strides_and_alignments(pad, offset, V, dtype):
    """Slices of wider arrays, whose units of 16 bytes lie otherwise than the dense gradient's; NaN around them."""
    logits, teacher, tokens, mask, grad, _ = distill_inputs(2, 3, V, 5, dtype, V)
    check(logits, teacher, tokens, mask, grad, on_gpu=strided(logits, pad, offset))
    wide = torch.full((2, 7, V), float("nan"), dtype=dtype, device=DEV)   # every other token, the last one left out
    wide[:, :6:2] = logits.to(DEV)
    check(logits, teacher, tokens, mask, grad, on_gpu=wide[:, :6:2])


def test_repeated_tokens():
    """One token K times, and pairs of them over the chunks of a warp."""
    logits, teacher, tokens, _, grad, _ = distill_inputs(1, 3, 500, 200, F32, 5)
    tokens[0, 0] = 7
    tokens[0, 1] = torch.arange(200) % 100
    check(logits, teacher, tokens, None, grad)


def test_expanded_arguments_and_empty_sizes():
    logits, teacher, tokens, _, grad, _ = distill_inputs(2, 4, 60, 3, F32, 6)
    one = teacher[:, :1].to(DEV).expand(2, 4, 3)
    a = L().distill_loss(logits.to(DEV), one, tokens.to(DEV))
    assert torch.equal(a, L().distill_loss(logits.to(DEV), one.contiguous(), tokens.to(DEV)))
    w = torch.full((1, 1), 0.5, device=DEV).expand(2, 4)
    assert torch.equal(L().distill_loss_and_grad(w, logits.to(DEV), one, tokens.to(DEV))[1],
                       L().distill_loss_and_grad(w.contiguous(), logits.to(DEV), one, tokens.to(DEV))[1])
    for N, T in ((0, 4), (2, 0)):
        z, th, tok = torch.zeros(N, T, 9, device=DEV), torch.zeros(N, T, 3, device=DEV), torch.zeros(N, T, 3, dtype=torch.long, device=DEV)
        loss, norm = L().distill_loss(z, th, tok, return_normalizers=True)
        assert loss.shape == (N, T) and norm.shape == (N, T, 2)
        assert L().distill_loss_backward(loss, z, th, tok, norm).shape == z.shape
        assert L().distill_loss_and_grad(loss, z, th, tok)[1].shape == z.shape


def test_autograd():
    logits, teacher, tokens, mask, grad, _ = distill_inputs(2, 5, 400, 6, BF16, 7)
    leaf = logits.to(DEV).requires_grad_()
    loss = L().distill_loss(leaf, teacher.to(DEV), tokens.to(DEV), 2.0, mask.to(DEV))
    want, g = L().distill_loss_and_grad(grad.to(DEV), logits.to(DEV), teacher.to(DEV), tokens.to(DEV), 2.0, mask.to(DEV))
    assert torch.equal(loss, want)
    (got,) = torch.autograd.grad((loss * grad.to(DEV)).sum(), leaf, create_graph=True)
    torch.testing.assert_close(got, g, rtol=2 ** -7, atol=1e-30)
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        torch.autograd.grad(got.float().sum(), leaf)
    with pytest.raises(ValueError, match="detach"):
        L().distill_loss(leaf, teacher.to(DEV).requires_grad_(), tokens.to(DEV))


def test_streams_and_graphs():
    args = [distill_inputs(2, 40, V, 6, BF16, V)[:5] for V in (300, 9000, 50000)]
    for logits, teacher, tokens, mask, grad in args:
        dev = [t.to(DEV) for t in (logits, teacher, tokens)]
        w, m = grad.to(DEV), mask.to(DEV)
        want = L().distill_loss_and_grad(w, *dev, mask=m)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = L().distill_loss_and_grad(w, *dev, mask=m)
        side.synchronize()
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                loss, norm = L().distill_loss(*dev, mask=m, return_normalizers=True)
                g = L().distill_loss_backward(w, *dev, norm, mask=m)
                both = L().distill_loss_and_grad(w, *dev, mask=m)
            graphs.append((graph, loss, g, *both))
        dev[0].copy_(-dev[0])
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = L().distill_loss_and_grad(w, *dev, mask=m)
        for _, loss, g, a, b in graphs:
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])
            torch.testing.assert_close(loss, want[0], rtol=1e-5, atol=1e-5)
            torch.testing.assert_close(g, want[1], rtol=2 ** -7, atol=1e-7)
    L().workspace_status()


def test_offsets_past_32_bits():
    """2^31 logits and more: the last rows against the same rows alone."""
    N, T, V, K = 1, 17000, 131072, 4
    logits = torch.empty(N, T, V, dtype=BF16, device=DEV)
    some, teacher, tokens, _, grad, _ = distill_inputs(1, 3, V, K, BF16, 8)
    logits[:] = 0
    logits[0, -3:] = some[0].to(DEV)
    th, tok = torch.zeros(N, T, K, device=DEV), torch.zeros(N, T, K, dtype=torch.int32, device=DEV)
    w = torch.zeros(N, T, device=DEV)
    th[0, -3:], tok[0, -3:], w[0, -3:] = teacher[0].to(DEV), tokens[0].to(DEV, torch.int32), grad[0].to(DEV)
    loss, g = L().distill_loss_and_grad(w, logits, th, tok)
    want, gw = L().distill_loss_and_grad(w[:, -3:].contiguous(), logits[:, -3:], th[:, -3:], tok[:, -3:])
    torch.testing.assert_close(loss[:, -3:], want, rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(g[:, -3:], gw, rtol=2 ** -7, atol=1e-7)
    torch.testing.assert_close(L().distill_loss(logits, th, tok), loss, rtol=1e-5, atol=1e-5)


def test_refusals():
    z, th = torch.zeros(2, 3, 9, device=DEV), torch.zeros(2, 3, 4, device=DEV)
    tok, w = torch.zeros(2, 3, 4, dtype=torch.long, device=DEV), torch.zeros(2, 3, device=DEV)
    f = L().distill_loss
    with pytest.raises(TypeError, match="teacher_tokens"):
        f(z, th, tok.float())
    with pytest.raises(TypeError, match="teacher_logits"):
        f(z, th.half(), tok)
    with pytest.raises(ValueError, match="teacher_tokens shape"):
        f(z, th, tok[..., :3])
    with pytest.raises(ValueError, match="256"):
        f(z, torch.zeros(2, 3, 257, device=DEV), tok)
    with pytest.raises(ValueError, match="256"):
        f(z, th[..., :0], tok[..., :0])
    for tau in (0.0, -1.0, float("nan"), float("inf"), 0):
        with pytest.raises(ValueError, match="temperature"):
            f(z, th, tok, tau)
    with pytest.raises(ValueError, match="vocabulary"):
        f(z[..., :0], th, tok)
    with pytest.raises(ValueError, match="mask shape"):
        f(z, th, tok, mask=torch.ones(2, 4, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="normalizers"):
        L().distill_loss_backward(w, z, th, tok, None)
    with pytest.raises(TypeError, match="grad_loss"):
        L().distill_loss_backward(w.double(), z, th, tok, torch.zeros(2, 3, 2, device=DEV))
    with pytest.raises(TypeError, match="grad_loss"):
        L().distill_loss_and_grad(None, z, th, tok)
    assert torch.equal(f(z, th, tok, 1), f(z, th, tok, 1.0))


def test_logits_on_the_host_are_refused():
    """Rows of logits come by bulk copies, which are for device memory: others end with an error in front of any launch."""
    from linear_recurrence_scan_gb300 import _native, token_policy as tp
    z, th = torch.zeros(2, 3, 16).pin_memory(), torch.zeros(2, 3, 4, device=DEV)
    tok, loss, w = torch.zeros(2, 3, 4, dtype=torch.long, device=DEV), torch.full((2, 3), 7.0, device=DEV), torch.ones(2, 3, device=DEV)
    norm, grad = torch.zeros(2, 3, 2, device=DEV), torch.zeros(2, 3, 16, device=DEV)
    args = tp._DISTILL_ARGS.pack(2, 3, 16, 4, 0, 0, 8, z.data_ptr(), 48, 16, th.data_ptr(), tok.data_ptr(), 0, 1.0)
    lib, memory = _native.lib(), 10
    assert lib.rlscan_distill_loss(args, loss.data_ptr(), None, None) == memory
    assert lib.rlscan_distill_loss_backward(args, w.data_ptr(), norm.data_ptr(), grad.data_ptr(), None) == memory
    assert lib.rlscan_distill_loss_and_grad(args, w.data_ptr(), loss.data_ptr(), norm.data_ptr(), grad.data_ptr(), None) == memory
    torch.cuda.synchronize()
    assert (loss == 7).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [7, 8, 127, 135, 255, 256, 263, 264, 511, 519, 1023, 1031, 1032, 2047, 2055, 2056, 3079, 6151, 12807])
def test_rows_at_the_ends_of_each_kind(V, dtype):
    """One value less and more than lanes, warps and stages hold, rows that start anywhere in 16 bytes; the teacher has
    the first and the last token, the last one twice."""
    K = min(V, 40)
    logits, teacher, tokens, mask, grad, rng = distill_inputs(3, 5, V, K, dtype, V)
    tokens[..., 0], tokens[..., -1] = 0, V - 1
    if K > 2:
        tokens[:, ::2, K // 2] = V - 1
    check(logits, teacher, tokens, mask, grad)


LEVELS = [1e6, -1e7, 1.2e7, 1e8, -1e8, 5e9, -5e9, 1e10, -1e10, 1e12, -1e20, 1e20, -1e29, 1e29]


def far_rows(V, K, dtype, level, rng):
    """Logits around `level` (from 1e10 on, and for bfloat16 sooner, all the same value), one in three -infinity, one in
    seven the type's lowest; the teacher knows the others alone."""
    z = torch.from_numpy((level + 2 * rng.standard_normal((1, 1, V))).astype(np.float32)).to(dtype)
    places = np.arange(V)
    some = np.flatnonzero((places % 3 != 1) & (places % 7 != 2))
    z[..., places % 7 == 2] = torch.finfo(dtype).min
    z[..., places % 3 == 1] = -float("inf")
    return z, torch.from_numpy(rng.choice(some, (1, 1, K)))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [5, 300, 2047, 5000, 9001, 50257, 131075])
def test_logits_far_from_zero(V, dtype):
    """Rows whose largest logit lies anywhere between 0 and the type's ends, as a row masked with -1e10 throughout: finite
    losses and gradients, by each kernel (a warp's rows, blocks', clusters').  The exponent (z - m) / tau has the error
    that token_policy_cases.py derives: logits of one row differ by little."""
    K, rng = 5, np.random.default_rng(V)
    rows = []
    for level in LEVELS:
        z, tokens = far_rows(V, K, dtype, level, rng)
        teacher = torch.from_numpy((2 * rng.standard_normal((1, 1, K))).astype(np.float32))
        grad = torch.from_numpy(rng.standard_normal((1, 1)).astype(np.float32))
        loss, g = check(z, teacher, tokens, None, grad)
        assert torch.isfinite(loss).all() and torch.isfinite(g).all(), level
        rows.append((z, teacher, tokens, grad))
    z, teacher, tokens, grad = (torch.cat(t, 1).to(DEV) for t in zip(*rows))   # one behind the other
    loss, g = L().distill_loss_and_grad(grad, z, teacher, tokens)
    assert torch.isfinite(loss).all() and torch.isfinite(g).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 3001, 50257])
@pytest.mark.parametrize("level,tau", [(1e4, 1e-6), (-5e3, 1e-6), (-3e9, 0.5), (7.0, 1e-6), (1e30, 1e6)])
def test_far_logits_at_low_and_high_temperatures(level, tau, V, dtype):
    """What counts is the logit over the temperature; the teacher's differ by a few temperatures."""
    K, rng = 6, np.random.default_rng(1)
    z = torch.full((1, 2, V), level).to(dtype)
    z[0, 1, V // 2:] = -float("inf")
    teacher = torch.from_numpy((rng.integers(0, 5, (1, 2, K)) * tau).astype(np.float32))
    tokens = torch.from_numpy(rng.integers(0, V // 2, (1, 2, K)))
    grad = torch.from_numpy(rng.standard_normal((1, 2)).astype(np.float32))
    loss, g = check(z, teacher, tokens, None, grad, tau)
    assert torch.isfinite(loss).all() and torch.isfinite(g).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 2000, 5000, 50257, 140001])
def test_normalizers_of_any_alignment(V, dtype):
    """A [N,T,2] view one float behind a 16-byte boundary, read by the gradient's call and written through the C entry
    points: the same bits as a dense tensor's."""
    from linear_recurrence_scan_gb300 import _native, token_policy as tp
    from linear_recurrence_scan_gb300.api import _stream_handle
    N, T, K = 2, 3, 4
    logits, teacher, tokens, mask, grad, _ = distill_inputs(N, T, V, K, dtype, V)
    dev = [t.to(DEV) for t in (logits, teacher, tokens)]
    m, w = mask.to(DEV), grad.to(DEV)
    loss, norm = L().distill_loss(*dev, 2.0, m, return_normalizers=True)
    g = L().distill_loss_backward(w, *dev, norm, 2.0, m)
    flat = torch.full((2 * N * T + 2,), 7.0, device=DEV)
    view = flat[1:-1].view(N, T, 2)
    view.copy_(norm)
    assert view.data_ptr() % 8 == 4
    assert torch.equal(L().distill_loss_backward(w, *dev, view, 2.0, m), g)
    lib, s = _native.lib(), _stream_handle(flat.device)
    args = tp._DISTILL_ARGS.pack(N, T, V, K, tp._TYPES[dtype], 0, 8, dev[0].data_ptr(), T * V, V, dev[1].data_ptr(), dev[2].data_ptr(),
                                 m.data_ptr(), 2.0)
    both_loss, both_norm, both_grad = torch.empty_like(loss), torch.empty_like(norm), torch.empty_like(g)
    assert lib.rlscan_distill_loss_and_grad(args, w.data_ptr(), both_loss.data_ptr(), both_norm.data_ptr(), both_grad.data_ptr(), s) == 0
    for call, want in ((lambda: lib.rlscan_distill_loss(args, loss.data_ptr(), view.data_ptr(), s), norm),
                       (lambda: lib.rlscan_distill_loss_and_grad(args, w.data_ptr(), both_loss.data_ptr(), view.data_ptr(),
                                                                 both_grad.data_ptr(), s), both_norm)):
        view.zero_()
        assert call() == 0 and torch.equal(view, want)
        assert flat[0] == 7 and flat[-1] == 7


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("V", [30, 5000, 60000])
@pytest.mark.parametrize("tau", [0.7, 0.01])
def test_tokens_that_the_student_masks(tau, V, dtype):
    """The teacher knows a token whose logit is the type's lowest value: the loss is large, but a float32 as long as the
    token's probability over the temperature times that value is one."""
    logits, teacher, tokens, _, grad, _ = distill_inputs(1, 3, V, 4, dtype, 3)
    tokens[0] = torch.arange(4)
    logits[0, :, 3] = torch.finfo(dtype).min
    teacher = 0.1 * teacher * tau
    teacher[0, :, 3] = teacher[0, :, :3].amax(-1) - 8 * tau   # exp(-8) / 0.01 is about 1/30
    loss, g = check(logits, teacher, tokens, None, grad, tau)
    assert (loss > 1e34).all() and torch.isfinite(loss).all() and torch.isfinite(g).all()


@pytest.mark.parametrize("V", [300, 5000, 60000])
def test_the_smallest_probability_of_a_token_ruled_out(V):
    """The student rules out a token to which a hot teacher gives exp(-87.2) / 200, next to float32's end: an infinite
    loss, no NaN."""
    K, tau = 200, 1e6
    z = torch.zeros(1, 2, V, device=DEV)
    z[..., K - 1] = -float("inf")
    teacher = torch.zeros(1, 2, K, device=DEV)
    teacher[..., K - 1] = -87.2 * tau
    tokens = torch.arange(K, device=DEV).expand(1, 2, K)
    loss, g = L().distill_loss_and_grad(torch.ones(1, 2, device=DEV), z, teacher, tokens, tau)
    assert (loss == float("inf")).all() and torch.isfinite(g).all()
    assert torch.equal(L().distill_loss(z, teacher, tokens, tau), loss)


@pytest.mark.parametrize("V", [30, 5000, 60000])
def test_tokens_at_both_ends_at_a_high_temperature(V):
    """Every teacher's token has the type's lowest value, the others 0 or 3e38: a difference past float32, but not over
    the temperature of 10."""
    logits, teacher, tokens, _, grad, _ = distill_inputs(1, 3, V, 4, F32, 4)
    tokens[0] = torch.arange(4)
    logits[0, :2], logits[0, 2] = 0, 3e38
    logits[..., :4] = torch.finfo(F32).min
    loss, g = check(logits, teacher, tokens, None, grad, 10.0)
    assert (loss > 3e37).all() and torch.isfinite(loss).all() and torch.isfinite(g).all()
