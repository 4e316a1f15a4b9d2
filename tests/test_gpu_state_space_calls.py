"""The state-space layer's calls as torch sees them: what autograd follows,
refuses and notices, the device a call runs on, empty arrays."""
import pytest
import torch

from state_space_cases import DEV, scan_inputs, to_dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def L():
    import linear_recurrence_scan_gb300 as lib
    return lib


@pytest.fixture(params=["native", "python"])
def layer(request, monkeypatch):
    """The calls through the native call layer and the Python way."""
    from linear_recurrence_scan_gb300 import state_space as ss
    ss._load_fast()
    if request.param == "python":
        monkeypatch.setattr(ss, "_fast", ss._NoFastCall)
    return request.param


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_scan_without_channels_or_rows(layer, dtype):
    """Nothing to scan over many tokens: empty results, and gradients of B and C that are zeros, not left as they were."""
    T, S = 600, 16
    for N, D in ((2, 0), (0, 64), (0, 0)):
        x, bc = torch.zeros(N, T, D, dtype=dtype, device=DEV), torch.randn(N, T, S, device=DEV).to(dtype)
        A, D1 = -torch.ones(D, S, device=DEV), torch.ones(D, device=DEV)
        y, final = L().selective_scan(x, x, A, bc, bc, D1, x, D1)
        assert y.shape == (N, T, D) and final.shape == (N, D, S)
        _, _, marks = L().selective_scan(x, x, A, bc, bc, D1, x, D1, return_checkpoints=True)
        for _ in range(2):   # what the allocator hands out next is not zero
            junk = [torch.full((N, T, S), 7.0, dtype=dtype, device=DEV) for _ in range(8)]
            del junk
            g = L().selective_scan_backward(x, x, x, A, bc, bc, marks, D1, x, D1)
            assert g.B.shape == g.C.shape == (N, T, S) and not g.B.any() and not g.C.any()
            assert g.x.shape == x.shape and g.A.shape == (D, S) and not g.A.any() and not g.D.any()


def test_checkpoints_do_not_detach(layer):
    """return_checkpoints with inputs that want a gradient: the same gradients as without."""
    N, T, D, S = 2, 40, 32, 16
    a, init, resets, _, _ = scan_inputs(N, T, D, S, F32, 41, "packed")
    grads = []
    for more in (False, True):
        leaves = {k: v.to(DEV).requires_grad_() for k, v in {**a, "initial_state": init}.items()}
        out = L().selective_scan(**leaves, resets=to_dev(resets), return_checkpoints=more)
        assert out[0].requires_grad and out[1].requires_grad and len(out) == 2 + more
        if more:
            assert not out[2].requires_grad
            plain = L().selective_scan(**{k: v.detach() for k, v in leaves.items()}, resets=to_dev(resets),
                                       return_checkpoints=True)
            assert all(torch.equal(p, q) for p, q in zip(out, plain))
        (out[0].square().sum() + out[1].sum()).backward()
        grads.append([v.grad for v in leaves.values()])
    for p, q in zip(*grads):
        assert torch.equal(p, q)


def test_forward_mode_is_refused(layer):
    """A tangent would be lost without a word: dual tensors are refused, others pass inside a dual level."""
    import torch.autograd.forward_ad as fwd
    N, T, D, S, K = 2, 20, 16, 4, 4
    a, init, _, _, _ = scan_inputs(N, T, D, S, F32, 42)
    dev = {k: v.to(DEV) for k, v in a.items()}
    step = {k: (v[:, 0].contiguous() if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
    x, w, nw = dev["x"], torch.randn(D, K, device=DEV), torch.ones(D, device=DEV)
    _, _, marks = L().selective_scan(**dev, return_checkpoints=True)
    scan = ("x", "delta", "A", "B", "C", "D", "z", "delta_bias")
    calls = [(lambda f, k=k: L().selective_scan(**{**dev, k: f(dev[k])})) for k in scan]
    calls += [(lambda f, k=k: L().selective_scan_step(init.to(DEV), **{**step, k: f(step[k])})) for k in scan]
    calls += [
        lambda f: L().selective_scan(**dev, initial_state=f(init.to(DEV))),
        lambda f: L().selective_scan(**{**dev, "x": f(x)}, return_checkpoints=True),
        lambda f: L().selective_scan_step(f(init.to(DEV)), **step),
        lambda f: L().selective_scan_backward(f(x), x, dev["delta"], dev["A"], dev["B"], dev["C"], marks),
        lambda f: L().selective_scan_backward(x, x, f(dev["delta"]), dev["A"], dev["B"], dev["C"], marks),
        lambda f: L().causal_conv(f(x), w), lambda f: L().causal_conv(x, f(w)), lambda f: L().causal_conv(x, w, f(nw)),
        lambda f: L().causal_conv(x, w, initial_state=f(torch.zeros(N, K - 1, D, device=DEV))),
        lambda f: L().causal_conv_step(torch.zeros(N, K - 1, D, device=DEV), f(step["x"]), w),
        lambda f: L().causal_conv_backward(f(x), x, w), lambda f: L().causal_conv_backward(x, x, f(w)),
        lambda f: L().add_rms_norm(f(step["x"]), nw), lambda f: L().add_rms_norm(step["x"], f(nw)),
        lambda f: L().add_rms_norm(step["x"], nw, f(step["x"])),
        lambda f: L().add_rms_norm(f(step["x"]), nw, out_dtype=torch.float8_e4m3fn),
        lambda f: L().add_rms_norm_backward(f(step["x"]), step["x"], nw),
        lambda f: L().add_rms_norm_backward(step["x"], f(step["x"]), nw)]
    with fwd.dual_level():
        for call in calls:
            call(lambda t: t)
            with pytest.raises(RuntimeError, match="forward-mode"):
                call(lambda t: fwd.make_dual(t, torch.ones_like(t)))
            with pytest.raises(RuntimeError, match="forward-mode"), torch.no_grad():
                call(lambda t: fwd.make_dual(t, torch.ones_like(t)))


def test_states_updated_in_place_are_seen_by_autograd(layer):
    """A step changes its state: a graph that saved the state refuses to go back with the changed one."""
    N, T, D, S, K = 2, 12, 16, 4, 4
    a, init, _, _, _ = scan_inputs(N, T, D, S, F32, 43)
    dev = {k: v.to(DEV) for k, v in a.items()}
    step = {k: (v[:, 0].contiguous() if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
    state, window, w = init.to(DEV), torch.randn(N, K - 1, D, device=DEV), torch.randn(D, K, device=DEV)
    scale = torch.ones(1, device=DEV, requires_grad=True)
    kept, before = scale * state, (state._version, window._version)
    y, _ = L().causal_conv(dev["x"], w.clone().requires_grad_(), initial_state=window)
    with torch.no_grad():
        L().selective_scan_step(state, **step)
        L().causal_conv_step(window, step["x"], w)
    assert state._version > before[0] and window._version > before[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.sum().backward()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():   # tensors without a version counter
        L().selective_scan_step(init.to(DEV), **step)
        L().causal_conv_step(torch.zeros(N, K - 1, D, device=DEV), step["x"], w)


def test_a_call_runs_on_its_tensors_device(monkeypatch):
    """Another device is current (as far as the calls can tell): each makes its tensors' own current while it plans
    and launches, and the native call layer leaves the call to Python."""
    from linear_recurrence_scan_gb300 import state_space as ss
    N, T, D, S, K = 2, 20, 16, 4, 4
    a, init, _, _, _ = scan_inputs(N, T, D, S, F32, 44)
    dev = {k: v.to(DEV) for k, v in a.items()}
    step = {k: (v[:, 0].contiguous() if k in ("x", "delta", "z", "B", "C") else v) for k, v in dev.items()}
    x, w, nw = dev["x"], torch.randn(D, K, device=DEV), torch.ones(D, device=DEV)
    y, _, marks = L().selective_scan(**dev, return_checkpoints=True)
    rows = step["x"]

    def calls():
        state, window = init.to(DEV), torch.ones(N, K - 1, D, device=DEV)
        yield L().selective_scan(**dev)
        yield L().selective_scan_backward(y, x, dev["delta"], dev["A"], dev["B"], dev["C"], marks)
        yield L().selective_scan_step(state, **step), state
        yield L().causal_conv(x, w)
        yield L().causal_conv_backward(y, x, w)
        yield L().causal_conv_step(window, rows, w), window
        yield L().add_rms_norm(rows, nw, rows)
        yield L().add_rms_norm_backward(rows, rows, nw, rows)

    want = list(calls())
    entered, now = [], [7]

    class Device(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            now[0] = self.idx
            super().__enter__()

        def __exit__(self, *args):
            now[0] = 7
            return super().__exit__(*args)

    lib = ss._native.lib()

    class Watched:
        """the library, used on the tensors' device alone"""
        def __getattr__(self, name):
            assert now[0] == 0, name
            return getattr(lib, name)

    fast = ss._load_fast()
    monkeypatch.setattr(ss, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    try:
        ss._setup(fast)
        assert fast.add_rms_norm(rows, nw, None, 1e-6, None) is None and fast.causal_conv(x, w, None, "silu", None, None,
                                                                                          None) is None
        monkeypatch.setattr(ss._native, "lib", Watched)
        got = list(calls())
        assert entered == [0] * len(want) and now == [7]
    finally:
        monkeypatch.undo()
        ss._setup(fast)
    assert fast is ss._NoFastCall or fast.add_rms_norm(rows, nw, None, 1e-6, None) is not None
    for p, q in zip(want, got):
        for u, v in zip(p, q):
            assert (u is None and v is None) or torch.equal(u, v)


ORDER = """
import ctypes, sys, torch
import linear_recurrence_scan_gb300 as rl

class KernelNode(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS
    _fields_ = ([("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in "gx gy gz bx by bz smem".split()] +
                [(n, ctypes.c_void_p) for n in "params extra kern ctx".split()])

def grids(graph):
    cuda, g, n = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert cuda.cuGraphGetNodes(g, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cuda.cuGraphGetNodes(g, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        kind, p = ctypes.c_int(), KernelNode()
        assert cuda.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cuda.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)) == 0
            out.append((p.gx, p.bx))
    return sorted(out)

def call(dtype):   # 14 warps a row in either type
    D = 3584 if dtype is torch.float32 else 7168
    x, r = (torch.randn(4001, D, device="cuda").to(dtype) for _ in range(2))
    w = torch.ones(D, device="cuda")
    rl.add_rms_norm(x, w, r), rl.add_rms_norm_backward(x, r, w, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        rl.add_rms_norm(x, w, r), rl.add_rms_norm_backward(x, r, w, x)
    return grids(graph)

found = {name: call(getattr(torch, name)) for name in sys.argv[1].split(",")}
print(sorted(found.items()))
"""


def test_the_first_type_of_a_process_does_not_shape_the_others():
    """The norm's grids are those of the call's own kernel, whichever type ran first."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    grids = []
    for order in ("float32,bfloat16", "bfloat16,float32"):
        r = subprocess.run([sys.executable, "-c", ORDER, order], capture_output=True, text=True, cwd=root, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        grids.append(r.stdout.splitlines()[-1])
    assert grids[0].count("(") >= 2 * 3 and grids[0] == grids[1]


def test_norm_without_channels_or_weight(layer):
    for shape in ((2, 3, 0), (3, 0), (0, 3, 5), (2, 0, 5)):
        x, w = torch.zeros(shape, device=DEV), torch.ones(shape[-1], device=DEV)
        n = L().add_rms_norm(x, w, x)
        assert n.y.shape == n.residual.shape == shape
        q = L().add_rms_norm(x, w, x, out_dtype=torch.float8_e4m3fn)
        assert q.y.shape == shape and q.scales.shape == (*shape[:-1], -(-shape[-1] // 128))
        g = L().add_rms_norm_backward(x, x, w, x)
        assert g.x.shape == shape and g.weight.shape == w.shape and not g.weight.any()
    with pytest.raises(TypeError, match="weight"):
        L().add_rms_norm(torch.zeros(2, 8, device=DEV), None)
    with pytest.raises(TypeError, match="weight"):
        L().add_rms_norm_backward(torch.zeros(2, 8, device=DEV), torch.zeros(2, 8, device=DEV), None)


def test_a_float32_residual_through_autograd():
    M, D = 37, 200
    x, nw = torch.randn(M, D, device=DEV).to(BF16), torch.rand(D, device=DEV) + 0.5
    r, gy, gr = torch.randn(M, D, device=DEV), torch.randn(M, D, device=DEV).to(BF16), torch.randn(M, D, device=DEV)
    leaves = [t.clone().requires_grad_() for t in (x, nw, r)]
    n = L().add_rms_norm(*leaves, eps=1e-5)
    assert n.y.dtype == BF16 and n.residual.dtype == F32
    torch.autograd.backward([n.y, n.residual], [gy, gr])
    g = L().add_rms_norm_backward(gy, n.residual.detach(), nw, gr, eps=1e-5)
    assert torch.equal(leaves[0].grad, g.x) and torch.equal(leaves[1].grad, g.weight)
    assert leaves[2].grad.dtype == F32 and torch.equal(leaves[2].grad, g.residual)


def test_captured_steps(layer):
    """A token of a layer in a graph: norm, convolution and scan steps, replayed on new inputs and moving states."""
    N, D, S, K = 5, 64, 16, 4
    a, init, _, _, _ = scan_inputs(N, 1, D, S, BF16, 45, step=True)
    dev = {k: v.to(DEV) for k, v in a.items()}
    w, nw = torch.randn(D, K, device=DEV), torch.ones(D, device=DEV)
    slots = torch.tensor([4, 0, -1, 2, 1], dtype=torch.int32, device=DEV)
    residual = torch.randn(N, D, device=DEV)

    def token(state, window):
        n = L().add_rms_norm(dev["x"], nw, residual)
        x = L().causal_conv_step(window, n.y, w, slots=slots)
        return L().selective_scan_step(state, **{**dev, "x": x}, slots=slots), n.residual

    states = [(init.to(DEV), torch.zeros(N, K - 1, D, device=DEV).to(BF16)) for _ in range(2)]
    for s in states:
        token(*s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token(*states[0])
    for seed in (46, 47):
        b, _, _, _, _ = scan_inputs(N, 1, D, S, BF16, seed, step=True)
        for k in ("x", "delta", "z", "B", "C"):
            dev[k].copy_(b[k])
        graph.replay()
        want = token(*states[1])
        for p, q in zip((*out, *states[0]), (*want, *states[1])):
            assert torch.equal(p, q)
