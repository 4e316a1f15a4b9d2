"""What is measured of the state-space layer's operators: the selective scan,
its short causal convolution and the root-mean-square norm in front of them,
each over prompts, in training and (scan and convolution) for single tokens.

``listed()`` gives the measured cases, ``draw(rng)`` more of the same ranges;
``prepare`` makes a case's inputs, ``run`` is one pass (in plain torch, or
with ``own`` through the framework's kernels), ``exact`` the same outputs in
64 bits and ``work`` the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
EPS = 1e-5
BLOCK = 128          # columns that share one scale of an 8-bit output
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100   # smallest block maximum a scale is made from


def listed():
    return [
        # one token of one conversation: the call's latency
        dict(name="scan_step_1x1536", op="scan_step", N=1, D=1536, S=16, dtype="bfloat16"),
        # one token of each of 256 running responses, states in a slot pool
        dict(name="scan_step_256x4096", op="scan_step", N=256, D=4096, S=16, dtype="bfloat16"),
        # a short prompt of one conversation, odd length: little work in parallel
        dict(name="scan_1x509x1536", op="scan", N=1, T=509, D=1536, S=16, dtype="bfloat16",
             ragged=False, packed=False),
        # two rows of 16384 tokens (the framework's Retrace length) packed with several episodes each
        dict(name="scan_2x16384x2048_packed", op="scan", N=2, T=16384, D=2048, S=16,
             dtype="bfloat16", ragged=False, packed=True),
        # a full batch of prompts, padded to the longest
        dict(name="scan_8x4096x4096_ragged", op="scan", N=8, T=4096, D=4096, S=16,
             dtype="bfloat16", ragged=True, packed=False),
        # training in 32 bits at odd sizes: odd row strides, a state that is no power of two
        dict(name="scan_train_3x1001x1111_f32", op="scan_train", N=3, T=1001, D=1111, S=12,
             dtype="float32", ragged=True, packed=False),
        # a training step's forward and backward over packed token rollouts
        dict(name="scan_train_8x2048x4096", op="scan_train", N=8, T=2048, D=4096, S=16,
             dtype="bfloat16", ragged=False, packed=True),
        # one token of each of 64 responses through the convolution
        dict(name="conv_step_64x4096", op="conv_step", N=64, D=4096, K=4, dtype="bfloat16"),
        # the convolution of a training step, forward and backward, packed rollouts
        dict(name="conv_train_8x4096x4096", op="conv_train", N=8, T=4096, D=4096, K=4,
             dtype="bfloat16", ragged=False, packed=True),
        # the norm of a decoding step: four tokens, 8-bit output for the next product
        dict(name="norm8_4x2048", op="norm8", N=4, D=2048, dtype="bfloat16"),
        # the norm over a full batch of prompts, 8-bit output
        dict(name="norm8_32768x4096", op="norm8", N=32768, D=4096, dtype="bfloat16"),
        # the norm in training, forward and backward, a width that is no power of two
        dict(name="norm_train_16384x2560", op="norm_train", N=16384, D=2560, dtype="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "conv", "conv_train",
                     "conv_step", "norm8", "norm", "norm_train"])
    c = dict(op=op, dtype=rng.choice(["bfloat16", "bfloat16", "float32"]))
    D = _log(rng, 64, 4096)
    c["D"] = D if rng.random() < 0.3 else max(16, D // 16 * 16)
    if op.startswith("norm"):
        c["N"] = _log(rng, 1, 32768)
        return c
    if op.startswith("scan"):
        c["S"] = rng.choice([16, 16, 16, 8, 32, 12])
    else:
        c["K"] = rng.choice([4, 4, 3, 2])
    c["N"] = _log(rng, 1, 256 if op.endswith("step") else 16)
    if not op.endswith("step"):
        T = _log(rng, 1, 16384)
        # a pass of a scan holds at most 2^30 state values (2^29 with its gradients), one of a convolution 2^27 inputs
        most = {"scan": 2 ** 30, "scan_train": 2 ** 29}.get(op, 2 ** 27 * 16)
        T = min(T, most // (c["N"] * c["D"] * c.get("S", 16)))
        c["T"] = max(1, T)
        c["ragged"] = rng.random() < 0.4
        c["packed"] = not c["ragged"] and rng.random() < 0.6
    return c


# ---------------------------------------------------------------------------
# inputs

def _flags(case, g):
    """resets: episodes of 512 tokens on average begin at a flag; lengths: rows of T/4 to T tokens, one of them full."""
    N, T = case["N"], case["T"]
    resets = lengths = None
    if case.get("packed"):
        resets = (torch.rand(N, T, generator=g, device=DEV) < 1 / 512).to(torch.uint8)
    if case.get("ragged"):
        low = max(1, T // 4)
        lengths = (low + torch.rand(N, generator=g, device=DEV) * (T - low + 1)).to(torch.int32).clamp_(max=T)
        lengths[N // 2] = T
    return resets, lengths


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, N, D, dtype = case["op"], case["N"], case["D"], TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(to)

    s = {"op": op}
    if op.startswith("norm"):
        s.update(x=normal(N, D), residual=normal(N, D, scale=2.0), weight=1 + normal(D, scale=0.2, to=torch.float32))
        if op == "norm_train":
            s.update(grad_y=normal(N, D), grad_residual=normal(N, D))
        return s
    if op.startswith("conv"):
        K = case["K"]
        s.update(weight=normal(D, K, scale=K ** -0.5, to=torch.float32), bias=normal(D, scale=0.1, to=torch.float32))
        if op == "conv_step":
            s.update(x=normal(N, D), state=normal(N + N // 4, K - 1, D),
                     slots=torch.randperm(N + N // 4, generator=g, device=DEV)[:N].to(torch.int32))
            return s
        # the projection's output holds the convolution's input beside the gate
        s["x"] = normal(N, case["T"], 2 * D)[..., :D]
        s["resets"], s["lengths"] = _flags(case, g)
        if op == "conv_train":
            s["grad_y"] = normal(N, case["T"], D)
        return s
    S = case["S"]
    # decay rates -1 .. -S for each channel and time steps between 1e-3 and 1e-1, as such layers begin
    rates = torch.arange(1, S + 1, device=DEV).float().repeat(D, 1)
    s["A"] = -rates * torch.exp(normal(D, S, scale=0.1, to=torch.float32))
    dt = torch.exp(torch.rand(D, generator=g, device=DEV) * math.log(100.0) + math.log(1e-3))
    s["delta_bias"] = dt + torch.log(-torch.expm1(-dt))
    s["D"] = 1 + normal(D, scale=0.1, to=torch.float32)
    lead = (N,) if op == "scan_step" else (N, case["T"])
    s["x"] = torch.nn.functional.silu(torch.randn(*lead, D, generator=g, device=DEV)).to(dtype)
    s["z"] = normal(*lead, 2 * D)[..., D:]
    s["delta"] = normal(*lead, D, scale=0.5)
    R = -(-D // 16 // 8) * 8   # the rank of the time steps' projection, whose output holds B and C too
    bc = normal(*lead, R + 2 * S)
    s["B"], s["C"] = bc[..., R:R + S], bc[..., R + S:]
    if op == "scan_step":
        s.update(state=normal(N + N // 4, D, S, scale=0.1, to=torch.float32),
                 slots=torch.randperm(N + N // 4, generator=g, device=DEV)[:N].to(torch.int32))
        return s
    s["resets"], s["lengths"] = _flags(case, g)
    if op == "scan_train":
        s["grad_y"] = normal(N, case["T"], D)
    else:
        s["initial_state"] = normal(N, D, S, scale=0.1, to=torch.float32)
    return s


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits, rounded once at the end

def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 1 from h = 0: pairs of steps are joined, the joined sequence is solved the same way, and the steps between follow."""
    T = a.shape[1]
    if T < 2:
        return b
    n = T // 2
    a1 = a[:, 1:2 * n:2]
    odd = _recurrence(a[:, 0:2 * n:2] * a1, b[:, 1:2 * n:2] + a1 * b[:, 0:2 * n:2])
    h = torch.empty_like(b)
    h[:, 1::2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = b[:, 2::2] + a[:, 2::2] * odd[:, :(T - 1) // 2]
    return h


def _inside(s):
    """[N,T] truth values of the tokens that are no padding, or None."""
    if s["lengths"] is None:
        return None
    return torch.arange(s["x"].shape[1], device=DEV)[None, :] < s["lengths"][:, None]


def _plain_scan(s, train):
    x, raw, B, C = (s[k].float() for k in ("x", "delta", "B", "C"))
    z, out = s["z"].float(), s["x"].dtype
    N, T, D = x.shape
    live = _inside(s)
    pre = raw + s["delta_bias"]
    dt = _softplus(pre)
    if live is not None:
        dt = dt * live[..., None]
    a = torch.exp(dt[..., None] * s["A"])
    if s["resets"] is not None:
        a = a * (s["resets"] == 0)[..., None, None]
    b = (dt * x)[..., None] * B[:, :, None, :]
    if not train:
        b[:, 0] += a[:, 0] * s["initial_state"]
    h = _recurrence(a, b)
    del b
    y = (h * C[:, :, None, :]).sum(-1) + s["D"] * x
    gate = torch.sigmoid(z)
    result = y * (z * gate)
    if live is not None:
        result = result * live[..., None]
    if not train:
        return result.to(out), h[:, -1].clone()
    gy = s["grad_y"].float()
    if live is not None:
        gy = gy * live[..., None]
    gz = gy * y * gate * (1 + z * (1 - gate))
    gy = gy * z * gate
    # the gradient of the states runs the same recurrence backwards
    back = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1).flip(1)
    gh = _recurrence(back, (gy[..., None] * C[:, :, None, :]).flip(1)).flip(1)
    del back
    gC = (gy[..., None] * h).sum(2)
    gB = (gh * (dt * x)[..., None]).sum(2)
    through = (gh * B[:, :, None, :]).sum(-1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1).mul_(a).mul_(gh)   # gh a h_{t-1}
    gA = (before * dt[..., None]).sum((0, 1))
    gdt = (before * s["A"]).sum(-1) + through * x
    graw = gdt * torch.sigmoid(pre)
    if live is not None:
        graw = graw * live[..., None]
    gx = through * dt + gy * s["D"]
    return (result.to(out), h[:, -1].clone(), gx.to(out), graw.to(out), gA, gB.to(out), gC.to(out),
            (gy * x).sum((0, 1)), gz.to(out), graw.sum((0, 1)))


def _plain_scan_step(s):
    x, z, at = s["x"].float(), s["z"].float(), s["slots"].long()
    dt = _softplus(s["delta"].float() + s["delta_bias"])
    h = s["state"][at] * torch.exp(dt[..., None] * s["A"]) + (dt * x)[..., None] * s["B"].float()[:, None, :]
    s["state"][at] = h
    y = (h * s["C"].float()[:, None, :]).sum(-1) + s["D"] * x
    return (y * z * torch.sigmoid(z)).to(s["x"].dtype), s["state"]


def _plain_conv(s, train):
    x, w = s["x"].float(), s["weight"]
    N, T, D = x.shape
    K, out = w.shape[1], s["x"].dtype
    live = _inside(s)
    padded = torch.cat([x.new_zeros(N, K - 1, D), x], 1)
    # the episode of each position: a tap counts where it lies in its token's episode
    resets = torch.zeros(N, T, device=DEV) if s["resets"] is None else s["resets"]
    episode = torch.cat([torch.zeros(N, K - 1, device=DEV), resets], 1).cumsum(1)
    taps = padded.unfold(1, K, 1) * (episode.unfold(1, K, 1) == episode[:, K - 1:, None])[:, :, None, :]
    pre = (taps * w).sum(-1) + s["bias"]
    gate = torch.sigmoid(pre)
    y = pre * gate
    if live is not None:
        y = y * live[..., None]
    last = torch.full((N,), T, device=DEV) if live is None else s["lengths"].long()
    at = last[:, None] + torch.arange(K - 1, device=DEV)   # positions in `padded` of the K-1 last inputs
    state = torch.gather(padded, 1, at[..., None].expand(-1, -1, D))
    state = state * (torch.gather(episode, 1, at) == torch.gather(episode, 1, (last + K - 2)[:, None]))[..., None]
    if not train:
        return y.to(out), state.to(out)
    g = s["grad_y"].float() * gate * (1 + pre * (1 - gate))
    if live is not None:
        g = g * live[..., None]
    gw = (taps * g[..., None]).sum((0, 1))
    # a token's gradient comes from its own output and the K-1 after it, of its episode
    after = torch.nn.functional.pad(g, (0, 0, 0, K - 1)).unfold(1, K, 1)
    episode = torch.nn.functional.pad(episode[:, K - 1:], (0, K - 1), value=-1.0)
    after = after * (episode.unfold(1, K, 1) == episode[:, :T, None])[:, :, None, :]
    gx = (after * w.flip(1)).sum(-1)
    return y.to(out), state.to(out), gx.to(out), gw, g.sum((0, 1))


def _plain_conv_step(s):
    at, x = s["slots"].long(), s["x"]
    window = torch.cat([s["state"][at], x[:, None, :]], 1)
    s["state"][at] = window[:, 1:]
    pre = (window.float() * s["weight"].t()).sum(1) + s["bias"]
    return (pre * torch.sigmoid(pre)).to(x.dtype), s["state"]


def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    return h * r * s["weight"], h.to(s["x"].dtype)


def _plain_norm8(s):
    y, h = _plain_norm(s)
    N, D = y.shape
    blocks = torch.nn.functional.pad(y, (0, -D % BLOCK)).view(N, -1, BLOCK)
    scales = blocks.abs().amax(-1).clamp(min=SCALE_FLOOR) / E4M3_MAX
    q = (blocks / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(N, -1)[:, :D], scales, h


def _plain_norm_train(s):
    y, stored = _plain_norm(s)
    out, w, D = s["x"].dtype, s["weight"], s["x"].shape[1]
    h, gy = stored.float(), s["grad_y"].float()
    r = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n, gn = h * r, gy * w
    gh = r * (gn - n * ((gn * n).sum(-1, keepdim=True) / D)) + s["grad_residual"].float()
    return y.to(out), stored, gh.to(out), (gy * n).sum(0)


# ---------------------------------------------------------------------------
# the framework's calls

def _own(s):
    import linear_recurrence_scan_gb300 as rl
    op = s["op"]
    if op == "scan":
        return rl.selective_scan(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["delta_bias"],
                                 initial_state=s["initial_state"], resets=s["resets"], lengths=s["lengths"])
    if op == "scan_train":
        y, final, kept = rl.selective_scan(s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                           s["delta_bias"], resets=s["resets"], lengths=s["lengths"],
                                           return_checkpoints=True)
        g = rl.selective_scan_backward(s["grad_y"], s["x"], s["delta"], s["A"], s["B"], s["C"], kept, s["D"], s["z"],
                                       s["delta_bias"], resets=s["resets"], lengths=s["lengths"])
        return y, final, g.x, g.delta, g.A, g.B, g.C, g.D, g.z, g.delta_bias
    if op == "scan_step":
        y = rl.selective_scan_step(s["state"], s["x"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"],
                                   s["delta_bias"], slots=s["slots"])
        return y, s["state"]
    if op == "conv":
        return rl.causal_conv(s["x"], s["weight"], s["bias"], resets=s["resets"], lengths=s["lengths"])
    if op == "conv_train":
        y, state = rl.causal_conv(s["x"], s["weight"], s["bias"], resets=s["resets"], lengths=s["lengths"])
        g = rl.causal_conv_backward(s["grad_y"], s["x"], s["weight"], s["bias"], resets=s["resets"],
                                    lengths=s["lengths"])
        return y, state, g.x, g.weight, g.bias
    if op == "conv_step":
        return rl.causal_conv_step(s["state"], s["x"], s["weight"], s["bias"], slots=s["slots"]), s["state"]
    if op == "norm8":
        n = rl.add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS, out_dtype=torch.float8_e4m3fn)
        return n.y, n.scales, n.residual
    n = rl.add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
    if op == "norm":
        return n.y, n.residual
    g = rl.add_rms_norm_backward(s["grad_y"], n.residual, s["weight"], s["grad_residual"], eps=EPS)
    return n.y, n.residual, g.x, g.weight


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op in ("scan", "scan_train"):
        return _plain_scan(state, op == "scan_train")
    if op in ("conv", "conv_train"):
        return _plain_conv(state, op == "conv_train")
    if op == "norm":
        y, h = _plain_norm(state)
        return y.to(h.dtype), h
    return {"scan_step": _plain_scan_step, "conv_step": _plain_conv_step, "norm8": _plain_norm8,
            "norm_train": _plain_norm_train}[op](state)


# ---------------------------------------------------------------------------
# bytes and operations

def work(case):
    op, N, D = case["op"], case["N"], case["D"]
    e = 2 if case["dtype"] == "bfloat16" else 4
    if op.startswith("norm"):
        n = N * D
        if op == "norm8":
            return {"bytes": n * (3 * e + 1) + 4 * N * -(-D // BLOCK) + 4 * D, "flops": 7 * n}
        if op == "norm":
            return {"bytes": n * 4 * e + 4 * D, "flops": 5 * n}
        return {"bytes": n * 8 * e + 8 * D, "flops": 17 * n}   # forward 4; backward reads 3, writes 1
    if op.startswith("conv"):
        K = case["K"]
        if op == "conv_step":   # the state is read and written
            return {"bytes": N * D * e * (2 + 2 * (K - 1)) + 4 * D * (K + 1), "flops": N * D * (2 * K + 5)}
        n = N * case["T"] * D
        if op == "conv":
            return {"bytes": 2 * n * e, "flops": n * (2 * K + 5)}
        return {"bytes": 5 * n * e, "flops": n * (8 * K + 20)}   # forward 2; backward reads 2, writes 1
    S = case["S"]
    if op == "scan_step":
        return {"bytes": N * (8 * D * S + 4 * D * e + 2 * S * e) + 4 * D * (S + 2), "flops": N * D * (7 * S + 20)}
    n = N * case["T"] * D
    if op == "scan":   # x, delta, z read, y written; product, exponential, product, two multiply-adds a state
        return {"bytes": 4 * n * e + 2 * N * case["T"] * S * e + 8 * N * D * S + 4 * D * (S + 2),
                "flops": n * (7 * S + 20)}
    # backward: x, delta, z, grad_y read, three gradients written; states made again and run backwards
    return {"bytes": 11 * n * e + 6 * N * case["T"] * S * e + 4 * N * D * S + 12 * D * (S + 2),
            "flops": n * (7 * S + 20) + n * (25 * S + 40)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one token after the other

def _sigmoid64(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _exact_scan(s, train):
    f = {k: s[k].double() for k in ("x", "delta", "A", "B", "C", "D", "z", "delta_bias")}
    N, T, D = s["x"].shape
    S = s["A"].shape[1]
    h = torch.zeros(N, D, S, dtype=torch.float64, device=DEV) if train else s["initial_state"].double()
    pre = f["delta"] + f["delta_bias"]
    dt = torch.logaddexp(pre, torch.zeros((), dtype=torch.float64, device=DEV))
    length = torch.full((N,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    y = torch.zeros(N, T, D, dtype=torch.float64, device=DEV)
    kept = torch.empty(T + 1, N, D, S, dtype=torch.float64, device=DEV) if train else None
    reset = torch.zeros(N, T, dtype=torch.bool, device=DEV) if s["resets"] is None else s["resets"] != 0
    for t in range(T):
        if train:
            kept[t] = h
        start = torch.where(reset[:, t, None, None], 0.0, h)
        new = torch.exp(dt[:, t, :, None] * f["A"]) * start + (dt[:, t] * f["x"][:, t])[..., None] * f["B"][:, t, None, :]
        h = torch.where((t < length)[:, None, None], new, h)
        y[:, t] = (h * f["C"][:, t, None, :]).sum(-1) + f["D"] * f["x"][:, t]
    live = (torch.arange(T, device=DEV)[None, :] < length[:, None])[..., None]
    sg = _sigmoid64(f["z"])
    result = torch.where(live, y * f["z"] * sg, 0.0)
    if not train:
        return result, h
    kept[T] = h
    gout = torch.where(live, s["grad_y"].double(), 0.0)
    gz = gout * y * (sg + f["z"] * sg * (1 - sg))
    gy = gout * f["z"] * sg
    del gout, result
    result = y.mul_(f["z"] * sg).mul_(live)
    gx, gpre = torch.empty_like(dt), torch.empty_like(dt)
    gB, gC = torch.empty_like(f["B"]), torch.empty_like(f["C"])
    gA, gh = torch.zeros_like(f["A"]), torch.zeros(N, D, S, dtype=torch.float64, device=DEV)
    for t in range(T - 1, -1, -1):
        on = (t < length)[:, None]
        gh = gh + gy[:, t, :, None] * f["C"][:, t, None, :]
        gC[:, t] = (gy[:, t, :, None] * kept[t + 1]).sum(1)
        prior = torch.where(reset[:, t, None, None], 0.0, kept[t])
        a = torch.exp(dt[:, t, :, None] * f["A"])
        drive = torch.where(on, (gh * f["B"][:, t, None, :]).sum(-1), 0.0)
        gB[:, t] = torch.where(on, (gh * (dt[:, t] * f["x"][:, t])[..., None]).sum(1), 0.0)
        decay = torch.where(on[..., None], gh * a * prior, 0.0)
        gA += (decay * dt[:, t, :, None]).sum(0)
        gpre[:, t] = ((decay * f["A"]).sum(-1) + drive * f["x"][:, t]) * _sigmoid64(pre[:, t])
        gx[:, t] = drive * dt[:, t] + gy[:, t] * f["D"]
        back = torch.where(reset[:, t, None, None], 0.0, gh * a)
        gh = torch.where(on[..., None], back, gh)
    return result, h, gx, gpre, gA, gB, gC, (gy * f["x"]).sum((0, 1)), gz, gpre.sum((0, 1))


def _exact_scan_step(s):
    state, at = s["state"].double(), s["slots"].long()
    dt = torch.logaddexp(s["delta"].double() + s["delta_bias"].double(), torch.zeros((), dtype=torch.float64, device=DEV))
    x, z = s["x"].double(), s["z"].double()
    h = torch.exp(dt[..., None] * s["A"].double()) * state[at] + (dt * x)[..., None] * s["B"].double()[:, None, :]
    state[at] = h
    return (torch.einsum("nds,ns->nd", h, s["C"].double()) + s["D"].double() * x) * z * _sigmoid64(z), state


def _exact_conv(s, train):
    x, w = s["x"].double(), s["weight"].double()
    N, T, D = x.shape
    K = w.shape[1]
    length = [T] * N if s["lengths"] is None else s["lengths"].tolist()
    resets = torch.zeros(N, T, dtype=torch.int64, device=DEV) if s["resets"] is None else s["resets"].long()
    episode = torch.cumsum(resets, 1)
    live = torch.arange(T, device=DEV)[None, :] < torch.tensor(length, device=DEV)[:, None]

    def same(d):   # tokens whose neighbour d before them is of their episode
        return (episode[:, d:] == episode[:, :T - d])[..., None]

    pre = s["bias"].double().expand(N, T, D).clone()
    for d in range(min(K, T)):
        pre[:, d:] += torch.where(same(d), x[:, :T - d] * w[:, K - 1 - d], 0.0)
    sg = _sigmoid64(pre)
    y = torch.where(live[..., None], pre * sg, 0.0)
    state = torch.zeros(N, K - 1, D, dtype=torch.float64, device=DEV)
    for n in range(N):
        for k in range(K - 1):
            t = length[n] - (K - 1) + k
            if t >= 0 and bool(episode[n, t] == episode[n, length[n] - 1]):
                state[n, k] = x[n, t]
    if not train:
        return y, state
    g = torch.where(live[..., None], s["grad_y"].double() * (sg + pre * sg * (1 - sg)), 0.0)
    gx, gw = torch.zeros_like(x), torch.zeros_like(w)
    for d in range(min(K, T)):
        gd = torch.where(same(d), g[:, d:], 0.0)
        gx[:, :T - d] += gd * w[:, K - 1 - d]
        gw[:, K - 1 - d] = (gd * x[:, :T - d]).sum((0, 1))
    return y, state, gx, gw, g.sum((0, 1))


def _exact_conv_step(s):
    state, at, x = s["state"].double(), s["slots"].long(), s["x"].double()
    w = s["weight"].double()
    K = w.shape[1]
    pre = s["bias"].double() + x * w[:, K - 1]
    old = state[at]
    for k in range(K - 1):
        pre = pre + old[:, k] * w[:, k]
    state[at] = torch.cat([old[:, 1:], x[:, None]], 1)
    return pre * _sigmoid64(pre), state


def _exact_norm(s, op):
    h, w = s["x"].double() + s["residual"].double(), s["weight"].double()
    D = h.shape[1]
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / D + EPS) * w
    if op == "norm":
        return y, h
    if op == "norm8":
        scales = torch.empty(h.shape[0], -(-D // BLOCK), dtype=torch.float64, device=DEV)
        q = torch.empty_like(y)
        for b in range(scales.shape[1]):
            part = y[:, b * BLOCK:(b + 1) * BLOCK]
            scales[:, b] = part.abs().max(1).values.clamp(min=SCALE_FLOOR) / E4M3_MAX
            q[:, b * BLOCK:(b + 1) * BLOCK] = part / scales[:, b:b + 1]
        return q, scales, h
    # the backward pass works from the sum as it is stored, in the inputs' type
    k = (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
    root = torch.sqrt((k * k).sum(1, keepdim=True) / D + EPS)
    gy = s["grad_y"].double()
    gh = gy * w / root - k * ((gy * w * k).sum(1, keepdim=True) / (D * root ** 3)) + s["grad_residual"].double()
    return y, h, gh, (gy * k / root).sum(0)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("scan", "scan_train"):
        return _exact_scan(s, op == "scan_train")
    if op in ("conv", "conv_train"):
        return _exact_conv(s, op == "conv_train")
    if op == "scan_step":
        return _exact_scan_step(s)
    if op == "conv_step":
        return _exact_conv_step(s)
    return _exact_norm(s, op)
