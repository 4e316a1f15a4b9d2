"""What is measured of a token policy's gated recurrent block and of the loss
that teaches it from another model: the gated recurrence (``gated_scan``), the
feed-forward block's two projections with the activation and the product
(``gated_projection``) and the distillation from a teacher's top logits
(``distill_loss``), each with its gradients, and for single tokens where a
policy answers token by token.

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


def listed():
    return [
        # one token of one conversation: the call's latency
        dict(name="scan_step_1x1536", op="scan_step", N=1, D=1536, dtype="bfloat16"),
        # one token of each of 256 running responses, states in a slot pool
        dict(name="scan_step_256x4096", op="scan_step", N=256, D=4096, dtype="bfloat16"),
        # a short prompt of one conversation, odd length: little work in parallel
        dict(name="scan_1x509x1536", op="scan", N=1, T=509, D=1536, dtype="bfloat16", ragged=False, packed=False),
        # two rows of 16384 tokens (the framework's Retrace length) packed with several episodes each
        dict(name="scan_2x16384x2048_packed", op="scan", N=2, T=16384, D=2048, dtype="bfloat16",
             ragged=False, packed=True),
        # training in 32 bits at odd sizes, rows padded to the longest
        dict(name="scan_train_3x1001x1111_f32", op="scan_train", N=3, T=1001, D=1111, dtype="float32",
             ragged=True, packed=False),
        # a training step's forward and backward over packed token rollouts
        dict(name="scan_train_8x2048x4096", op="scan_train", N=8, T=2048, D=4096, dtype="bfloat16",
             ragged=False, packed=True),
        # the feed-forward block of one token: the weights are read for a single row
        dict(name="projection_1x2048x8192", op="projection", M=1, D=2048, F=8192, act="silu"),
        # the feed-forward block over a batch of prompts
        dict(name="projection_16384x4096x12288", op="projection", M=16384, D=4096, F=12288, act="silu"),
        # the block's forward and backward over the tokens of a training step, sizes that fill no whole tiles
        dict(name="projection_train_5000x2560x6912", op="projection_train", M=5000, D=2560, F=6912, act="gelu"),
        # the example policy's vocabulary and rollouts: a small step's forward and backward
        dict(name="distill_train_8x40x64_f32", op="distill_train", N=8, T=40, V=64, K=8, dtype="float32", tau=1.0,
             masked=True),
        # the teacher's divergence as a reward of every token of long responses: no gradient
        dict(name="distill_8x1024x131072", op="distill", N=8, T=1024, V=131072, K=64, dtype="bfloat16", tau=1.0,
             masked=False),
        # a training step with an odd vocabulary, prompts masked
        dict(name="distill_train_4x1023x50257", op="distill_train", N=4, T=1023, V=50257, K=32, dtype="bfloat16",
             tau=2.0, masked=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "projection", "projection",
                     "projection_train", "projection_train", "distill", "distill_train", "distill_train"])
    c = dict(op=op)
    if op.startswith("projection"):
        c["M"] = _log(rng, 1, 16384)
        D = _log(rng, 64, 4096)
        F = _log(rng, 64, 12288)
        odd = rng.random() < 0.25
        c["D"], c["F"] = (D, F) if odd else (D // 16 * 16, F // 16 * 16)
        c["act"] = rng.choice(["silu", "silu", "gelu"])
        if op == "projection_train":   # eight products where a forward pass has two
            c["M"] = max(1, min(c["M"], 5000 * 2560 * 6912 // (c["D"] * c["F"])))
        return c
    c["dtype"] = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op.startswith("distill"):
        c["V"] = _log(rng, 16, 131072)
        c["K"] = min(c["V"], _log(rng, 1, 128))
        c["N"] = _log(rng, 1, 16)
        most = 2 ** 30 if op == "distill" else 2 ** 27 * 3 // 2   # logits of a pass
        c["T"] = max(1, min(_log(rng, 1, 4096), most // (c["N"] * c["V"])))
        c["tau"] = rng.choice([1.0, 1.0, 2.0, 0.7])
        c["masked"] = rng.random() < 0.5
        return c
    D = _log(rng, 64, 4096)
    c["D"] = D if rng.random() < 0.3 else max(16, D // 16 * 16)
    c["N"] = _log(rng, 1, 256 if op == "scan_step" else 16)
    if op != "scan_step":
        c["T"] = max(1, min(_log(rng, 1, 16384), 2 ** 26 // (c["N"] * c["D"])))
        c["ragged"] = rng.random() < 0.4
        c["packed"] = not c["ragged"] and rng.random() < 0.6
    return c


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    dtype = TYPES[case.get("dtype", "bfloat16")]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(to)

    s = {"op": op}
    if op.startswith("projection"):
        M, D, F = case["M"], case["D"], case["F"]
        s.update(act=case["act"], x=normal(M, D), gate_weight=normal(F, D, scale=D ** -0.5),
                 up_weight=normal(F, D, scale=D ** -0.5))
        if op == "projection_train":
            s["grad_h"] = normal(M, F)
        return s
    if op.startswith("distill"):
        N, T, V, K = (case[k] for k in "NTVK")
        s["tau"] = case["tau"]
        # K different tokens: a random start and a step that has no divisor in common with V
        step = next(k for k in range(max(1, V // 3), 2 * V + 2) if math.gcd(k, V) == 1)
        first = (torch.rand(N, T, 1, generator=g, device=DEV) * V).long().clamp_(max=V - 1)
        s["teacher_tokens"] = (first + torch.arange(K, device=DEV) * step) % V
        s["teacher_logits"] = normal(N, T, K, scale=2.0, to=torch.float32).sort(-1, descending=True).values
        # the student finds the teacher's tokens likely too
        logits = torch.randn(N, T, V, generator=g, device=DEV)
        logits.scatter_add_(2, s["teacher_tokens"], 0.5 * s["teacher_logits"] + 6.0)
        s["logits"] = logits.to(dtype)
        s["mask"] = None
        if case["masked"]:   # the prompt: the first quarter of a row
            s["mask"] = (torch.arange(T, device=DEV) >= T // 4).to(torch.uint8).expand(N, T).contiguous()
        if op == "distill_train":
            s["grad_loss"] = (0.5 + torch.rand(N, T, generator=g, device=DEV)) / (N * T)
        return s
    N, D = case["N"], case["D"]
    # decays between 0.9 and 0.999 a token where the gate is fully open, as such layers begin
    s["log_decay"] = torch.log(0.9 + 0.099 * torch.rand(D, generator=g, device=DEV))
    lead = (N,) if op == "scan_step" else (N, case["T"])
    s["x"] = normal(*lead, D)
    gates = normal(*lead, 2 * D)   # one projection's output holds both gates
    s["gate"], s["input_gate"] = gates[..., :D], gates[..., D:]
    if op == "scan_step":
        s.update(state=normal(N + N // 4, D, scale=0.5, to=torch.float32),
                 slots=torch.randperm(N + N // 4, generator=g, device=DEV)[:N].to(torch.int32))
        return s
    T = case["T"]
    s["resets"] = s["lengths"] = None
    if case["packed"]:   # episodes of 512 tokens on average
        s["resets"] = (torch.rand(N, T, generator=g, device=DEV) < 1 / 512).to(torch.uint8)
    if case["ragged"]:   # rows of T/4 to T tokens, one of them full
        low = max(1, T // 4)
        lengths = (low + torch.rand(N, generator=g, device=DEV) * (T - low + 1)).to(torch.int32).clamp_(max=T)
        lengths[N // 2] = T
        s["lengths"] = lengths
    s["initial_state"] = normal(N, D, scale=0.5, to=torch.float32)
    if op == "scan_train":
        s["grad_y"] = normal(N, T, D)
    return s


# ---------------------------------------------------------------------------
# plain forms: elementary torch operations in 32 bits, rounded once at the end

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


def _coefficients(s):
    """x, both gates after their sigmoid, the decay and the root in front of the input, in 32 bits"""
    x, r, i = s["x"].float(), torch.sigmoid(s["gate"].float()), torch.sigmoid(s["input_gate"].float())
    log_a = s["log_decay"] * r
    return x, r, i, torch.exp(log_a), torch.sqrt(-torch.expm1(2 * log_a))


def _plain_scan(s, train):
    x, r, i, a, root = _coefficients(s)
    T, out = x.shape[1], s["x"].dtype
    live = None
    if s["lengths"] is not None:
        live = (torch.arange(T, device=DEV)[None, :] < s["lengths"][:, None])[..., None]
    keep = a
    if s["resets"] is not None:
        keep = a * (s["resets"] == 0)[..., None]
    b = root * i * x
    if live is not None:
        keep, b = torch.where(live, keep, 1.0), b * live
    b[:, 0] += keep[:, 0] * s["initial_state"]
    h = _recurrence(keep, b)
    y = h if live is None else h * live
    if not train:
        return y.to(out), h[:, -1].clone()
    gy = s["grad_y"].float()
    if live is not None:
        gy = gy * live
    # the gradient of the states runs the same recurrence backwards
    back = torch.cat([keep[:, 1:], torch.zeros_like(keep[:, :1])], 1).flip(1)
    gh = _recurrence(back, gy.flip(1)).flip(1)
    before = torch.cat([s["initial_state"][:, None], h[:, :-1]], 1)
    gb = gh if live is None else gh * live
    gx, gi = gb * root * i, gb * root * x * i * (1 - i)
    # log a moves the decay by a and the root by -a^2 / root
    glog = gh * keep * before - gb * i * x * a * a / root
    if live is not None:
        glog = glog * live
    gr = glog * s["log_decay"] * r * (1 - r)
    return (y.to(out), h[:, -1].clone(), gx.to(out), gr.to(out), gi.to(out), (glog * r).sum((0, 1)),
            gh[:, 0] * keep[:, 0])


def _plain_scan_step(s):
    x, _, i, a, root = _coefficients(s)
    at = s["slots"].long()
    h = a * s["state"][at] + root * i * x
    s["state"][at] = h
    return h.to(s["x"].dtype), s["state"]


def _activation(z, kind):
    """act(z) and its derivative"""
    if kind == "silu":
        g = torch.sigmoid(z)
        return z * g, g * (1 + z * (1 - g))
    half = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
    return z * half, half + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _plain_projection(s, train):
    x, wg, wu = s["x"].float(), s["gate_weight"].float(), s["up_weight"].float()
    out = s["x"].dtype
    u = x @ wu.t()
    a, slope = _activation(x @ wg.t(), s["act"])
    h = (a * u).to(out)
    if not train:
        return h
    gh = s["grad_h"].float()
    gu, gz = gh * a, gh * u * slope
    return h, (gz @ wg + gu @ wu).to(out), (gz.t() @ x).to(out), (gu.t() @ x).to(out)


def _plain_distill(s, train):
    z = s["logits"].float() / s["tau"]
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    t = s["teacher_logits"] / s["tau"]
    t = t - t.amax(-1, keepdim=True)
    t = t - torch.log(torch.exp(t).sum(-1, keepdim=True))   # the teacher's log probabilities over its K tokens
    q = torch.exp(t)
    loss = (q * (t - (torch.gather(z, 2, s["teacher_tokens"]) - top - torch.log(total)))).sum(-1)
    if s["mask"] is not None:
        loss = loss * s["mask"]
    if not train:
        return loss
    weight = s["grad_loss"] if s["mask"] is None else s["grad_loss"] * s["mask"]
    weight = (weight / s["tau"])[..., None]
    g = (e / total * weight).scatter_add_(2, s["teacher_tokens"], -q * weight)
    return loss, g.to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# the framework's calls

def _own(s):
    import linear_recurrence_scan_gb300 as rl
    op = s["op"]
    if op == "scan":
        return rl.gated_scan(s["x"], s["gate"], s["input_gate"], s["log_decay"], initial_state=s["initial_state"],
                             resets=s["resets"], lengths=s["lengths"])
    if op == "scan_train":
        y, final, kept = rl.gated_scan(s["x"], s["gate"], s["input_gate"], s["log_decay"],
                                       initial_state=s["initial_state"], resets=s["resets"], lengths=s["lengths"],
                                       return_checkpoints=True)
        g = rl.gated_scan_backward(s["grad_y"], s["x"], s["gate"], s["input_gate"], s["log_decay"], kept,
                                   resets=s["resets"], lengths=s["lengths"])
        return y, final, g.x, g.gate, g.input_gate, g.log_decay, g.initial_state
    if op == "scan_step":
        return rl.gated_scan_step(s["state"], s["x"], s["gate"], s["input_gate"], s["log_decay"],
                                  slots=s["slots"]), s["state"]
    if op == "projection":
        return rl.gated_projection(s["x"], s["gate_weight"], s["up_weight"], s["act"])
    if op == "projection_train":
        h = rl.gated_projection(s["x"], s["gate_weight"], s["up_weight"], s["act"])
        g = rl.gated_projection_backward(s["grad_h"], s["x"], s["gate_weight"], s["up_weight"], s["act"])
        return h, g.x, g.gate_weight, g.up_weight
    if op == "distill":
        return rl.distill_loss(s["logits"], s["teacher_logits"], s["teacher_tokens"], s["tau"], s["mask"])
    return rl.distill_loss_and_grad(s["grad_loss"], s["logits"], s["teacher_logits"], s["teacher_tokens"], s["tau"],
                                    s["mask"])


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "scan_step":
        return _plain_scan_step(state)
    kind, train = op.split("_")[0], op.endswith("_train")
    return {"scan": _plain_scan, "projection": _plain_projection, "distill": _plain_distill}[kind](state, train)


# ---------------------------------------------------------------------------
# bytes and operations

def work(case):
    op = case["op"]
    e = 2 if case.get("dtype", "bfloat16") == "bfloat16" else 4
    if op.startswith("projection"):
        M, D, F = case["M"], case["D"], case["F"]
        if op == "projection":
            return {"bytes": 2 * (M * D + 2 * F * D + M * F), "flops": 4 * M * D * F}
        # the gradients' products start from both projections, which a pass makes once; four more follow
        return {"bytes": 2 * (2 * M * D + 4 * F * D + 2 * M * F), "flops": 12 * M * D * F}
    if op.startswith("distill"):
        N, T, V, K = (case[k] for k in "NTVK")
        read = N * (T - T // 4 if case["masked"] else T)
        small = read * K * 12 + N * T * (4 + (1 if case["masked"] else 0))
        if op == "distill":
            return {"bytes": read * V * e + small, "flops": read * (3 * V + 10 * K)}
        return {"bytes": read * V * e + N * T * V * e + small + 4 * N * T, "flops": read * (6 * V + 12 * K)}
    N, D = case["N"], case["D"]
    if op == "scan_step":   # the state is read and written
        return {"bytes": N * D * (8 + 4 * e) + 4 * D + 4 * N, "flops": 25 * N * D}
    n = N * case["T"] * D
    if op == "scan":   # x and both gates read, y written
        return {"bytes": 4 * n * e + 8 * N * D + 4 * D, "flops": 25 * n}
    # a pass reads x, both gates and grad_y and writes y and three gradients
    return {"bytes": 8 * n * e + 12 * N * D + 8 * D, "flops": 65 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one token after the other

def _sigmoid64(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _exact_scan(s, train):
    f = {k: s[k].double() for k in ("x", "gate", "input_gate", "log_decay", "initial_state")}
    N, T, D = f["x"].shape
    r, i = _sigmoid64(f["gate"]), _sigmoid64(f["input_gate"])
    log_a = f["log_decay"] * r
    a, square = torch.exp(log_a), -torch.expm1(2 * log_a)
    root = square ** 0.5
    length = torch.full((N,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    reset = torch.zeros(N, T, dtype=torch.bool, device=DEV) if s["resets"] is None else s["resets"] != 0
    h, y, kept = f["initial_state"], torch.zeros_like(f["x"]), []
    for t in range(T):
        if train:
            kept.append(h)
        new = a[:, t] * torch.where(reset[:, t, None], 0.0, h) + root[:, t] * i[:, t] * f["x"][:, t]
        on = (t < length)[:, None]
        h = torch.where(on, new, h)
        y[:, t] = torch.where(on, new, 0.0)
    if not train:
        return y, h
    gy = s["grad_y"].double()
    gx, gr, gi = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(y)
    gd, gh = torch.zeros_like(f["log_decay"]), torch.zeros_like(h)
    for t in range(T - 1, -1, -1):
        on = (t < length)[:, None]
        total = gh + gy[:, t]
        prior = torch.where(reset[:, t, None], 0.0, kept[t])
        x_t, r_t, i_t = f["x"][:, t], r[:, t], i[:, t]
        gx[:, t] = torch.where(on, total * root[:, t] * i_t, 0.0)
        gi[:, t] = torch.where(on, total * root[:, t] * x_t * i_t * (1 - i_t), 0.0)
        through = total * (prior * a[:, t] - i_t * x_t * (1 - square[:, t]) / root[:, t])
        gr[:, t] = torch.where(on, through * f["log_decay"] * r_t * (1 - r_t), 0.0)
        gd += torch.where(on, through * r_t, 0.0).sum(0)
        gh = torch.where(on, torch.where(reset[:, t, None], 0.0, total * a[:, t]), gh)
    return y, h, gx, gr, gi, gd, gh


def _exact_scan_step(s):
    state, at = s["state"].double(), s["slots"].long()
    log_a = s["log_decay"].double() * _sigmoid64(s["gate"].double())
    gain = torch.sqrt(1 - torch.exp(2 * log_a)) * _sigmoid64(s["input_gate"].double())
    state[at] = torch.exp(log_a) * state[at] + gain * s["x"].double()
    return state[at], state


def _exact_projection(s, train):
    x, wg, wu = s["x"].double(), s["gate_weight"].double(), s["up_weight"].double()
    z, u = torch.einsum("md,fd->mf", x, wg), torch.einsum("md,fd->mf", x, wu)
    if s["act"] == "silu":
        gate = _sigmoid64(z)
        slope = gate + z * gate * (1 - gate)
    else:
        gate = torch.special.ndtr(z)
        slope = gate + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    h = z * gate * u
    if not train:
        return h
    gh = s["grad_h"].double()
    gz, gu = gh * u * slope, gh * z * gate
    return (h, torch.einsum("mf,fd->md", gz, wg) + torch.einsum("mf,fd->md", gu, wu),
            torch.einsum("mf,md->fd", gz, x), torch.einsum("mf,md->fd", gu, x))


def _exact_distill(s, train):
    N, T, V = s["logits"].shape
    loss = torch.zeros(N, T, dtype=torch.float64, device=DEV)
    grad = torch.zeros(N, T, V, dtype=torch.float64, device=DEV) if train else None
    for n in range(N):   # a row at a time: the logits in 64 bits are large
        z = s["logits"][n].double() / s["tau"]
        logp = z - torch.logsumexp(z, -1, keepdim=True)
        t = s["teacher_logits"][n].double() / s["tau"]
        logq = t - torch.logsumexp(t, -1, keepdim=True)
        on = torch.ones(T, dtype=torch.float64, device=DEV) if s["mask"] is None else s["mask"][n].double()
        q = torch.exp(logq)
        for k in range(q.shape[-1]):
            at = s["teacher_tokens"][n, :, k:k + 1]
            loss[n] += q[:, k] * (logq[:, k] - torch.gather(logp, 1, at)[:, 0]) * on
        if train:
            grad[n] = torch.exp(logp).scatter_add(1, s["teacher_tokens"][n], -q)
            grad[n] *= (s["grad_loss"][n].double() * on / s["tau"])[:, None]
    return (loss, grad) if train else loss


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "scan_step":
        return _exact_scan_step(s)
    kind, train = op.split("_")[0], op.endswith("_train")
    return {"scan": _exact_scan, "projection": _exact_projection, "distill": _exact_distill}[kind](s, train)
