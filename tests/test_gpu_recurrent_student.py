"""The token policy's operators together: examples/recurrent_student.py runs,
its single tokens continue its prompts, and the gradients of a whole layer and
its loss are those of plain float64 torch."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    from linear_recurrence_scan_gb300 import build
    build.build()


def test_runs():
    import recurrent_student
    history = recurrent_student.run(steps=3)
    assert len(history) == 3 and all(torch.isfinite(torch.tensor(v)) for v in history)


def test_single_tokens_continue_a_prompt():
    import recurrent_student as rs
    torch.manual_seed(1)
    model = rs.Student().to(DEV)
    tokens = torch.randint(0, 64, (5, 30), device=DEV)
    with torch.no_grad():
        whole, _ = model(tokens)
        _, states = model(tokens[:, :20])
        steps = torch.stack([model.step(tokens[:, t], states) for t in range(20, 30)], 1)
    # two ways through bfloat16 layers: each of four products and norms a layer, two layers and the head rounds by 2^-8
    torch.testing.assert_close(steps.float(), whole[:, 20:].float(), rtol=0, atol=18 * 2 ** -8 * float(whole.abs().max()))


def plain(layer, head, x, residual, teacher, tokens, mask):
    """The layer and its loss in plain torch, in the parameters' type."""
    sig = torch.sigmoid

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w

    h = x + residual
    u, g, i = (norm(h, layer["norm"]) @ layer["into"].t()).chunk(3, -1)
    a = torch.exp(-8 * torch.nn.functional.softplus(layer["rate"]) * sig(g))
    b = torch.sqrt(1 - a * a) * sig(i) * u
    state, ys = torch.zeros_like(b[:, 0]), []
    for t in range(b.shape[1]):
        state = a[:, t] * state + b[:, t]
        ys.append(state)
    h = h + torch.stack(ys, 1) @ layer["out"].t()
    gate, up = layer["up"].chunk(2)
    n = norm(h, layer["norm2"])
    z = n @ gate.t()
    out = (z * sig(z) * (n @ up.t())) @ layer["down"].t()
    logits = (out + h) @ head.t()
    q = torch.softmax(teacher, -1)
    logp = torch.log_softmax(logits, -1).gather(-1, tokens)
    return ((q * (torch.log(q) - logp)).sum(-1) * mask).sum()


def test_gradients_of_a_layer_and_its_loss():
    """All parameters' gradients through norm, recurrence, feed-forward block and loss.  The layer's values pass about
    a dozen roundings to bfloat16 on their way to the loss and as many back; each is off by at most 2^-8 of itself,
    and as these are independent the gradients' 2-norms stay within 24 * 2^-8 of their own."""
    import linear_recurrence_scan_gb300 as rl
    import recurrent_student as rs
    torch.manual_seed(2)
    layer = rs.GatedLayer(64, 96, 160).to(DEV)
    head = (torch.randn(200, 64, device=DEV) / 8).requires_grad_()
    x, residual = (torch.randn(3, 50, 64, device=DEV).bfloat16() for _ in range(2))
    teacher = torch.randn(3, 50, 7, device=DEV)
    tokens = torch.rand(3, 50, 200, device=DEV).topk(7, -1).indices
    mask = torch.rand(3, 50, device=DEV) < 0.7
    out, res, _ = layer(x, residual)
    logits = (out + res) @ head.t().bfloat16()
    rl.distill_loss(logits, teacher, tokens, 1.0, mask).sum().backward()
    p64 = {k: v.detach().double().requires_grad_() for k, v in layer.named_parameters()}
    h64 = head.detach().double().requires_grad_()
    plain(p64, h64, x.double(), residual.double(), teacher.double(), tokens, mask.double()).backward()
    for k, v in {**dict(layer.named_parameters()), "head": head}.items():
        want = h64.grad if k == "head" else p64[k].grad
        assert float((v.grad.double() - want).norm()) <= 24 * 2 ** -8 * float(want.norm()), k
