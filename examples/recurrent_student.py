"""A small recurrent token policy that learns from a teacher: each layer is a
gated recurrence and a gated feed-forward block, and the loss is the divergence
from the teacher's top logits on responses that the student writes itself.

    python examples/recurrent_student.py

The teacher is the state-space policy of state_space_policy.py.  Prompts of
different lengths go through the prompt forms (``lengths``), the responses
through the single-token form on a pool of state slots, and training through
the differentiable forms, with ``mask`` on the response's tokens.
"""
import os
import sys

import torch
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import linear_recurrence_scan_gb300 as rl  # noqa: E402
from state_space_policy import Policy  # noqa: E402


class GatedLayer(nn.Module):
    """norm -> projections -> gated recurrence -> projection; norm -> feed-forward block.  Activations and products
    are bfloat16, parameters float32."""

    def __init__(self, width, channels, features):
        super().__init__()
        self.channels = channels
        self.norm, self.norm2 = nn.Parameter(torch.ones(width)), nn.Parameter(torch.ones(width))
        self.into = nn.Parameter(torch.randn(3 * channels, width) * width ** -0.5)
        # decays between 0.9 and 0.999 where the gate is open: log_decay = -8 softplus(rate)
        start = -torch.log(0.9 + 0.099 * torch.rand(channels)) / 8
        self.rate = nn.Parameter(start + torch.log(-torch.expm1(-start)))
        self.out = nn.Parameter(torch.randn(width, channels) * channels ** -0.5)
        self.up = nn.Parameter(torch.randn(2 * features, width) * width ** -0.5)   # both projections
        self.down = nn.Parameter(torch.randn(width, features) * features ** -0.5)

    def log_decay(self):
        return -8 * nn.functional.softplus(self.rate)

    def _inputs(self, x, residual):
        n = rl.add_rms_norm(x, self.norm, residual)
        return (n.y @ self.into.t().to(x.dtype)).split(self.channels, -1), n.residual

    def _rest(self, y, residual):
        n = rl.add_rms_norm(y @ self.out.t().to(y.dtype), self.norm2, residual)
        gate, up = self.up.to(y.dtype).chunk(2)
        return rl.gated_projection(n.y, gate, up) @ self.down.t().to(y.dtype), n.residual

    def forward(self, x, residual, lengths=None):
        """x, residual [N,T,width] -> (output, the new residual, state)"""
        (u, gate, input_gate), residual = self._inputs(x, residual)
        y, state = rl.gated_scan(u, gate, input_gate, self.log_decay(), lengths=lengths)
        return (*self._rest(y, residual), state)

    def step(self, x, residual, state, slots):
        """One token of each sequence: x, residual [N,width]; the state's slots are updated in place."""
        (u, gate, input_gate), residual = self._inputs(x, residual)
        return self._rest(rl.gated_scan_step(state, u, gate, input_gate, self.log_decay(), slots=slots), residual)


class Student(nn.Module):
    def __init__(self, vocabulary=64, width=128, channels=256, features=384, layers=2):
        super().__init__()
        self.embed = nn.Embedding(vocabulary, width)
        self.layers = nn.ModuleList(GatedLayer(width, channels, features) for _ in range(layers))
        self.norm = nn.Parameter(torch.ones(width))
        self.head = nn.Parameter(torch.randn(vocabulary, width) * width ** -0.5)

    def _logits(self, x, residual):
        return rl.add_rms_norm(x, self.norm, residual).y @ self.head.t().to(x.dtype)

    def forward(self, tokens, lengths=None):
        """(logits [N,T,V], each layer's final state)"""
        residual = self.embed(tokens).bfloat16()
        x, states = torch.zeros_like(residual), []
        for layer in self.layers:
            x, residual, state = layer(x, residual, lengths)
            states.append(state)
        return self._logits(x, residual), states

    def step(self, tokens, states, slots=None):
        """logits [N,V] of one token of each sequence"""
        residual = self.embed(tokens).bfloat16()
        x = torch.zeros_like(residual)
        for layer, state in zip(self.layers, states):
            x, residual = layer.step(x, residual, state, slots)
        return self._logits(x, residual)


@torch.no_grad()
def respond(model, prompts, lengths, count, generator):
    """`count` sampled tokens for each prompt (padded rows of `lengths` tokens)."""
    logits, states = model(prompts, lengths)
    N = prompts.shape[0]
    last = logits[torch.arange(N, device=prompts.device), (lengths - 1).long()]
    slots = torch.arange(N - 1, -1, -1, dtype=torch.int32, device=prompts.device)   # another order than the batch's
    states = [s.flip(0).contiguous() for s in states]
    tokens = []
    for _ in range(count):
        u = torch.rand(last.shape, generator=generator, device=last.device)
        tokens.append((last.float() - torch.log(-torch.log(u))).argmax(-1))   # a sample, by Gumbel's maximum
        last = model.step(tokens[-1], states, slots)
    return torch.stack(tokens, 1)


def batch(prompts, lengths, responses):
    """Rows of prompt and response, their lengths, and the mask of the positions whose next token is a response's."""
    N, R = responses.shape
    T = prompts.shape[1] + R
    tokens = torch.zeros(N, T, dtype=torch.long, device=prompts.device)
    tokens[:, :prompts.shape[1]] = prompts
    at = lengths.long()[:, None] + torch.arange(R, device=prompts.device)
    tokens.scatter_(1, at, responses)
    places = torch.arange(T, device=prompts.device)
    full = lengths + R
    mask = (places >= lengths[:, None] - 1) & (places < full[:, None] - 1)
    return tokens, full.to(torch.int32), mask


def train_step(student, teacher, optimiser, prompts, lengths, responses, top=8, temperature=1.0):
    """One step down the divergence from the teacher on the student's own tokens; (loss, a token's mean divergence)."""
    tokens, full, mask = batch(prompts, lengths, responses)
    with torch.no_grad():
        best = teacher(tokens, lengths=full)[0].float().topk(top, -1)
    logits, _ = student(tokens, full)
    divergence = rl.distill_loss(logits, best.values, best.indices, temperature, mask)
    loss = divergence.sum() / mask.sum()
    optimiser.zero_grad()
    loss.backward()
    optimiser.step()
    return loss.item()


def run(steps=60, device="cuda", seed=0):
    """Teaches a fresh student; the mean divergence, step by step."""
    torch.manual_seed(seed)
    generator = torch.Generator(device=device)
    generator.manual_seed(seed)
    teacher, student = Policy().to(device), Student().to(device)
    for p in teacher.parameters():
        p.requires_grad_(False)
    optimiser = torch.optim.Adam(student.parameters(), lr=2e-3)
    history = []
    for _ in range(steps):
        prompts = torch.randint(0, 64, (16, 24), generator=generator, device=device)
        lengths = torch.randint(4, 25, (16,), generator=generator, device=device, dtype=torch.int32)
        responses = respond(student, prompts, lengths, 16, generator)
        history.append(train_step(student, teacher, optimiser, prompts, lengths, responses))
    return history


if __name__ == "__main__":
    losses = run()
    for i in range(0, len(losses), 10):
        print(f"step {i:3d}: divergence from the teacher {losses[i]:.4f}")
