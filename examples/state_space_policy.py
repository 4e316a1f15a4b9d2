"""A small token policy with state-space layers: it writes responses to
prompts one token at a time and learns from them with this library's GAE.

    python examples/state_space_policy.py

Each layer is norm -> projection -> causal convolution -> projections ->
selective scan -> projection, with the residual kept by the norm.  Prompts of
different lengths go through the prompt forms (``lengths``), the response
through the single-token forms on a pool of state slots, and training through
the differentiable forms on rows that pack two episodes (``resets``), with
``compute_gae``'s mask on the response's tokens.
"""
import os
import sys

import torch
import torch.nn.functional as F
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_recurrence_scan_gb300 as rl  # noqa: E402


class StateSpaceLayer(nn.Module):
    def __init__(self, width, channels, states=16, taps=4):
        super().__init__()
        self.channels, self.states, self.taps, self.rank = channels, states, taps, max(8, width // 16)
        self.norm = nn.Parameter(torch.ones(width))
        self.into = nn.Linear(width, 2 * channels, bias=False)
        self.conv = nn.Parameter(torch.randn(channels, taps) / taps ** 0.5)
        self.conv_bias = nn.Parameter(torch.zeros(channels))
        self.mix = nn.Linear(channels, self.rank + 2 * states, bias=False)
        self.to_delta = nn.Linear(self.rank, channels, bias=False)
        dt = torch.exp(torch.rand(channels) * 4.6 - 6.9)   # time steps between 1e-3 and 1e-1
        self.delta_bias = nn.Parameter(dt + torch.log(-torch.expm1(-dt)))
        self.log_rates = nn.Parameter(torch.log(torch.arange(1.0, states + 1)).repeat(channels, 1))
        self.skip = nn.Parameter(torch.ones(channels))
        self.out = nn.Linear(channels, width, bias=False)

    def _scan_inputs(self, x):
        low, B, C = self.mix(x).split([self.rank, self.states, self.states], -1)
        return self.to_delta(low), -torch.exp(self.log_rates), B, C

    def forward(self, x, residual, resets=None, lengths=None):
        """x, residual [N,T,width] -> (output, the new residual, (window, state))"""
        n = rl.add_rms_norm(x, self.norm, residual)
        x, z = self.into(n.y).split(self.channels, -1)
        x, window = rl.causal_conv(x, self.conv, self.conv_bias, resets=resets, lengths=lengths)
        delta, A, B, C = self._scan_inputs(x)
        y, state = rl.selective_scan(x, delta, A, B, C, self.skip, z, self.delta_bias, resets=resets, lengths=lengths)
        return self.out(y), n.residual, (window, state)

    def step(self, x, residual, cache, slots):
        """One token of each sequence: x, residual [N,width]; the cache's slots are updated in place."""
        window, state = cache
        n = rl.add_rms_norm(x, self.norm, residual)
        x, z = self.into(n.y).split(self.channels, -1)
        x = rl.causal_conv_step(window, x, self.conv, self.conv_bias, slots=slots)
        delta, A, B, C = self._scan_inputs(x)
        y = rl.selective_scan_step(state, x, delta, A, B, C, self.skip, z, self.delta_bias, slots=slots)
        return self.out(y), n.residual


class Policy(nn.Module):
    def __init__(self, vocabulary=64, width=128, channels=256, layers=2):
        super().__init__()
        self.embed = nn.Embedding(vocabulary, width)
        self.layers = nn.ModuleList(StateSpaceLayer(width, channels) for _ in range(layers))
        self.norm = nn.Parameter(torch.ones(width))
        self.policy, self.value = nn.Linear(width, vocabulary), nn.Linear(width, 1)

    def _heads(self, x, residual):
        y = rl.add_rms_norm(x, self.norm, residual).y
        return self.policy(y), self.value(y)[..., 0]

    def forward(self, tokens, resets=None, lengths=None):
        """(logits [N,T,V], values [N,T], each layer's final (window, state))"""
        residual = self.embed(tokens)
        x, caches = torch.zeros_like(residual), []
        for layer in self.layers:
            x, residual, cache = layer(x, residual, resets, lengths)
            caches.append(cache)
        return (*self._heads(x, residual), caches)

    def step(self, tokens, caches, slots=None):
        """(logits [N,V], values [N]) of one token of each sequence"""
        residual = self.embed(tokens)
        x = torch.zeros_like(residual)
        for layer, cache in zip(self.layers, caches):
            x, residual = layer.step(x, residual, cache, slots)
        return self._heads(x, residual)


@torch.no_grad()
def respond(model, prompts, lengths, count, generator):
    """`count` sampled tokens for each prompt (padded rows of `lengths` tokens)."""
    logits, _, caches = model(prompts, lengths=lengths)
    N = prompts.shape[0]
    last = logits[torch.arange(N, device=prompts.device), (lengths - 1).long()]
    # the sequences take the pool's slots in another order than the batch's
    slots = torch.arange(N - 1, -1, -1, dtype=torch.int32, device=prompts.device)
    caches = [tuple(t.flip(0).contiguous() for t in c) for c in caches]
    tokens = []
    for _ in range(count):
        u = torch.rand(last.shape, generator=generator, device=last.device)
        tokens.append((last.float() - torch.log(-torch.log(u))).argmax(-1))   # a sample, by Gumbel's maximum
        last, _ = model.step(tokens[-1], caches, slots)
    return torch.stack(tokens, 1)


def train_step(model, optimiser, prompts, lengths, responses, target):
    """One policy-gradient step; a response token earns 1 where it is the target token."""
    N, R = responses.shape
    device = prompts.device
    rows = [torch.cat([prompts[n, :int(lengths[n])], responses[n]]) for n in range(N)]
    T = max(len(a) + len(b) for a, b in zip(rows[::2], rows[1::2]))
    tokens = torch.zeros(N // 2, T, dtype=torch.long, device=device)
    resets = torch.zeros(N // 2, T, dtype=torch.uint8, device=device)
    mask = torch.zeros(N // 2, T, device=device)     # steps whose action is a response token
    done = torch.zeros(N // 2, T, device=device)
    full = torch.zeros(N // 2, dtype=torch.int32, device=device)
    for i, pair in enumerate(zip(rows[::2], rows[1::2])):   # two episodes a row
        at = 0
        for row in pair:
            tokens[i, at:at + len(row)] = row
            resets[i, at] = 1
            mask[i, at + len(row) - R - 1:at + len(row) - 1] = 1
            done[i, at + len(row) - 2:at + len(row)] = 1
            at += len(row)
        full[i] = at
    logits, values, _ = model(tokens, resets, full)
    actions = torch.cat([tokens[:, 1:], tokens[:, :1]], 1)
    rewards = (actions == target).float() * mask
    advantages, = rl.compute_gae_and_returns(rewards, values.detach().float(), done, None, 0.9, 0.9,
                                             outputs=("advantages",))
    logp = torch.gather(F.log_softmax(logits.float(), -1), 2, actions[..., None])[..., 0]
    entropy = -(logits.float().softmax(-1) * F.log_softmax(logits.float(), -1)).sum(-1)
    returns = advantages + values.detach()
    loss = ((-(advantages * logp) + 0.5 * (values - returns).square() - 0.003 * entropy) * mask).sum() / mask.sum()
    optimiser.zero_grad()
    loss.backward()
    optimiser.step()
    return loss.item(), float(rewards.sum() / mask.sum())


def run(steps=60, device="cuda", seed=0):
    """Trains from scratch; the share of target tokens in the responses, step by step."""
    torch.manual_seed(seed)
    generator = torch.Generator(device=device)
    generator.manual_seed(seed)
    model = Policy().to(device)
    optimiser = torch.optim.Adam(model.parameters(), lr=3e-3)
    shares = []
    for _ in range(steps):
        prompts = torch.randint(0, 64, (16, 24), generator=generator, device=device)
        lengths = torch.randint(4, 25, (16,), generator=generator, device=device, dtype=torch.int32)
        responses = respond(model, prompts, lengths, 16, generator)
        shares.append(train_step(model, optimiser, prompts, lengths, responses, target=7)[1])
    return shares


if __name__ == "__main__":
    history = run()
    for i in range(0, len(history), 10):
        print(f"step {i:3d}: target token in {100 * history[i]:5.1f}% of the response")
