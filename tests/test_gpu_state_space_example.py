"""The example policy: its single-token forms give the prompt forms' logits,
packed rows give the separate rows' logits, and it learns."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module")
def example():
    from linear_recurrence_scan_gb300 import build
    build.build()
    import state_space_policy
    return state_space_policy


def test_tokens_one_at_a_time_are_the_prompt(example):
    torch.manual_seed(1)
    model = example.Policy().cuda()
    tokens = torch.randint(0, 64, (3, 20), device="cuda")
    lengths = torch.tensor([9, 4, 12], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        whole, values, _ = model(tokens)
        _, _, caches = model(tokens, lengths=lengths)
        for k in range(8):
            at = (lengths + k).long()
            logits, value = model.step(tokens[torch.arange(3), at], caches)
            # two float32 evaluations of the same sums, of order 1: 2^-24 times a few hundred roundings
            assert torch.allclose(logits, whole[torch.arange(3), at], atol=1e-3, rtol=1e-3)
            assert torch.allclose(value, values[torch.arange(3), at], atol=1e-3, rtol=1e-3)


def test_packed_episodes_are_separate_rows(example):
    torch.manual_seed(2)
    model = example.Policy().cuda()
    a, b = torch.randint(0, 64, (1, 11), device="cuda"), torch.randint(0, 64, (1, 17), device="cuda")
    resets = torch.zeros(1, 28, dtype=torch.uint8, device="cuda")
    resets[0, 0] = resets[0, 11] = 1
    with torch.no_grad():
        packed, _, _ = model(torch.cat([a, b], 1), resets)
        first, second = model(a)[0], model(b)[0]
    assert torch.allclose(packed[:, :11], first, atol=1e-3, rtol=1e-3)
    assert torch.allclose(packed[:, 11:], second, atol=1e-3, rtol=1e-3)


def test_the_policy_learns(example):
    shares = example.run(steps=40)
    assert sum(shares[-5:]) / 5 > 4 * max(sum(shares[:5]) / 5, 1 / 64)
