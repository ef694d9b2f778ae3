"""The example model of examples/layer_stack.py with its third layer (unit, turned queries
and keys and the gated delta rule) on a GPU: its whole gradient against differences of its
loss, and tokens generated one by one from ragged prompts get the logits of a full pass."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_gradient_is_the_difference_of_the_loss(cuda_lib):
    """Along the gradient direction, in fp32.  The loss (~4) is good to ~1e-6; over
    a step that changes it by ~1e-2 each way that is 1e-4 of the difference, the
    curvature's share is of the same order, and 2 % leaves a factor of 50."""
    import torch
    import layer_stack
    m = layer_stack.Stack(width=32, delta=True)
    tokens = torch.randint(0, 64, (3, 90), device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(3))

    def loss():
        return torch.nn.functional.cross_entropy(m.train_logits(tokens[:, :-1]).flatten(0, 1),
                                                 tokens[:, 1:].flatten())
    loss().backward()
    for chosen in (m.parameters(), list(m.layers[2].p.values())):
        norm2 = sum(float((p.grad.double() ** 2).sum()) for p in chosen)
        e = 1e-2 / norm2
        with torch.no_grad():
            for p in chosen:
                p += e * p.grad
            up = float(loss())
            for p in chosen:
                p -= 2 * e * p.grad
            dn = float(loss())
            for p in chosen:
                p += e * p.grad
        assert abs((up - dn) / (2 * e) - norm2) <= 2e-2 * norm2


def test_bf16_model_runs(cuda_lib):
    import layer_stack
    import torch
    losses = layer_stack.train(layer_stack.Stack(dtype=torch.bfloat16, delta=True), 3)
    assert all(0.0 < v < 20.0 for v in losses)


def test_generation_matches_a_full_pass(cuda_lib):
    """fp32 throughout; the projections' sums are in another order for one token
    than for many, a few 1e-6 of the logits each, through three layers."""
    import layer_stack
    import torch
    with torch.no_grad():
        d, top = layer_stack.generate(layer_stack.Stack(delta=True), lengths=(70, 0, 7, 64))
    assert d <= 1e-4 * top
