"""The example model of examples/layer_stack.py on a GPU: its whole gradient
against differences of its loss, training lowers the loss, and tokens generated
one by one from ragged prompts get the logits of a full pass."""
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
    m = layer_stack.Stack(width=32)
    tokens = torch.randint(0, 64, (3, 50), device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(3))

    def loss():
        return torch.nn.functional.cross_entropy(m.train_logits(tokens[:, :-1]).flatten(0, 1),
                                                 tokens[:, 1:].flatten())
    loss().backward()
    ps = m.parameters()
    for chosen in (ps, [v for l in m.layers for v in l.p.values()]):
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


def test_training_lowers_the_loss(cuda_lib):
    import layer_stack
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        losses = layer_stack.train(layer_stack.Stack(dtype=dtype), 30)
        assert losses[-1] < 0.75 * losses[0]


def test_generation_matches_a_full_pass(cuda_lib):
    """fp32 throughout; the projections' sums are in another order for one token
    than for many, a few 1e-6 of the logits each, through two layers."""
    import layer_stack
    import torch
    with torch.no_grad():
        d, top = layer_stack.generate(layer_stack.Stack())
    assert d <= 1e-4 * top
