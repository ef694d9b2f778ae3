"""The delta layer of examples/layer_stack.py in a serving batch with an empty row, on a GPU."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_an_empty_row_moves_no_position(cuda_lib):
    """Two sequences decoded with an empty row beside them are what they are by themselves, and
    the last slot, which index -1 would name, keeps its cache."""
    import layer_stack
    import torch
    m = layer_stack.Stack(delta=True)
    text = torch.randint(0, 64, (3, 8), device="cuda", generator=torch.Generator("cuda").manual_seed(0))

    def decode(slots):
        c = m.cache(3)
        at = torch.tensor(slots, dtype=torch.int32, device="cuda")
        out = [m.token_logits(text[:len(slots), i], c, at) for i in range(8)]
        return torch.stack(out, 1)[:2], [[t.clone() for t in layer] for layer in c]
    (alone, c1), (beside, c2) = decode([1, 0]), decode([1, 0, -1])
    # (the projections' sums may be in another order for three rows than for two)
    assert float((alone - beside).abs().max()) <= 1e-4 * float(alone.abs().max())
    assert c2[2][2].tolist() == [8, 8, 0] and c1[2][2].tolist() == [8, 8, 0]
    for x, y in zip(c1, c2):
        for p, q in zip(x, y):
            assert float((p.float() - q.float()).abs().max()) <= 1e-4 * max(1.0, float(p.float().abs().max()))
