"""The packed training example: the loss falls, and a backward pass agrees with the same
layer differentiated by torch in 32 bits on the values that the packed tensors stand for."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import packed_training

    return packed_training


def test_the_loss_falls(example):
    losses = example.run(steps=20, tokens=2048, dim=256, vocab=3000, say=lambda *a: None)
    assert losses[-1] < 0.8 * losses[0], losses


def test_gradients_agree_with_torch(example):
    """Each gradient within 6% (2-norm) of the unpacked layer's: four roundings to e4m3
    (2^-4 at most, 2^-5.3 in the mean square) lie between, and the weights are the packed
    ones on both sides."""
    import bit_packing_amd as ibp

    model = example.Model(500, 192, 384, 7)
    ids = torch.randint(500, (1000,), device="cuda")
    y, kept = model.forward(ids)
    dy = (torch.randn_like(y.float()) * 0.01).to(torch.bfloat16)
    grads = model.backward(dy, kept)
    value = lambda layer: ibp.ibp_mx_unpack(layer.w4, dtype=torch.float32).requires_grad_()  # noqa: E731
    wg, wu, wd = value(model.gate), value(model.up), value(model.down)
    table = model.table.float().requires_grad_()
    x = table[ids] * model.scale
    h = torch.nn.functional.silu(x @ wg.t()) * (x @ wu.t())
    (h @ wd.t()).backward(dy.float())
    # the weights' packings along the other axis round apart: those two gradients and the
    # table's pass through them
    for name, want, bound in (("down", wd.grad, 0.06), ("gate", wg.grad, 0.2), ("up", wu.grad, 0.2), ("table", table.grad, 0.25)):
        got = grads[name].float()
        off = ((got - want).norm() / want.norm()).item()
        assert off < bound, (name, off)
