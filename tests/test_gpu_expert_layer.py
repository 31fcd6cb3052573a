"""The operators together: the example's layer of experts on pooled embeddings."""
import importlib.util
import os

import pytest
import torch

import table_embedding_bag_gb300 as tbe

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def widened(weights):
    q, scale = weights
    s = scale.repeat_interleave(128, 1)[:, :q.shape[1]].repeat_interleave(128, 2)[:, :, :q.shape[2]]
    return q.double() * s.double()


def test_layer_and_its_gradients(example):
    """Against the same layer in 64 bits with autograd.  The experts' inputs (and
    in the backward pass the gradients of their outputs) are rounded to 8 bits
    twice: 2^-4 of a value at most each time, so the results may be 2^-3 off in
    the 2-norm, and are a good deal nearer."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    layer = example.ExpertLayer(width=144, hidden=272, experts=6, k=2, generator=g)
    x = torch.randn(300, 144, generator=g, device="cuda")
    grad_out = torch.randn(300, 144, generator=g, device="cuda")
    out = layer.forward(x)
    grad_x, grad_router = layer.backward(x, grad_out)

    xd, router = x.double().requires_grad_(), layer.router.double().requires_grad_()
    w = torch.softmax((xd @ router.T).gather(1, layer.ids), 1)
    up, down = widened(layer.up), widened(layer.down)
    ref = 0
    for j in range(2):
        h = torch.relu(torch.einsum("nw,nhw->nh", xd, up[layer.ids[:, j]]))
        ref = ref + w[:, j:j + 1] * torch.einsum("nh,nwh->nw", h, down[layer.ids[:, j]])
    ref.backward(grad_out.double())
    for got, want in ((out, ref.detach()), (grad_x, xd.grad), (grad_router, router.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -3


def test_training_lowers_the_loss(example):
    losses, norms = example.train(steps=12, bags=512, rows=400)
    assert all(n > 0 for n in norms)
    assert losses[-1] < 0.9 * losses[0]
    assert torch.isfinite(torch.tensor(losses)).all()


def test_single_tokens(example):
    """One token at a time gives what the batch gives, row by row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    layer = example.ExpertLayer(width=256, hidden=512, experts=8, k=2, generator=g)
    x = torch.randn(5, 256, generator=g, device="cuda")
    whole = layer.forward(x).clone()
    ids = layer.ids.clone()
    for i in range(5):
        one = layer.forward(x[i:i + 1])
        assert torch.equal(layer.ids[0], ids[i])
        # the sums over blocks may be split differently, and one of the 512 hidden values may then
        # be rounded the other way: 2^-3 of it at most, well below 2^-6 of the largest result
        assert float((one[0] - whole[i]).abs().max()) <= 2.0 ** -6 * float(whole[i].abs().max())
    assert tbe.tbe_kernel_launches() > 0
