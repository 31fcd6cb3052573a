"""A layer of experts on pooled embeddings, trained for a few steps.

    python examples/expert_layer.py [--steps 20]

Eight embedding tables are pooled into one vector per bag (a token).  A router
sends each token to two of sixteen experts, two 8-bit matrices with a ReLU between
them, and the weighted sum of what they answer is compared with a target.  The
tables and the router learn; the experts' weights are frozen in 8 bits.  One step:

  tables       TableBatchedEmbedding.forward               pooled vectors
  forward      tbe_expert_sort, tbe_expert_dispatch_fp8    rows to their experts, in 8 bits
               tbe_expert_product, tbe_quantize_rows       the experts
               tbe_expert_combine                          back, weighted
  backward     tbe_expert_combine_backward                 of the rows and the weights
               tbe_expert_product                          of the inputs: transposed weights
               tbe_expert_dispatch_backward                back to the tokens
  clipping     tbe_grad_clip                               all gradients to one norm
  tables       TableBatchedEmbedding.backward              one Adagrad step
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import table_embedding_bag_gb300 as tbe  # noqa: E402


class ExpertLayer:
    """out = sum over a token's k experts of weight * down(relu(up(token)))."""

    def __init__(self, width, hidden, experts, k, generator):
        self.experts, self.k = experts, k
        up, down = (torch.randn(experts, n, m, generator=generator, device="cuda") / m ** 0.5
                    for n, m in ((hidden, width), (width, hidden)))
        self.up, self.down = tbe.tbe_quantize_weights(up), tbe.tbe_quantize_weights(down)
        # the gradients of the inputs go through the transposed weights: the same 8-bit values
        self.up_t = tbe.tbe_quantize_weights(up.transpose(1, 2).contiguous())
        self.down_t = tbe.tbe_quantize_weights(down.transpose(1, 2).contiguous())
        self.router = torch.randn(experts, width, generator=generator, device="cuda") / width ** 0.5

    def _product(self, rows, weights, out_dtype):
        q, scale = rows
        return tbe.tbe_expert_product(q, scale, *weights, self.offsets, out_dtype=out_dtype)

    def forward(self, x):
        top, self.ids = (x @ self.router.T).topk(self.k, dim=1)
        self.weights = torch.softmax(top, 1)
        self.offsets, _, self.position = tbe.tbe_expert_sort(self.ids, self.experts)
        rows = tbe.tbe_expert_dispatch_fp8(x, self.offsets, self.position)
        self.hidden = torch.relu_(self._product(rows, self.up, torch.bfloat16))
        self.rows = self._product(tbe.tbe_quantize_rows(self.hidden), self.down, torch.float32)
        return tbe.tbe_expert_combine(self.rows, self.position, self.weights)

    def backward(self, x, grad_out):
        """Gradients of the tokens and of the router."""
        grad_rows, grad_weights = tbe.tbe_expert_combine_backward(
            grad_out, self.rows, self.offsets, self.position, self.weights)
        grad_hidden = self._product(tbe.tbe_quantize_rows(grad_rows), self.down_t, torch.bfloat16)
        grad_hidden.mul_(self.hidden > 0)
        grad_in = self._product(tbe.tbe_quantize_rows(grad_hidden), self.up_t, torch.float32)
        grad_x = tbe.tbe_expert_dispatch_backward(grad_in, self.position)
        # softmax over the chosen experts' scores
        w = self.weights
        grad_top = w * (grad_weights - (w * grad_weights).sum(1, keepdim=True))
        grad_scores = torch.zeros(x.shape[0], self.experts, device=x.device)
        grad_scores.scatter_(1, self.ids, grad_top)
        return grad_x.addmm_(grad_scores, self.router), grad_scores.T @ x


def train(steps=20, bags=2048, tables=8, rows=5000, dim=128, length=8, hidden=512, experts=16, k=2,
          lr=0.05, max_norm=1.0, seed=0, log=None):
    """Losses of the steps and the gradients' norms before clipping."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = tables * bags * length
    emb = tbe.TableBatchedEmbedding([rows] * tables, [dim] * tables, bags, n, lr=lr)
    emb.weights.copy_(torch.randn(emb.weights.shape, generator=g, device="cuda") * 0.3)
    layer = ExpertLayer(tables * dim, hidden, experts, k, g)
    indices = torch.randint(0, rows, (n,), generator=g, device="cuda")
    offsets = torch.arange(0, n + 1, length, device="cuda")
    target = torch.randn(bags, tables * dim, generator=g, device="cuda")
    losses, norms = [], []
    for step in range(steps):
        x = emb.forward(indices, offsets)
        out = layer.forward(x)
        error = out - target
        losses.append(error.square().mean())
        grad_x, grad_router = layer.backward(x, error * (2.0 / error.shape[1]))
        norms.append(tbe.tbe_grad_clip([grad_x, grad_router], max_norm))
        layer.router.sub_(grad_router, alpha=lr)
        emb.backward(grad_x, indices, offsets)
        if log:
            log(f"step {step}: loss {float(losses[-1]):.4f}, gradient norm {float(norms[-1]):.3f}")
    return [float(v) for v in losses], [float(v) for v in norms]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    train(steps=ap.parse_args().steps, log=print)
