"""A block of a language model on token embeddings, trained for a few steps.

    python examples/token_layer.py [--steps 20]

Tokens are looked up in a table, a residual stream runs past the block, and the block
normalises it, routes each token to two of sixteen experts by a sigmoid score with a bias for
balance, and adds what the experts answer.  The table, the norm's weight and the router
learn; the experts' weights are frozen in 8 bits.  One step:

  forward      tbe_embed                                   tokens to vectors
               tbe_rms_norm                                residual added, normalised
               tbe_expert_route, tbe_expert_sort           experts of each token, by score and bias
               tbe_expert_dispatch_fp8, tbe_expert_product rows to their experts, in 8 bits
               tbe_expert_combine                          back, weighted
  backward     tbe_expert_combine_backward                 of the rows and the weights
               tbe_expert_product                          of the inputs: transposed weights
               tbe_expert_dispatch_backward                back to the tokens
               tbe_expert_route_backward                   of the router's logits
               tbe_rms_norm_backward                       of the stream and the norm's weight
               tbe_embed_backward                          of the table
  clipping     tbe_grad_clip                               all gradients to one norm
  balance      the bias of an expert with many tokens falls, that of one with few rises
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import table_embedding_bag_gb300 as tbe  # noqa: E402


class TokenLayer:
    """out = h + sum over a token's k experts of weight * expert(norm(h)), where
    h = scale * table[token] + position."""

    def __init__(self, rows, width, experts, k, generator, dtype=torch.bfloat16):
        rand = lambda *s: torch.randn(*s, generator=generator, device="cuda")
        self.rows, self.k, self.scale = rows, k, width ** 0.5
        self.table = (rand(rows, width) / width ** 0.5).to(dtype)
        self.weight = torch.ones(width, device="cuda")
        self.router = rand(experts, width) / width ** 0.5
        self.bias = torch.zeros(experts, device="cuda")
        w = rand(experts, width, width) / width ** 0.5
        # the gradients of the inputs go through the transposed weights: the same 8-bit values
        self.experts = tbe.tbe_quantize_weights(w)
        self.experts_t = tbe.tbe_quantize_weights(w.mT.contiguous())

    def forward(self, ids, position):
        self.ids = ids
        x = tbe.tbe_embed(self.table, ids, self.scale)
        self.y, self.h = tbe.tbe_rms_norm(x, self.weight, residual=position)
        self.logits = self.y.float() @ self.router.T
        self.chosen, self.weights = tbe.tbe_expert_route(
            self.logits, self.k, bias=self.bias, score="sigmoid")
        self.offsets, _, self.position = tbe.tbe_expert_sort(self.chosen, self.router.shape[0])
        rows = tbe.tbe_expert_dispatch_fp8(self.y, self.offsets, self.position)
        self.answers = tbe.tbe_expert_product(*rows, *self.experts, self.offsets,
                                              out_dtype=torch.float32)
        return self.h.float() + tbe.tbe_expert_combine(self.answers, self.position, self.weights)

    def backward(self, grad_out):
        """Gradients of the table (its type), the norm's weight and the router (fp32)."""
        dtype = self.h.dtype
        grad_rows, grad_weights = tbe.tbe_expert_combine_backward(
            grad_out, self.answers, self.offsets, self.position, self.weights)
        grad_in = tbe.tbe_expert_product(*tbe.tbe_quantize_rows(grad_rows), *self.experts_t,
                                         self.offsets, out_dtype=torch.float32)
        grad_y = tbe.tbe_expert_dispatch_backward(grad_in, self.position)
        grad_logits = tbe.tbe_expert_route_backward(grad_weights, self.logits, self.chosen,
                                                    score="sigmoid")
        grad_y.addmm_(grad_logits, self.router)
        grad_x, grad_weight = tbe.tbe_rms_norm_backward(
            grad_y.to(dtype), self.h, self.weight, grad_h=grad_out.to(dtype))
        grad_table = tbe.tbe_embed_backward(grad_x, self.ids, self.rows, self.scale)
        return grad_table, grad_weight, grad_logits.T @ self.y.float()


def train(steps=20, tokens=4096, rows=8000, width=512, experts=16, k=2, lr=0.05, max_norm=1.0,
          balance=1e-3, seed=0, log=None):
    """Losses of the steps and the gradients' norms before clipping."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    layer = TokenLayer(rows, width, experts, k, g)
    ids = torch.randint(0, rows, (tokens,), generator=g, device="cuda")
    position = (0.1 * torch.randn(tokens, width, generator=g, device="cuda")).bfloat16()
    target = torch.randn(tokens, width, generator=g, device="cuda")
    losses, norms = [], []
    for step in range(steps):
        error = layer.forward(ids, position) - target
        losses.append(error.square().mean())
        grads = layer.backward(error * (2.0 / width))
        norms.append(tbe.tbe_grad_clip(grads, max_norm))
        for p, grad in zip((layer.table, layer.weight, layer.router), grads):
            p.sub_(grad, alpha=lr)
        load = layer.offsets.diff().float()
        layer.bias.add_(torch.sign(load.mean() - load), alpha=balance)
        if log:
            log(f"step {step}: loss {float(losses[-1]):.4f}, gradient norm {float(norms[-1]):.3f}")
    return [float(v) for v in losses], [float(v) for v in norms]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    train(steps=ap.parse_args().steps, log=print)
