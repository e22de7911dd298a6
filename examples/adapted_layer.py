"""A layer of frozen block-quantized weights with trained adapters, an expert layer behind it, and a small
training run of its adapters and of an embedding's additions.

    tokens -> Q6_K embedding lookup (plus a trained fp32 addition)
           -> Q4_K projection, with every request's own low-rank adapter beside it
           -> experts: tokens sorted by expert and gathered, one Q4_K product each, weighted and summed
              back onto the projection's result
           -> squared error against a target

The products run in the library's quantized kernels; what is trained is small and in fp32.  The gradient
with respect to the frozen weights' inputs uses the expanded weights (embed with the ids of all rows).

    python examples/adapted_layer.py [--steps 20] [--tokens 256]
"""
import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_quantized_matmul_quantize_amd as qmm  # noqa: E402
import synth  # noqa: E402

VOCAB, K, N_EXP, TOP_K, RANK, REQUESTS = 2000, 512, 8, 2, 8, 3


def weights(qtype, rows, k, seed):
    (rng,) = synth.rngs(seed, 1)
    return torch.from_numpy(np.ascontiguousarray(synth.gen_weights(qtype, rows, k, rng))).cuda()


def expand(w, qtype, rows, k):
    return qmm.embed(w, qtype, rows, k, torch.arange(rows, dtype=torch.int32, device="cuda"))


class Layer:
    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.table = weights(qmm.Q6_K, VOCAB, K, 1)
        self.proj = weights(qmm.Q4_K, K, K, 2)
        self.experts = [weights(qmm.Q4_K, K, K, 10 + e) for e in range(N_EXP)]
        self.proj_f = expand(self.proj, qmm.Q4_K, K, K)
        self.experts_f = [expand(w, qmm.Q4_K, K, K) for w in self.experts]
        # the synthetic weights' sizes: activations stay near 1
        self.unit = 1.0 / float(expand(self.table, qmm.Q6_K, VOCAB, K).std())
        self.norm = float(self.proj_f.norm(dim=1).mean())
        # trained: additions to the embedding, the requests' adapters
        self.extra = torch.zeros((VOCAB, K), device="cuda")
        self.a = (torch.randn((REQUESTS, RANK, K), generator=g) * K ** -0.5).cuda()
        self.b = torch.zeros((REQUESTS, K, RANK), device="cuda")
        self.scale = torch.full((REQUESTS,), 2.0, device="cuda")

    def step(self, tokens, requests, experts, gates, target, rate):
        """One step: forward, gradients of what is trained, update.  Returns the loss."""
        x = qmm.embed(self.table, qmm.Q6_K, VOCAB, K, tokens, self.unit)
        x = x + qmm.embed(self.extra, qmm.F32, VOCAB, K, tokens)
        p = qmm.matmul(self.proj, qmm.Q4_K, K, K, x) / self.norm
        y, h = qmm.lora(x, self.a, self.b, requests, self.scale, base=p, keep_h=True)
        order, pos, bounds = qmm.sort_ids(experts, N_EXP)
        xs = qmm.gather_sorted(y, pos, bounds)
        seg = bounds.tolist()
        hs = torch.zeros_like(xs)
        for e in range(N_EXP):
            if seg[e + 1] > seg[e]:
                hs[seg[e]:seg[e + 1]] = qmm.matmul(self.experts[e], qmm.Q4_K, K, K, xs[seg[e]:seg[e + 1]]) / self.norm
        z = qmm.combine(hs, pos, gates, base=y)
        diff = z - target
        loss = float((diff * diff).mean())
        dz = diff * (2.0 / diff.numel())
        # back: combine, experts, gather, adapters beside the projection, embedding
        dhs, _ = qmm.combine_backward(dz, hs, pos, gates, bounds)
        dxs = torch.zeros_like(xs)
        for e in range(N_EXP):
            dxs[seg[e]:seg[e + 1]] = dhs[seg[e]:seg[e + 1]] @ self.experts_f[e] / self.norm
        dy = dz + qmm.combine(dxs, pos)
        dx, da, db = qmm.lora_backward(x, dy, h, self.a, self.b, requests, self.scale,
                                       dx_base=dy @ self.proj_f / self.norm)
        de = qmm.embed_backward(dx, tokens, VOCAB)
        for value, grad in ((self.a, da), (self.b, db), (self.extra, de)):
            value -= grad * (rate / (float(grad.norm()) + 1e-12))   # steps of one length
        return loss


def main(steps=20, tokens=256, rate=0.1, quiet=False):
    layer = Layer()
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, VOCAB, (tokens,), generator=g, dtype=torch.int32)
    ids[-2:] = -1   # padding
    requests = (torch.arange(tokens) * REQUESTS // tokens).to(torch.int32)
    requests[:4] = -1   # no adapter
    top, experts = torch.topk(torch.randn((tokens, N_EXP), generator=g), TOP_K, dim=1)
    args = (ids.cuda(), requests.cuda(), experts.to(torch.int32).cuda().contiguous(), torch.softmax(top, 1).cuda(),
            torch.randn((tokens, K), generator=g).cuda())
    losses = [layer.step(*args, rate) for _ in range(steps)]
    if not quiet:
        for i, v in enumerate(losses):
            print(f"step {i}: loss {v:.5f}")
    return losses[0], losses[-1]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=256)
    o = ap.parse_args()
    main(o.steps, o.tokens)
