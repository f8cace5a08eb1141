"""A mixture-of-experts layer on NVFP4 weights and the choice of the next token,
the second half of a decode step:

  h      = norm(x)
  ids, w = moe_route(h, router, k)              which experts, and how much of each
  x      = moe(experts, h, ids, w, residual=x)  their products
  logits = linear(Whead, norm(x))               the vocabulary's projection
  token  = sample(logits, u, temperature, top_k, top_p)

Quantizes the experts in one grouped call, captures the step once in a CUDA
graph and replays it on fresh inputs.  Every output is compared with the same
layer in plain fp32 on the dequantized weights, every token with the one that
the definition of sampling gives for the step's logits.

  python examples/moe_layer.py [--hidden 4096] [--experts 64] ...
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import nvfp4_block_scale_gb300 as nv
from decode_layer import norm


class Layer:
    def __init__(self, hidden, inner, experts, top_k, vocabulary, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda *s: (torch.randn(s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
        self.top_k = top_k
        self.router = make(experts, hidden)
        self.experts = nv.Experts.quantize(make(experts, inner, hidden), make(experts, hidden, inner),
                                           make(experts, inner, hidden), mode=nv.FOUR_OVER_SIX)
        head = make(vocabulary, hidden)
        self.head = (*nv.quantize(head, nv.FOUR_OVER_SIX), vocabulary, hidden)

    def __call__(self, x, u, settings, space):
        h = norm(x)
        ids, w = nv.moe_route(h, self.router, self.top_k)
        x = nv.moe(self.experts, h, ids, w, residual=x, workspace=space["moe"])
        logits = nv.linear(*self.head, norm(x), workspace=space["head"])
        return x, logits, nv.sample(logits, u, **settings)

    def space(self, batch):
        return {"moe": nv.moe_workspace(self.experts, batch, self.top_k),
                "head": nv.linear_workspace(self.head[3], self.head[4], batch)}

    def reference(self, x):
        """The layer's output and logits for one token in plain fp32 on the dequantized weights."""
        h = norm(x)
        logit = self.router.double() @ h.double()
        ids = torch.argsort(logit, descending=True, stable=True)[:self.top_k]
        weight = logit[ids].softmax(0).float()
        y = x.float()
        for e, w in zip(ids.tolist(), weight):
            up, down, gate = (nv.dequantize(m[0][e], m[1][e], m[2][e:e + 1], *s).float() for m, s in
                              zip(self.experts.tensors, [(self.experts.inner, self.experts.hidden),
                                                         (self.experts.hidden, self.experts.inner),
                                                         (self.experts.inner, self.experts.hidden)]))
            y = y + w * (down @ (torch.nn.functional.silu(gate @ h.float()) * (up @ h.float())))
        return y, nv.dequantize(*self.head).float() @ norm(y).float()


def choose(logits, u, temperature, top_k, top_p):
    """The token of one row by the definition, in fp64."""
    order = torch.argsort(logits.double(), descending=True, stable=True)[:top_k]
    w = torch.exp((logits[order].double() - logits.max().double()) / temperature)
    order = order[torch.cumsum(w, 0) - w < top_p * w.sum()]
    order = torch.sort(order)[0]
    upto = torch.cumsum(torch.exp((logits[order].double() - logits.max().double()) / temperature), 0)
    return int(order[int((upto <= u.double() * upto[-1]).sum())])


def run(hidden=2048, inner=1024, experts=32, top_k=4, vocabulary=32000, batch=8, steps=4, seed=0):
    """Returns the largest relative error of a step's output and logits (2-norm,
    per sequence), the chosen tokens and those of the definition, and the
    microseconds of one replayed step."""
    layer = Layer(hidden, inner, experts, top_k, vocabulary, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    f32 = lambda v: torch.tensor(float(torch.tensor(v, dtype=torch.float32)), dtype=torch.float64, device="cuda")  # noqa: E731
    settings = dict(temperature=0.8, top_k=50, top_p=0.9)
    x, u = torch.empty((batch, hidden), dtype=torch.bfloat16, device="cuda"), torch.empty(batch, device="cuda")
    x.normal_(generator=g)
    u.uniform_(generator=g)
    space = layer.space(batch)
    layer(x, u, settings, space)  # first call: one-time set-up outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, logits, token = layer(x, u, settings, space)
    worst, tokens, want = 0.0, [], []
    for _ in range(steps):
        x.normal_(generator=g)
        u.uniform_(generator=g)
        graph.replay()
        for i in range(batch):
            y, plain = layer.reference(x[i])
            for a, b in ((out[i], y), (logits[i], plain)):
                worst = max(worst, float((a.float() - b).norm() / b.norm()))
            want.append(choose(logits[i], u[i], f32(0.8), 50, f32(0.9)))
        tokens += token.tolist()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        graph.replay()
    b.record()
    b.synchronize()
    return worst, tokens, want, a.elapsed_time(b) * 1000 / 20


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=6)
    ap.add_argument("--vocabulary", type=int, default=128256)
    ap.add_argument("--batch", type=int, default=8)
    a = ap.parse_args()
    worst, tokens, want, us = run(a.hidden, a.inner, a.experts, a.top_k, a.vocabulary, a.batch)
    print(f"{a.batch} sequences, 4 steps: largest relative error {worst:.4f}, "
          f"{sum(t == w for t, w in zip(tokens, want))} of {len(want)} tokens as defined, {us:.1f} us a step")


if __name__ == "__main__":
    main()
