"""A decoder layer on NVFP4 weights, one token per sequence at a time.

Quantizes a layer's seven projections, takes in ragged prompts, then decodes a
few tokens per sequence with the library's decode-step operators:

  qkv  = linear(Wqkv, norm(x))             the product, its bias in the epilogue
  q    = kv_append(cache, qkv, ...)        rotates q and k, stores k and v
  a    = paged_attention(cache, q, ...)    the new token over its sequence
  x    = linear(Wo, a, residual=x)
  up   = linear(Wup, norm(x))
  gate = linear(Wgate, norm(x), activation="silu", gate=up)
  x    = linear(Wdown, gate, residual=x)

The step is captured once in a CUDA graph and replayed.  Every output is
compared with the same layer in plain fp32 on the dequantized weights and an
unpaged cache.

  python examples/decode_layer.py [--cache e4m3] [--hidden 4096] ...
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import nvfp4_block_scale_gb300 as nv

EPS = 1e-5


def norm(x):
    """Root-mean-square norm without a weight, in fp32."""
    f = x.float()
    return (f * torch.rsqrt(f.pow(2).mean(-1, keepdim=True) + EPS)).to(torch.bfloat16)


class Layer:
    def __init__(self, hidden, inner, q_heads, kv_heads, head_dim, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.hidden = q_heads, kv_heads, head_dim, hidden
        wide = (q_heads + 2 * kv_heads) * head_dim
        shapes = {"qkv": (wide, hidden), "o": (hidden, q_heads * head_dim), "up": (inner, hidden), "gate": (inner, hidden),
                  "down": (hidden, inner)}
        self.w, self.plain = {}, {}
        for name, (rows, cols) in shapes.items():
            w = (torch.randn((rows, cols), generator=g, device="cuda") * cols ** -0.5).to(torch.bfloat16)
            codes, scales, alpha = nv.quantize(w, nv.FOUR_OVER_SIX)
            self.w[name] = (codes, scales, alpha, rows, cols)
            self.plain[name] = nv.dequantize(codes, scales, alpha, rows, cols).float()  # for the comparison only
        self.bias = (0.1 * torch.randn(wide, generator=g, device="cuda")).to(torch.bfloat16)

    def __call__(self, x, cache, seq, pos, table, lengths, cos_sin, space):
        """One step: x bf16 [sequences, hidden] -> the layer's output."""
        ws = space.get
        qkv = nv.linear(*self.w["qkv"], norm(x), bias=self.bias, workspace=ws("qkv"))
        q = nv.kv_append(cache, qkv, self.q_heads, seq, pos, table, cos_sin)
        a = nv.paged_attention(cache, q, table, lengths, workspace=ws("attention"))
        x = nv.linear(*self.w["o"], a.flatten(1), residual=x, workspace=ws("o"))
        h = norm(x)
        up = nv.linear(*self.w["up"], h, workspace=ws("up"))
        gate = nv.linear(*self.w["gate"], h, activation="silu", gate=up, workspace=ws("gate"))
        return nv.linear(*self.w["down"], gate, residual=x, workspace=ws("down"))

    def space(self, cache, batch):
        """The workspaces of a step, allocated once."""
        s = {n: nv.linear_workspace(w[3], w[4], batch) for n, w in self.w.items()}
        s["attention"] = nv.attention_workspace(cache, self.q_heads)
        return s

    def reference(self, x, keys, values, position, cos_sin):
        """The same for one sequence in plain fp32: x [hidden]; keys and values
        [tokens so far, kv_heads, head_dim].  Returns the output and the new key and value."""
        p, d, half = self.plain, self.head_dim, cos_sin.shape[1] // 2
        c, s = cos_sin[position, :half], cos_sin[position, half:]
        rotate = lambda t: torch.cat((t[..., :half] * c - t[..., half:] * s, t[..., half:] * c + t[..., :half] * s), -1)  # noqa: E731
        qkv = (p["qkv"] @ norm(x).float() + self.bias.float()).view(-1, d)
        q, k, v = qkv.split((self.q_heads, self.kv_heads, self.kv_heads))
        k, v = rotate(k), v
        keys, values = torch.cat((keys, k[None])), torch.cat((values, v[None]))
        g = self.q_heads // self.kv_heads
        score = torch.einsum("hgd,thd->hgt", rotate(q).view(self.kv_heads, g, d), keys) * d ** -0.5
        a = torch.einsum("hgt,thd->hgd", score.softmax(-1), values).reshape(-1)
        x = x.float() + p["o"] @ a
        h = norm(x).float()
        return x + p["down"] @ (torch.nn.functional.silu(p["gate"] @ h) * (p["up"] @ h)), keys, values


def run(hidden=2048, inner=5632, q_heads=16, kv_heads=4, head_dim=128, page=16, prompts=(700, 1, 33, 250), steps=4,
        kind=torch.bfloat16, seed=0):
    """Decodes `steps` tokens; returns the largest relative error of a step's
    output (2-norm, per sequence) and the microseconds of one replayed step."""
    layer, n = Layer(hidden, inner, q_heads, kv_heads, head_dim, seed), len(prompts)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    longest = max(prompts) + steps
    t = torch.arange(longest, device="cuda")[:, None] * 10000.0 ** (-torch.arange(head_dim // 2, device="cuda") / (head_dim // 2))
    cos_sin = torch.cat((t.cos(), t.sin()), 1).float().contiguous()

    # pages in a scattered order, enough for prompt and new tokens
    need = [-(-(p + steps) // page) for p in prompts]
    order = torch.randperm(sum(need), generator=g, device="cuda").int().split(need)
    table = torch.full((n, max(need)), -1, dtype=torch.int32, device="cuda")
    for i, o in enumerate(order):
        table[i, :len(o)] = o
    scale = torch.full((kv_heads,), 4.0 / 448.0, device="cuda") if kind != torch.bfloat16 else None
    cache = nv.KVCache.empty(sum(need), kv_heads, page, head_dim, kind, k_scale=scale, v_scale=scale)

    # the prompts' keys and values in one append (their queries are not needed here)
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor(prompts, device="cuda")).int()
    pos = torch.cat([torch.arange(p, device="cuda") for p in prompts]).int()
    kv = torch.randn((len(seq), 2 * kv_heads * head_dim), generator=g, device="cuda").to(torch.bfloat16)
    nv.kv_append(cache, kv, 0, seq, pos, table, cos_sin)
    plain = []
    for i in range(n):  # the reference's own cache: what the pages hold, read back in order
        rows = [(p[table[i, :need[i]].long()].transpose(1, 2).flatten(0, 1)[:prompts[i]]).float() *
                (1.0 if scale is None else scale[:, None]) for p in (cache.k, cache.v)]
        plain.append(rows)

    x = torch.randn((n, hidden), generator=g, device="cuda").to(torch.bfloat16)
    at = torch.tensor(prompts, dtype=torch.int32, device="cuda")  # position of the next token
    who, lengths = torch.arange(n, dtype=torch.int32, device="cuda"), at + 1
    space = layer.space(cache, n)
    layer(x, cache, who, at, table, lengths, cos_sin, space)  # first call: one-time set-up outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, cache, who, at, table, lengths, cos_sin, space)

    worst = 0.0
    for _ in range(steps):
        graph.replay()
        for i in range(n):
            want, k, v = layer.reference(x[i], *plain[i], int(at[i]), cos_sin)
            plain[i] = [k, v]
            worst = max(worst, float((out[i].float() - want).norm() / want.norm()))
        x.copy_(out)  # the next token's input
        at += 1
        lengths += 1

    at -= steps  # time the step at the prompts' lengths
    lengths -= steps
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        graph.replay()
    b.record()
    b.synchronize()
    return worst, a.elapsed_time(b) * 1000 / 20


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--inner", type=int, default=14336)
    ap.add_argument("--q-heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    a = ap.parse_args()
    kind = torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn
    worst, us = run(a.hidden, a.inner, a.q_heads, a.kv_heads, a.head_dim, kind=kind)
    print(f"4 sequences, 4 tokens each: largest relative error of a step {worst:.4f}, {us:.1f} us a step")


if __name__ == "__main__":
    main()
