"""Plain 64-bit form of a mixture-of-experts layer's products (numpy), with the
error bound of the library's, and seeded inputs for it."""
import numpy as np
import torch

from decode_ref import activation, weights


def experts(n, hidden, inner, gated, seed):
    """(up, down, gate) of n experts as nv.Experts takes them, on the host: random codes and scales."""
    g = torch.Generator().manual_seed(seed)

    def matrix(rows, cols):
        return (torch.randint(0, 256, (n, rows, cols // 2), generator=g, dtype=torch.uint8),
                torch.randint(60, 112, (n, rows, cols // 16), generator=g, dtype=torch.uint8),
                (0.5 + torch.rand(n, generator=g)) * cols ** -0.5 / 128.0)

    return matrix(inner, hidden), matrix(hidden, inner), matrix(inner, hidden) if gated else None


def _product(w, alpha, x, ex):
    """alpha W x for x off by up to ex, and how far fp32 sums of it may be off
    (any order of n additions: (n + 2) 2^-24 sum |w x|, the tensor cores' twice
    that; the factors alpha and the vector's power of two round twice)."""
    v = alpha * (w @ x)
    err = alpha * (np.abs(w) @ ex + 2 * (len(x) + 2) * 2.0 ** -24 * (np.abs(w) @ (np.abs(x) + ex)))
    return v, err + 2.0 ** -22 * np.abs(v)


def moe(up, down, gate, x, ids, wts, act, residual=None):
    """(y, bound): the layer's output, and how far it may be off before its
    rounding to bf16.  x enters the products off by at most 2^-39 of its largest
    entry; no activation is steeper than 1.13, their functions are good to
    2^-20 of their argument; h is rounded to 11 bits (2^-12 of an entry),
    and twice to a grid of 2^-38 of a largest entry at most (2^-39 each); the slots' sum rounds top_k + 2 times."""
    tokens, k = ids.shape
    hidden = x.shape[1]
    y, err = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    size = np.zeros((tokens, hidden))
    cache = {}

    def matrix(name, m, e):
        if (name, e) not in cache:
            cache[name, e] = weights(m[0][e].numpy(), m[1][e].view(torch.uint8).numpy())
        return cache[name, e], float(m[2][e])

    for t in range(tokens):
        xt = x[t].astype(np.float64)
        ex = np.full(hidden, 2.0 ** -39 * np.abs(xt).max(initial=0.0))
        for s in range(k):
            e = int(ids[t, s])
            if not 0 <= e < up[0].shape[0]:
                continue
            h, eh = _product(*matrix("up", up, e), xt, ex)
            if gate is not None:
                g, eg = _product(*matrix("gate", gate, e), xt, ex)
                a, ea = activation(g, act), 1.13 * eg + 2.0 ** -20 * np.abs(g)
                h, eh = a * h, ea * np.abs(h) + np.abs(a) * eh + ea * eh
            else:
                h, eh = activation(h, act), 1.13 * eh + 2.0 ** -20 * np.abs(h)
            eh = eh + 2.0 ** -24 * np.abs(h)
            eh = eh + 2.0 ** -12 * (np.abs(h) + eh) + 2.0 ** -38 * (np.abs(h) + eh).max()
            o, eo = _product(*matrix("down", down, e), h, eh)
            w = float(wts[t, s])
            y[t] += w * o
            err[t] += abs(w) * eo
            size[t] += np.abs(w) * (np.abs(o) + eo)
    if residual is not None:
        y, size = y + residual, size + np.abs(residual)
    return y, err + (k + 2) * 2.0 ** -24 * size
