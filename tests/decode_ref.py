"""Plain 64-bit forms of the decode-step operators (numpy), with the
magnitudes that their error bounds need, and seeded inputs for them."""
import math

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def weights(codes, scales):
    """codes [rows, cols/2] and scales [rows, cols/16] -> q * Delta in float64 (exact)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    rows, half = codes.shape
    n = np.empty((rows, 2 * half), np.uint8)
    n[:, 0::2], n[:, 1::2] = codes & 15, codes >> 4
    q = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    return q * np.repeat(E4M3[scales], 16, axis=1)


def activation(v, act):
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "gelu":
        return 0.5 * v * (1.0 + np.vectorize(math.erf)(v / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        return v / (1.0 + np.exp(-v))
    return v


def within(got, v, err):
    """Whether bf16 outputs can be roundings of values at most err from v:
    rounding to nearest keeps the order, so they lie between the rounded ends."""
    low, high = (torch.from_numpy(np.asarray(e, np.float64)).to(torch.bfloat16).double().numpy() for e in (v - err, v + err))
    return np.all((low <= got) & (got <= high))


def linear(codes, scales, alpha, x, bias=None, act="none", gate=None, residual=None):
    """(y, bound): the product with its epilogue, and how far it may be off
    before its rounding to bf16 (see within()).  Products of q * Delta (six bits) and x (eight) are exact in fp32;
    any order of fp32 additions of n terms is off by (n + 2) 2^-24 sum |w x| at
    most, the tensor cores' by twice that; x may enter the products with an
    absolute error of 2^-25 of its vector's largest entry.  No activation is
    steeper than 1.13.  The epilogue's own roundings (at most 8 of 2^-23 of the
    quantities that they round; the activations' functions are good to 2^-21)
    follow."""
    w, x = weights(codes, scales), np.asarray(x, np.float64)
    cols = w.shape[1]
    mag = alpha * (np.abs(x) @ np.abs(w).T)
    err = 2 * (cols + 2) * 2.0 ** -24 * mag + \
        alpha * 2.0 ** -25 * np.abs(x).max(axis=1, initial=0.0)[:, None] * np.abs(w).sum(1)[None, :]
    v = alpha * (x @ w.T)
    big = np.abs(v)
    if bias is not None:
        v = v + bias
        big = big + np.abs(bias)
    v, err = activation(v, act), 1.13 * err + 2.0 ** -20 * big
    if gate is not None:
        v, err = v * gate, err * np.abs(gate)
    if residual is not None:
        v = v + residual
    err = err + 2.0 ** -22 * (np.abs(v) + (0 if residual is None else np.abs(residual)))
    return v, err


def rotate(x, cos_sin, pos, interleaved):
    """[tokens, heads, dim] rotated by position in x's precision (each product and sum rounded to it)."""
    r = cos_sin.shape[1]
    c, s = cos_sin[pos][:, None, :r // 2], cos_sin[pos][:, None, r // 2:]
    out = x.copy()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    p, q = a * c - b * s, b * c + a * s
    if interleaved:
        out[..., 0:r:2], out[..., 1:r:2] = p, q
    else:
        out[..., :r // 2], out[..., r // 2:r] = p, q
    return out


def angles(positions, rotary):
    half = rotary // 2
    t = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(half) / half)[None, :]
    return np.concatenate((np.cos(t), np.sin(t)), 1).astype(np.float32)


def attend(q, keys, values, scale, window=0):
    """One head group: q [g, d], keys and values [n, d] (float64) -> out [g, d],
    lse [g], and the bounds of both.  The scores are sums of d products, off by
    2 (d + 2) 2^-24 scale sum |q k| and, through the exponential's argument and
    the exponential itself, 2^-21 (1 + |s|); the weights enter the second
    product rounded to bf16 or better (half a unit of 8 significant bits:
    2^-8); n additions of fp32 follow in any order.  The output's own rounding
    to bf16 is left to within()."""
    n = len(keys)
    lo = max(0, n - window) if window else 0
    keys, values = keys[lo:], values[lo:]
    g, d = q.shape
    if n == 0:
        return np.zeros((g, d)), np.full(g, -np.inf), np.zeros((g, d)), np.zeros(g)
    s = scale * (q @ keys.T)
    ds = (2 * (d + 2) * 2.0 ** -24 * abs(scale) * (np.abs(q) @ np.abs(keys).T)).max(1) + \
        2.0 ** -21 * (1 + np.abs(s).max(1))
    m = s.max(1)
    p = np.exp(s - m[:, None])
    total = p.sum(1)
    out, mag = p @ values / total[:, None], p @ np.abs(values) / total[:, None]
    rel = 2 * np.expm1(ds) + 2 * (n - lo + 8) * 2.0 ** -24
    lse = m + np.log(total)
    bound = (2.0 ** -8 + rel)[:, None] * mag
    return out, lse, bound, ds + rel + 2.0 ** -22 * np.abs(lse)


def page_table(lengths, page, pages, seed, spare=1):
    """Scattered pages for sequences of these lengths (int32 [n, width]); entries behind the last page are -1."""
    rng = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lengths]
    assert sum(need) <= pages
    perm = rng.permutation(pages)
    table = np.full((len(need), max(need, default=0) + spare), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table
