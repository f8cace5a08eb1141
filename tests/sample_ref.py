"""Plain 64-bit form of sampling with temperature, top-k, top-p and min-p (numpy, one row)."""
import numpy as np


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, margin) of one row: margin is how far the sums that decide
    lie from the decision, relative to the row's mass (a result of other
    arithmetic may differ where it is tiny).  Weights of 1 are exact in any
    arithmetic, and so are their sums and (24 bits times a sum below 2^20) the
    goals: such rows have a margin of 1."""
    x = np.asarray(x, np.float64)
    alive = np.flatnonzero(x > -np.inf)
    if len(alive) == 0:
        return -1, -np.inf, 1.0
    order = alive[np.argsort(-x[alive], kind="stable")]
    m = x[order[0]]
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x[order] == m, 1.0, np.exp((x[order] - m) / temperature))
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    margin = 1.0
    exact = bool((w == 1.0).all())
    if top_p < 1.0:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))
        goal = max(top_p, 0.0) * w.sum()
        stays = before < goal
        stays[0] = True
        margin = min(margin, np.abs(before[1:] - goal).min(initial=np.inf) / w.sum()) if len(w) > 1 else margin
        order, w = order[stays], w[stays]
    if min_p > 0:
        stays = w >= min(min_p, 1.0)
        margin = min(margin, (np.abs(w - min_p) / min_p).min())
        order, w = order[stays], w[stays]
    place = np.argsort(order)
    order, w = order[place], w[place]
    upto = np.cumsum(w)
    u = min(max(u, 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    goal = u * upto[-1]
    j = min(int((upto <= goal).sum()), len(w) - 1)
    edges = np.abs(upto - goal)[w > 0]
    if u > 0:
        margin = min(margin, edges.min() / upto[-1])
    return int(order[j]), float(np.log(w[j]) - np.log(upto[-1])), 1.0 if exact else margin
