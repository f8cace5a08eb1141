"""The experts' products against the plain 64-bit form, within the bound that
moe_ref derives."""
import numpy as np
import pytest
import torch

import moe_ref
import nvfp4_block_scale_gb300 as nv
from decode_ref import within

pytestmark = pytest.mark.gpu


def _inputs(tokens, hidden, n, k, seed, invalid=0.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((tokens, hidden), generator=g) * torch.exp(2 * torch.randn((tokens, 1), generator=g))).to(torch.bfloat16)
    ids = torch.stack([torch.randperm(n, generator=g)[:k] for _ in range(tokens)]).int() if k <= n else \
        torch.randint(0, n, (tokens, k), generator=g).int()
    if invalid:
        ids[torch.rand((tokens, k), generator=g) < invalid] = -1
    w = torch.rand((tokens, k), generator=g) + 0.1
    return x, ids, w, torch.randn((tokens, hidden), generator=g).to(torch.bfloat16)


def _cuda(ms):
    return [None if m is None else tuple(t.cuda() for t in m) for m in ms]


def _run(host, x, ids, w, act="silu", residual=None, **kw):
    ex = nv.Experts(*_cuda(host))
    y = nv.moe(ex, x.cuda(), ids.cuda(), w.cuda(), activation=act, residual=None if residual is None else residual.cuda(), **kw)
    torch.cuda.synchronize()
    return y


def _check(host, x, ids, w, act, residual, y):
    want, err = moe_ref.moe(*host, x.double().numpy(), ids.numpy(), w.double().numpy(), act,
                            None if residual is None else residual.double().numpy())
    assert within(y.double().cpu().numpy(), want, err)


# tokens, hidden, inner, experts, slots: one tile and less than a step; whole steps; a block beyond them (rows of codes
# that 16-byte loads do not fit); more pairs of an expert than a job takes; more experts than threads; vectors so long
# that a job takes few of them; more tiles than warps
SHAPES = [(1, 16, 16, 1, 1), (1, 64, 48, 4, 2), (3, 256, 128, 5, 3), (5, 144, 80, 3, 2), (7, 400, 272, 4, 4),
          (40, 128, 64, 2, 2), (33, 96, 32, 1, 1), (20, 64, 48, 700, 6), (1, 512, 96, 16, 8), (9, 9600, 32, 2, 2),
          (4, 32, 20480, 2, 1), (17, 2048, 256, 6, 2), (64, 256, 512, 8, 8)]


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_products(shape, gated):
    tokens, hidden, inner, n, k = shape
    host = moe_ref.experts(n, hidden, inner, gated, seed=sum(shape))
    x, ids, w, r = _inputs(tokens, hidden, n, k, 7)
    _check(host, x, ids, w, "silu", r, _run(host, x, ids, w, "silu", r))


# around the edges of what one MMA, a tile of several and a job take; columns in whole steps, and rows of codes on 8 bytes
@pytest.mark.parametrize("hidden,inner", [(512, 256), (272, 144)])
@pytest.mark.parametrize("pairs", [2, 7, 8, 9, 16, 17, 23, 24, 25, 31, 32, 33, 57, 65])
def test_pairs_of_an_expert(pairs, hidden, inner):
    host = moe_ref.experts(2, hidden, inner, pairs % 2 == 1, seed=pairs)
    x, ids, w, r = _inputs(pairs + 3, hidden, 2, 1, pairs)
    ids[:] = 1
    ids[torch.randperm(pairs + 3, generator=torch.Generator().manual_seed(pairs))[:pairs]] = 0
    _check(host, x, ids, w, "silu", r, _run(host, x, ids, w, "silu", r))


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [True, False])
def test_activations(act, gated):
    host = moe_ref.experts(4, 128, 64, gated, 3)
    x, ids, w, _ = _inputs(6, 128, 4, 2, 8)
    _check(host, x, ids, w, act or "none", None, _run(host, x, ids, w, act))


def test_slots_without_an_expert_and_named_twice():
    host = moe_ref.experts(5, 128, 64, True, 4)
    x, ids, w, r = _inputs(19, 128, 5, 6, 9, invalid=0.4)
    ids[0], ids[1], ids[2] = -1, 3, 5  # nobody; one expert six times; past the last
    ids[3] = torch.tensor([2, 2, -7, 2 ** 31 - 1, 4, -2 ** 31])
    for residual in (r, None):
        y = _run(host, x, ids, w, "silu", residual)
        _check(host, x, ids, w, "silu", residual, y)
        assert torch.equal(y[0].cpu(), (residual if residual is not None else torch.zeros_like(r))[0])
    empty = torch.full_like(ids, -1)
    assert torch.equal(_run(host, x, empty, w, "silu", r).cpu(), r)


# vectors so long that a job takes three pairs, or one; so long that one fits only beside eight warps' units (rows of codes
# in whole words and on any byte; of x, of h)
@pytest.mark.parametrize("shape", [(12, 48, 14336, 2, 2), (16, 14336, 32, 2, 2), (9, 16, 49152, 3, 2), (5, 49152, 16, 2, 2),
                                   (2, 16, 73728, 2, 2), (2, 16, 73744, 2, 2), (2, 73744, 16, 2, 2)])
def test_long_vectors(shape):
    tokens, hidden, inner, n, k = shape
    host = moe_ref.experts(n, hidden, inner, tokens % 2 == 0, seed=sum(shape))
    x, ids, w, r = _inputs(tokens, hidden, n, k, 13)
    _check(host, x, ids, w, "silu", r, _run(host, x, ids, w, "silu", r))


def test_longest_vectors_that_every_call_takes():
    """49152 columns with the most experts and pairs that a launch has.  The experts are one expert's tensors 1024
    times (0 bytes apart), so that a token's slots sum to its product times the sum of their weights."""
    host = moe_ref.experts(1, 16, 49152, False, 23)
    x, _, _, _ = _inputs(64, 16, 1024, 1, 24)
    g = torch.Generator().manual_seed(25)
    ids = torch.stack([torch.randperm(1024, generator=g)[:32] for _ in range(64)]).int()
    w = torch.rand((64, 32), generator=g) + 0.1
    up, down = (tuple(t.cuda().expand(1024, *t.shape[1:]) for t in m) for m in host[:2])
    y = nv.moe(nv.Experts(up, down), x.cuda(), ids.cuda(), w.cuda())
    want, err = moe_ref.moe(*host, x.double().numpy(), torch.zeros((64, 1), dtype=torch.int32).numpy(),
                            w.double().sum(1, keepdim=True).numpy(), "silu")
    # (31 more slots of one sign: as many more roundings of the slots' sum)
    assert within(y.double().cpu().numpy(), want, err + 31 * 2.0 ** -24 * (abs(want) + err))


def test_entries_down_to_the_smallest_bf16():
    """Vectors whose largest entry is 2^-95 or less enter the products exactly: bf16 ends at 2^-133.  The largest meets
    weights of 0, so that the others are what the output shows."""
    host = moe_ref.experts(2, 128, 64, False, 26)
    up, down, _ = host
    up[0][:, :, 0] &= 0xF0  # (a byte's lower half is the even column)
    host = (up[0], up[1], up[2] * 2.0 ** 100), (down[0], down[1], down[2] * 2.0 ** 30), None
    g = torch.Generator().manual_seed(27)
    x = torch.randint(-127, 128, (8, 128), generator=g).double() * 2.0 ** -133
    x[:, 0] = torch.tensor([2.0 ** e for e in (-95, -100, -110, -112, -113, -120, -126, -133)], dtype=torch.float64)
    exact = x.numpy().copy()
    x = x.to(torch.bfloat16)
    assert (x.double().numpy() == exact).all()
    ids, w = torch.arange(8).int()[:, None] % 2, torch.ones((8, 1))
    y = _run(host, x, ids, w, "none")
    _check(host, x, ids, w, "none", None, y)
    assert bool((y != 0).any(1).all())


def _one_slot(host, e, x, act):
    """(y, bound) of one token's only slot, of weight 1, as moe_ref.moe, with f16's own half step for h: 11 bits are 2^-11
    of a value at most (of 1 + 2^-11, say, whose neighbours are 1 and 1 + 2^-10); and fp32's end, twice, and that of f16
    under 2^126: 2^-150, 2^-150 and 2^-151."""
    up, down, gate = (None if m is None else (moe_ref.weights(m[0][e].numpy(), m[1][e].numpy()), float(m[2][e])) for m in host)
    ex = np.full(len(x), 2.0 ** -39 * np.abs(x).max())
    h, eh = moe_ref._product(*up, x, ex)
    if gate is not None:
        g, eg = moe_ref._product(*gate, x, ex)
        a, ea = moe_ref.activation(g, act), 1.13 * eg + 2.0 ** -20 * np.abs(g)
        h, eh = a * h, ea * np.abs(h) + np.abs(a) * eh + ea * eh
    else:
        h, eh = moe_ref.activation(h, act), 1.13 * eh + 2.0 ** -20 * np.abs(h)
    eh = eh + 2.0 ** -24 * np.abs(h)
    eh = eh + 2.0 ** -11 * (np.abs(h) + eh) + 2.0 ** -38 * (np.abs(h) + eh).max() + 2.5 * 2.0 ** -150
    y, err = moe_ref._product(*down, h, eh)
    return y, err + 3 * 2.0 ** -24 * (np.abs(y) + err)


def test_products_between_that_fp32_hardly_holds():
    """h around 2^-130: f16 of eight's common power of two ends no higher than fp32 itself."""
    up, down, _ = moe_ref.experts(2, 64, 128, False, 28)
    host = (up[0], up[1], up[2] * 2.0 ** -120), (down[0], down[1], down[2] * 2.0 ** 110), None
    g = torch.Generator().manual_seed(29)
    x = (torch.randn((6, 64), generator=g) * 2.0 ** torch.tensor([0.0, -4, -8, -10, -12, 4])[:, None]).to(torch.bfloat16)
    ids, w = torch.arange(6).int()[:, None] % 2, torch.ones((6, 1))
    y = _run(host, x, ids, w, "none").double().cpu().numpy()
    for t in range(6):
        assert within(y[t], *_one_slot(host, t % 2, x[t].double().numpy(), "none"))


@pytest.mark.parametrize("hidden,inner", [(16, 16), (32, 16), (48, 32), (16, 96), (64, 80)])
@pytest.mark.parametrize("act,gated", [("none", True), ("relu", True), ("gelu_tanh", True), ("silu", False)])
def test_small_layers(hidden, inner, act, gated):
    """So few columns that single roundings of h show in an output."""
    host = moe_ref.experts(30, hidden, inner, gated, hidden + inner)
    x, _, _, _ = _inputs(240, hidden, 30, 1, 31)
    ids, w = torch.arange(240).int()[:, None] % 30, torch.ones((240, 1))
    y = _run(host, x, ids, w, act).double().cpu().numpy()
    for t in range(240):
        assert within(y[t], *_one_slot(host, t % 30, x[t].double().numpy(), act))
