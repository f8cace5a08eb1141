"""The experts' products against the plain 64-bit form, within the bound that
moe_ref derives."""
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
