"""The router against its formulas in 64 bits: the experts and their order have
to be equal, the weights within fp32's roundings."""
import numpy as np
import pytest
import torch

import nvfp4_block_scale_gb300 as nv

pytestmark = pytest.mark.gpu


def _want(x, router, k, scoring, renormalize, bias, scale):
    logit = x.double().numpy() @ router.double().numpy().T
    if scoring == "sigmoid":
        p = 1.0 / (1.0 + np.exp(-logit))
        score = p + (0.0 if bias is None else bias.double().numpy())
    else:
        e = np.exp(logit - logit.max(1, keepdims=True))
        p, score = e / e.sum(1, keepdims=True), logit
    ids = np.argsort(-score, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    return ids, w * scale


def _check(x, router, k, scoring="softmax", renormalize=True, bias=None, scale=1.0):
    ids, w = nv.moe_route(x.cuda(), router.cuda(), k, scoring, renormalize, None if bias is None else bias.cuda(), scale)
    torch.cuda.synchronize()
    wi, ww = _want(x, router, k, scoring, renormalize, bias, scale)
    assert np.array_equal(ids.cpu().numpy(), wi)
    # many tokens and experts: chosen as if exactly, weighted by logits off by 2^-18 (2^-16.4 with an fp32 router) of
    # their vectors' norms at most, which move a weight by twice that of itself at most
    off = 0.0
    if x.shape[0] >= 128 or (x.shape[0] >= 16 and x.shape[0] * router.shape[0] >= 8192):
        off = 2 ** (-18 if router.dtype == torch.bfloat16 else -16.4) * \
            x.double().norm(dim=1).numpy()[:, None] * float(router.double().norm(dim=1).max())
    # an exponential good to 2 ulp of an argument off by 2^-24 of up to 40, a sum of up to 1024 of them in any order
    # (each lane's at most 64 roundings deep), a quotient and a product
    err = np.abs(w.double().cpu().numpy() - ww)
    assert np.all(err <= (2 * off + 2 * (2 ** -22 + 40 * 2.0 ** -24) + 64 * 2.0 ** -24 + 2 ** -23) * np.abs(ww) + 1e-44)
    return ids, w


# tokens, hidden, experts, k: one of everything; fewer experts than CTAs of a cluster; tokens that no cluster divides;
# more experts than threads; every expert chosen; columns that no lane divides; many tokens and experts (the tensor
# cores): fewer columns than warps, tokens that no tile divides, all of an expert's warps
SHAPES = [(1, 8, 1, 1), (1, 2048, 128, 8), (3, 264, 5, 5), (61, 512, 8, 2), (130, 72, 60, 6), (700, 40, 33, 3),
          (2, 136, 1024, 32), (9, 7168, 256, 8), (1, 1000, 3, 1),
          (128, 8, 64, 6), (129, 72, 8, 8), (33, 72, 256, 8), (200, 520, 256, 8), (16, 264, 512, 4), (47, 4096, 1000, 32), (300, 1032, 129, 1)]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scoring,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_choice_and_weights(shape, scoring, renormalize, kind):
    tokens, hidden, experts, k = shape
    g = torch.Generator().manual_seed(sum(shape))
    x = torch.randn((tokens, hidden), generator=g).to(torch.bfloat16)
    r = (1.5 * hidden ** -0.5 * torch.randn((experts, hidden), generator=g)).to(kind)
    bias = 0.2 * torch.randn(experts, generator=g) if scoring == "sigmoid" else None
    _check(x, r, k, scoring, renormalize, bias, 2.5 if scoring == "sigmoid" else 1.0)


@pytest.mark.parametrize("tokens", [5, 140])
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_scores_closer_than_fp32_tells_apart(kind, tokens):
    """Every logit is 2^14 (eleven 1024s and so on, large and cancelling ones
    among them) plus a multiple of 2^-12, which fp32 would drop."""
    g = torch.Generator().manual_seed(3)
    experts, hidden = 64, 512
    small = torch.randperm(experts, generator=g).double()
    r = torch.zeros((experts, hidden), dtype=torch.float64)
    r[:, 0::2] = 64.0 * torch.randint(1, 200, (experts, hidden // 2), generator=g)
    r[:, 1::2] = -r[:, 0::2]
    r = r[:, torch.randperm(hidden, generator=g)]
    x = torch.ones((tokens, hidden))
    r[:, 7], r[:, 300], r[:, 5] = 16384.0, small * 2.0 ** -12, 0.0
    r[:, 5] = 16384.0 - r.sum(1) + small * 2.0 ** -12  # what the pairs that were overwritten left over
    r = r.to(kind)
    exact = r.double().sum(1)
    ids, _ = nv.moe_route(x.to(torch.bfloat16).cuda(), r.cuda(), 32, "softmax", True)
    order = sorted(range(experts), key=lambda e: (-exact[e].item(), e))[:32]
    assert exact.unique().numel() > 32 and ids.cpu().tolist() == [order] * tokens


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_neighbours_in_every_token(kind):
    """Experts in pairs whose logits differ by 2^-20 of their terms' sizes: the tensor cores leave each pair open."""
    g = torch.Generator().manual_seed(11)
    x = torch.randn((70, 512), generator=g).to(torch.bfloat16)
    r = torch.randn((64, 512), generator=g).to(torch.bfloat16)
    r = torch.cat((r, r))
    r[64:, 3] = 0.0
    r[:64, 3] = 2.0 ** -12 * torch.randn(64, generator=g).to(torch.bfloat16)
    _check(x, r.to(kind), 16)
    _check(x, r.to(kind), 16, "sigmoid", True, 0.01 * torch.randn(64, generator=g).repeat(2))


def test_tokens_of_zeros_and_tiny_ones():
    g = torch.Generator().manual_seed(12)
    x = torch.randn((70, 256), generator=g)
    x[::7] = 0.0
    x[3] *= 2.0 ** -90
    r = torch.randn((128, 256), generator=g).to(torch.bfloat16)
    _check(x.to(torch.bfloat16), r, 5)
    _check(x.to(torch.bfloat16), torch.cat((r[:64], r[:64])), 5, "sigmoid", False, torch.zeros(128))


@pytest.mark.parametrize("tokens", [3, 200])
def test_experts_that_a_bias_masks(tokens):
    """A bias of -inf is below everything, one of inf above; of equal ones the lower first."""
    g = torch.Generator().manual_seed(14)
    x = torch.randn((tokens, 256), generator=g).to(torch.bfloat16)
    r = (0.1 * torch.randn((96, 256), generator=g)).to(torch.bfloat16)
    bias = 0.1 * torch.randn(96, generator=g)
    bias[torch.randperm(96, generator=g)[:70]] = -float("inf")
    _check(x, r, 8, "sigmoid", True, bias)
    _check(x, r, 30, "sigmoid", True, bias)  # (26 of them are not masked)
    bias[torch.randperm(96, generator=g)[:3]] = float("inf")
    _check(x, r, 8, "sigmoid", False, bias)


def test_rows_whose_squares_underflow():
    """Rows of 2^-75 whose products cancel to 2^-20 of their terms: experts that the tensor cores leave open, which
    norms of zero would not show."""
    g = torch.Generator().manual_seed(15)
    x = torch.randn((130, 256), generator=g).to(torch.bfloat16)
    x[:, 128:] = -x[:, :128]
    r = torch.randn((64, 128), generator=g).to(torch.bfloat16)
    r = torch.cat((r, r), 1)
    r[:, 3], r[:, 131] = 2.0 ** -14 * torch.randn(64, generator=g), 0.0
    _check(x, (r.float() * 2.0 ** -75).to(torch.bfloat16), 12)


def test_equal_scores_go_to_the_lower_expert():
    x = torch.randn((4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    row = torch.randn((1, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    ids, w = _check(x, row.expand(300, 64).contiguous(), 7)
    assert ids.cpu().tolist() == [list(range(7))] * 4 and torch.allclose(w, torch.full_like(w, 1 / 7))
    _check(x, torch.zeros((9, 64)), 9, "sigmoid", False, torch.tensor([0.0, -0.0, 1, 1, 0, -1, 2, 2, 0]))


def test_strides_streams_and_repeats():
    g = torch.Generator().manual_seed(5)
    x = torch.randn((20, 304), generator=g).to(torch.bfloat16).cuda()[:, :160]
    r = torch.randn((16, 168), generator=g).cuda()[:, :160]
    a = nv.moe_route(x, r, 4)
    b = nv.moe_route(x.contiguous(), r.contiguous(), 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = nv.moe_route(x, r, 4, stream=s)
    torch.cuda.synchronize()
    for p, q in zip(a + a, b + c):
        assert torch.equal(p, q)
    assert nv.moe_route(x[:0], r, 4)[0].shape == (0, 4)


def _exact_logits(tokens, experts, level, kind, seed):
    """Operands whose logits, `level` give or take a few tens, every order of fp32 sums forms exactly: multiples of
    1/8 (of level / 64) below 2^11."""
    g = torch.Generator().manual_seed(seed)
    x = torch.ones((tokens, 128))
    x[:, 64:] = 2.0 * torch.randint(0, 2, (tokens, 64), generator=g) - 1.0
    r = torch.full((experts, 128), level / 64)
    r[:, 64:] = torch.randint(-8, 9, (experts, 64), generator=g) / 8
    assert torch.equal(r.to(torch.bfloat16).float(), r)
    return x.to(torch.bfloat16), r.to(kind)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("level", [-300.0, -120.0, -95.0, -20.0])
@pytest.mark.parametrize("tokens", [3, 200])
def test_sigmoid_weights_of_strongly_negative_logits(tokens, level, kind):
    """Sigmoids too small for fp32: what they are of their sum is not."""
    x, r = _exact_logits(tokens, 64, level, kind, 17)
    bias = torch.randn(64, generator=torch.Generator().manual_seed(18))
    for k, b, renormalize in ((8, None, True), (8, bias, True), (1, None, True), (1, bias, True), (8, bias, False)):
        ids, w = nv.moe_route(x.cuda(), r.cuda(), k, "sigmoid", renormalize, None if b is None else b.cuda(), 2.5)
        torch.cuda.synchronize()
        wi, ww = _want(x, r, k, "sigmoid", renormalize, b, 2.5)
        assert np.array_equal(ids.cpu().numpy(), wi)
        # two exponentials good to 2 ulp (2^-22 each), a sum of 8 (5 roundings deep), at most four more roundings, and
        # what fp32 ends at: 2 ulp of an exponential there and three roundings, times 2.5
        assert np.all(np.abs(w.double().cpu().numpy() - ww) <= 2.0 ** -20 * ww + 1e-44)
        if k == 1 and renormalize:
            assert bool((w == 2.5).all())


@pytest.mark.parametrize("tokens", [5, 72, 130])
@pytest.mark.parametrize("neighbours", [False, True])
def test_tokens_of_zeros_choose_by_biases_closer_than_fp32_tells_apart(tokens, neighbours):
    """0.5 + bias in fp32 merges biases of some 1e-8; beside a token in doubt or not, the fp64 scores decide."""
    g = torch.Generator().manual_seed(19)
    experts = 128
    bias = 1e-8 * torch.randperm(experts, generator=g).float()
    r = torch.randn((experts, 256), generator=g).to(torch.bfloat16)
    x = torch.zeros((tokens, 256), dtype=torch.bfloat16)
    x[::3] = -0.0
    if neighbours:  # every other group of eight tokens: experts in pairs of equal logits
        r[64:] = r[:64]
        live = (torch.arange(tokens) // 8) % 2 == 1
        x[live] = torch.randn((int(live.sum()), 256), generator=g).to(torch.bfloat16)
    _check(x, r, 8, "sigmoid", True, bias)
    _check(x, r.float(), 8, "sigmoid", False, bias)
