"""Sampling against its definition in 64 bits: the tokens have to be equal."""
import pytest
import torch

import nvfp4_block_scale_gb300 as nv
import sample_ref

pytestmark = pytest.mark.gpu
INF = float("inf")

# The library's weights are off by 2^-30 of themselves or 2^-42, so its sums by as
# much of the row's mass; a decision may differ where a sum lies nearer to its
# goal than that.  (Seeded inputs lie further away; the test says so.)
NEAR = 2.0 ** -28


def _check(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """x [rows, vocabulary] and u [rows] on the host; settings numbers or host tensors [rows]."""
    settings = dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in settings.items()}
    token, logprob = nv.sample(x.cuda(), u.cuda(), return_logprob=True, **dev)
    torch.cuda.synchronize()
    one = lambda v, i: float(v[i]) if isinstance(v, torch.Tensor) else float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    xs = x.double().numpy()
    for i in range(x.shape[0]):
        want, lp, margin = sample_ref.sample(xs[i], float(u[i]), one(temperature, i), int(one(top_k, i)), one(top_p, i),
                                             one(min_p, i))
        assert margin > NEAR or margin == 0.0, "an input on the edge of a decision"
        assert int(token[i]) == want, (i, int(token[i]), want, margin)
        got = float(logprob[i])
        # the sum's 2^-28, the result's rounding, and that of (l - m) / T in 64 bits
        assert got == lp or abs(got - lp) <= 2.0 ** -28 + 2.0 ** -23 * abs(lp)
    return token


def test_a_top_k_past_32_bits_keeps_all():
    x, u = torch.zeros((1, 100)), torch.tensor([0.995])
    for k in (100, 2 ** 31, 2 ** 32 + 5, -2 ** 40):
        assert nv.sample(x.cuda(), u.cuda(), top_k=k).tolist() == [99]


def _logits(rows, vocabulary, kind, seed, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((rows, vocabulary), generator=g)).to(kind), torch.rand(rows, generator=g)


# one CTA and clusters; runs of one token; odd sizes (rows begin anywhere); more than a CTA keeps in shared memory
VOCABULARIES = [1, 2, 7, 513, 1000, 4097, 32000, 50257, 131072]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocabulary", VOCABULARIES)
def test_filters(vocabulary, kind):
    rows = 24
    x, u = _logits(rows, vocabulary, kind, vocabulary)
    for s in (dict(), dict(top_k=1), dict(top_k=5), dict(top_k=200), dict(top_p=0.9), dict(top_p=0.05), dict(top_k=40, top_p=0.8),
              dict(min_p=0.1), dict(temperature=0.3, top_k=100, top_p=0.95, min_p=0.02), dict(temperature=3.0, top_p=0.99),
              dict(temperature=0.0), dict(top_k=vocabulary, top_p=1.5, min_p=-1.0)):
        _check(x, u, **s)


def test_settings_by_row():
    rows, v = 40, 3000
    x, u = _logits(rows, v, torch.bfloat16, 1)
    g = torch.Generator().manual_seed(2)
    t = torch.rand(rows, generator=g) * 2
    t[::5] = 0.0
    k = torch.randint(-2, 60, (rows,), generator=g, dtype=torch.int32)
    _check(x, u, t, k, 0.5 + torch.rand(rows, generator=g), torch.rand(rows, generator=g) * 0.1)
    bad = float("nan")
    _check(x, u, torch.tensor([bad, -1.0, 1e-30, 1e30, 1.0] * 8))
    _check(x[:5], u[:5], top_p=torch.tensor([bad, 0.0, -1.0, 1e-30, 2.0]))
    _check(x[:5], u[:5], min_p=torch.tensor([bad, 0.0, 1.0, 7.0, 1e-30]))


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocabulary", [5, 700, 9001, 40000])
def test_masks(vocabulary, kind):
    rows = 30
    x, u = _logits(rows, vocabulary, kind, 3)
    g = torch.Generator().manual_seed(4)
    x[torch.rand((rows, vocabulary), generator=g) < 0.9] = -INF
    x[0] = -INF                      # nothing left
    x[1] = float("nan")
    x[2] = -INF
    x[2, vocabulary - 1] = -3.0      # one left
    x[3] = torch.finfo(kind).min     # a mask of the type's lowest value, everywhere and almost
    x[4] = torch.finfo(kind).min
    x[4, vocabulary // 2] = torch.finfo(kind).min / 2
    x[5, 1:3] = float("nan")
    x[6, 1], x[6, 3] = INF, INF
    x[7] = 0.0
    x[8] = -0.0
    x[8, ::2] = 0.0
    x[9] = torch.finfo(kind).max
    for s in (dict(), dict(top_k=3), dict(top_p=0.7), dict(top_k=50, top_p=0.5, min_p=0.01), dict(temperature=0.0)):
        token = _check(x, u, **s)
        assert token[0] == -1 and token[1] == -1 and token[2] == vocabulary - 1


def test_many_equal_logits():
    """Cuts inside runs of equal values go by index: bins that hold far more tokens than a CTA ranks."""
    v = 60000
    g = torch.Generator().manual_seed(5)
    x = torch.randint(0, 3, (8, v), generator=g).float()
    x[0] = 1.0
    u = torch.rand(8, generator=g)
    for kind in (torch.bfloat16, torch.float32):
        for s in (dict(top_k=1), dict(top_k=777), dict(top_k=59999), dict(top_k=25000, top_p=0.31), dict(top_p=0.5), dict()):
            _check(x.to(kind), u, **s)
    # values that one bin cannot tell apart, many of them
    x = 5.0 + 1e-5 * torch.rand((4, v), generator=g)
    _check(x, u[:4], top_k=12345)
    _check(x, u[:4], top_k=30000, top_p=0.4)


def test_ends_of_the_random_number():
    x, _ = _logits(6, 5000, torch.float32, 6)
    x[:, 0], x[:, -1] = -INF, -INF
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, 5.0, -1.0, float("nan")])
    token = nv.sample(x.cuda(), u.cuda()).cpu().tolist()
    assert token[0] == token[4] == token[5] == 1 and token[1] >= 4990 and token[3] >= 4990
    assert token[1:3] == [sample_ref.sample(x[i].double().numpy(), float(u[i]))[0] for i in (1, 2)]


def test_frequencies():
    """Every number of a fine grid: each token's share of them is its probability's, within two steps of the grid."""
    n = 4096
    x = torch.tensor([1.0, -INF, 0.5, 3.0, 2.0, -1.0])
    u = (torch.arange(n) + 0.5) / n
    token = nv.sample(x.repeat(n, 1).cuda(), u.cuda(), temperature=0.7).cpu().long()
    p = torch.softmax(x.double() / 0.7, 0)
    assert bool(((torch.bincount(token, minlength=6) / n - p).abs() <= 2 / n).all())


def test_strides_streams_graphs_and_many_rows():
    x, u = _logits(700, 1003, torch.bfloat16, 7)
    wide = torch.full((700, 1100), INF, dtype=torch.bfloat16)
    wide[:, 31:31 + 1003] = x
    xc, uc, wc = x.cuda(), u.cuda(), wide.cuda()[:, 31:31 + 1003]
    a = nv.sample(xc, uc, top_k=30, top_p=0.9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = nv.sample(wc, uc, top_k=30, top_p=0.9, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = nv.sample(xc, uc, top_k=30, top_p=0.9)
    xc.copy_(x.flip(0))
    uc.copy_(u.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.flip(0), c)
    assert nv.sample(xc[:0], uc[:0]).shape == (0,)
    assert nv.sample(xc[:, :0], uc).cpu().tolist() == [-1] * 700


def test_largest_vocabulary():
    x, u = _logits(2, 1 << 20, torch.float32, 8)
    for s in (dict(), dict(top_p=0.9), dict(top_k=1000, top_p=0.99)):
        _check(x, u, **s)
    with pytest.raises(nv.Nvfp4Error):
        nv.sample(torch.zeros((1, (1 << 20) + 1), device="cuda"), u[:1].cuda())


def test_cuts_at_the_end_of_a_range():
    """A cut among the last tokens of a range that is split again, tokens of the next range right behind them.  Values two
    steps of fp32 apart: a range of the exponent is 83300 of them wide, a finer one 64."""
    v, rows = 120000, 34
    g = torch.Generator().manual_seed(11)
    line = 1.0 - 2.0 ** -23 * torch.arange(v, dtype=torch.float64)
    x = torch.stack([line[torch.randperm(v, generator=g)] for _ in range(rows)]).float()
    u = torch.rand(rows, generator=g)
    edge = int((22 / (0.75 * 2048 * 1.4426950408889634)) * 2.0 ** 23)
    k = edge - 132 + 8 * torch.arange(rows, dtype=torch.int32)
    _check(x, u, top_k=k)
    w = torch.exp(line - 1.0)
    _check(x, u, top_p=((w.cumsum(0) - 0.5 * w)[k.long() - 1] / w.sum()).float())  # (half a token before the k-th's end)


def test_top_p_of_a_large_top_k_of_nearly_equal_weights():
    """Every weight is 1 in 42 bits, so the cuts go by count: 5795 tokens, then 5216 of them."""
    g = torch.Generator().manual_seed(447325616)
    x = 0.5 * torch.randn((7, 64418), generator=g)
    x[torch.rand(x.shape, generator=g) < 0.1] = -INF
    u = torch.rand(7, generator=g)
    for _ in range(3):
        _check(x.to(torch.bfloat16), u, temperature=1e30, top_k=5795, top_p=0.9)
