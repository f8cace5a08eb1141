"""nvfp4_linear on tensors that the tcgen05 product takes: its f16 half (up to
128 vectors of large tensors) and its bf16 half, whole and shared tiles, codes
by TMA and by the producers, against 64 bits on a sample of the rows.  Each case
names the kernel that has to run it, as the tracer reports it."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import nvfp4_block_scale_gb300 as nv

pytestmark = pytest.mark.gpu
F16, BF16 = "k_linear_tc<f16>", "k_linear_tc<bf16>"


def _randn(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g).to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _bound(wm, alpha, x, f16, bias, act, gate, residual):
    """Products of q * Delta (six bits) and x (eight) are exact; fp32 sums of n
    terms in any order, on the tensor cores, are off by 2 (n + 2) 2^-24 sum
    |w x|.  In f16 an entry of x, scaled so that its vector's largest is at
    least 2^13, is off by half of the smallest step, 2^-25: 2^-38 of the
    largest.  Then the epilogue as in decode_ref.linear: no activation steeper
    than 1.13, its functions and the roundings around it within 2^-20 of their
    operands, and 2^-22 of the result and the residual."""
    mag = alpha * (np.abs(x) @ np.abs(wm).T)
    err = 2 * (wm.shape[1] + 2) * 2.0 ** -24 * mag
    if f16:
        err = err + alpha * 2.0 ** -38 * np.abs(x).max(1)[:, None] * np.abs(wm).sum(1)[None, :]
    v = alpha * (x @ wm.T)
    big = np.abs(v) + (0.0 if bias is None else np.abs(bias))
    v = v if bias is None else v + bias
    v, err = ref.activation(v, act), 1.13 * err + 2.0 ** -20 * big
    if gate is not None:
        v, err = v * gate, err * np.abs(gate)
    v = v if residual is None else v + residual
    return v, err + 2.0 ** -22 * (np.abs(v) + (0.0 if residual is None else np.abs(residual)))


def _check(kernel, w, rows, cols, x, act="none", bias=None, gate=None, residual=None):
    c, s, a = w
    nv.nvfp4_profiler_reset()
    nv.nvfp4_profiler_enable(1)
    try:
        y = nv.linear(c, s, a, rows, cols, x, bias, act, gate, residual)
        torch.cuda.synchronize()
        assert set(nv.profiler_report()) == {kernel}
    finally:
        nv.nvfp4_profiler_enable(0)
        nv.nvfp4_profiler_reset()
    g = np.random.default_rng(rows + x.shape[0])
    at = np.unique(np.concatenate((np.arange(min(rows, 20)), np.arange(max(0, rows - 20), rows), g.integers(0, rows, 260))))
    i = torch.from_numpy(at).cuda()
    wm = ref.weights(c.view(rows, -1)[i].cpu().numpy(), s.view(rows, -1)[i].cpu().numpy())
    pick = lambda t: None if t is None else _f64(t[..., i])  # noqa: E731
    v, err = _bound(wm, a.item(), _f64(x), kernel == F16, pick(bias), act, pick(gate), pick(residual))
    got = pick(y)
    assert bool(torch.isfinite(y.float()).all())
    assert ref.within(got, v, err)
    assert torch.equal(y, nv.linear(c, s, a, rows, cols, x, bias, act, gate, residual))


def _weights(rows, cols, seed):
    return nv.quantize(_randn((rows, cols), seed, 0.02), nv.FOUR_OVER_SIX)


@pytest.mark.parametrize("rows,cols,batches,kernel", [
    (8192, 8192, (1, 8, 9, 16, 17, 24, 64, 65, 100, 128), F16),
    (8192, 8208, (24, 100), F16),       # rows of codes that are odd multiples of 8 bytes
    (8191, 8224, (33, 128), F16),       # of 16 bytes, scales of no power of two
    (20500, 4096, (24, 70), F16),       # whole and shared tiles on every CTA
    (40000, 2048, (20, 128), F16),      # two whole tiles a CTA, fewer shared steps than CTAs
    (40000, 2064, (20, 128), F16),
    (130, 262144, (40, 127), F16),      # entries of x behind those that stay in registers; one tile over many CTAs
    (20500, 2048, (24, 130), BF16),
    (28700, 8192, (130, 256), BF16),
])
def test_large_products(rows, cols, batches, kernel):
    w = _weights(rows, cols, rows + cols)
    bias = _randn((rows,), 3)
    for batch in batches:
        x = _randn((batch, cols), batch)
        _check(kernel, w, rows, cols, x)
        _check(kernel, w, rows, cols, x, act="silu", bias=bias, gate=_randn((batch, rows), 4), residual=_randn((batch, rows), 5))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("pad", [0, 3])
def test_epilogue_over_strided_rows(act, pad):
    """Rows of 16-byte multiples and odd ones; the residual updated in place."""
    rows, cols, batch = 8192, 8192, 29
    w, x = _weights(rows, cols, 7), _randn((batch, 2 * cols), 8)[:, cols:]
    gate, res = (_randn((batch, rows + pad), s)[:, :rows] for s in (9, 10))
    keep, ep = res.clone(), dict(bias=_randn((rows,), 11), act=act, gate=gate)
    _check(F16, w, rows, cols, x, residual=keep, **ep)
    want = nv.linear(*w, rows, cols, x, ep["bias"], act, gate, keep)
    got = nv.linear(*w, rows, cols, x, ep["bias"], act, gate, res, out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("rows,cols,batch", [(8192, 8192, 24), (8192, 8208, 100), (130, 262144, 40)])
def test_vectors_of_very_different_sizes(rows, cols, batch):
    """Each vector keeps its own precision: huge, tiny and zero ones side by
    side, entries far below their vector's largest, and a largest entry that
    meets zero weights only, so that the others decide the result."""
    w = _randn((rows, cols), 12, 0.02)
    w[:, 512:1024] = 0.0
    w[rows // 2] = 0.0
    q = nv.quantize(w, nv.MAX)
    x = _randn((batch, cols), 13)
    x[0] *= 2.0 ** 60
    x[1] *= 2.0 ** -70
    x[2] = 0.0
    x[3, ::7] *= 2.0 ** 20
    x[4, 700] = 2.0 ** 20
    x[5, 1023] = -2.0 ** 24
    x[6] *= 2.0 ** 100
    x[7] *= 2.0 ** -110
    x[8, 600] = 2.0 ** 90
    x[9, 1:] = 0.0
    x[10] = 0.0
    x[10, cols - 1] = 1.0
    _check(F16, q, rows, cols, x, residual=torch.zeros((batch, rows), dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("batch", [24, 100])
def test_capture_and_streams(batch):
    """The conversion of x and the product behind it, in one graph with other
    calls around them: each product waits for its own vectors."""
    rows, cols = 8192, 8192
    w, xs = _weights(rows, cols, 14), [_randn((batch, cols), 15 + i) for i in range(3)]
    want = [nv.linear(*w, rows, cols, x) for x in xs]
    x, y = torch.empty_like(xs[0]), torch.empty_like(want[0])
    space = nv.linear_workspace(rows, cols, batch)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = []
        for v in xs:
            x.copy_(v)
            nv.linear(*w, rows, cols, x, out=y, workspace=space)
            got.append(y.clone())
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("batch", [24, 100])
def test_a_wait_that_gives_up_gives_nan(batch):
    rows, cols = 8192, 8192
    w, x = _weights(rows, cols, 18), _randn((batch, cols), 19)
    want = nv.linear(*w, rows, cols, x)
    torch.cuda.synchronize()
    try:
        assert nv.nvfp4_test_first_wait_tries(0) == 0
        bad = nv.linear(*w, rows, cols, x)
        torch.cuda.synchronize()
    finally:
        nv.nvfp4_test_first_wait_tries(-1)
    assert bool(torch.isnan(bad).all())
    assert torch.equal(want, nv.linear(*w, rows, cols, x))
