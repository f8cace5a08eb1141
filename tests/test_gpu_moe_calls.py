"""How the mixture-of-experts layer and sampling are called: operands that lie
in other ways, slices, workspaces, streams, graphs, refusals, and a layer and a
step of them together."""
import os
import sys

import pytest
import torch

import moe_ref
import nvfp4_block_scale_gb300 as nv
from test_gpu_moe import _check, _cuda, _inputs

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
OOM, INVALID = 5, 1


def _setup(tokens=9, hidden=256, inner=128, n=6, k=3, gated=True, seed=20):
    host = moe_ref.experts(n, hidden, inner, gated, seed)
    x, ids, w, r = _inputs(tokens, hidden, n, k, seed + 1)
    return host, x, ids, w, r


def _moved(t, offset):
    """The same tensor, its bytes beginning `offset` past an allocation's."""
    flat = torch.empty(t.numel() + 64, dtype=torch.uint8, device="cuda")
    out = flat[offset:offset + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("hidden,inner", [(256, 128), (576, 320), (144, 208)])
@pytest.mark.parametrize("codes,scales", [(0, 0), (8, 0), (0, 1), (8, 3), (16, 4), (0, 2)])
def test_weights_anywhere(hidden, inner, codes, scales):
    """Codes on any 8 bytes and scales on any byte, read in whole words where they allow it."""
    host, x, ids, w, r = _setup(hidden=hidden, inner=inner)
    dev = [(_moved(m[0], codes), _moved(m[1], scales), m[2].cuda()) for m in host]
    y = nv.moe(nv.Experts(*dev), x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda())
    _check(host, x, ids, w, "silu", r, y)


def test_gate_and_up_in_one_tensor_and_experts_further_apart():
    host, x, ids, w, r = _setup()
    up, down, gate = _cuda(host)
    codes, scales = torch.cat((gate[0], up[0]), 1), torch.cat((gate[1], up[1]), 1)
    alpha = torch.stack((gate[2], up[2]), 1).contiguous()
    wide = [torch.zeros((11,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in down[:2]]
    for t, d in zip(wide, down[:2]):
        t[::2] = d
    ex = nv.Experts((codes[:, 128:], scales[:, 128:], alpha[:, 1]), (wide[0][::2], wide[1][::2], down[2]),
                    (codes[:, :128], scales[:, :128], alpha[:, 0]))
    y = nv.moe(ex, x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda())
    _check(host, x, ids, w, "silu", r, y)
    assert torch.equal(y, nv.moe(nv.Experts(up, down, gate), x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda()))


def test_rows_further_apart_and_outputs_in_place():
    host, x, ids, w, r = _setup()
    ex = nv.Experts(*_cuda(host))
    want = nv.moe(ex, x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda())
    wide = torch.full((9, 3 * 256 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    xs, rs, ys = wide[:, :256], wide[:, 264:520], wide[:, 521:777]  # (an odd output)
    xs.copy_(x)
    rs.copy_(r)
    before = wide.clone()
    assert nv.moe(ex, xs, ids.cuda(), w.cuda(), residual=rs, out=ys) is ys and torch.equal(ys, want)
    wide[:, 521:777] = before[:, 521:777]
    assert torch.equal(wide, before)
    nv.moe(ex, xs, ids.cuda(), w.cuda(), residual=rs, out=rs)
    assert torch.equal(rs, want)
    rs.copy_(r)
    nv.moe(ex, xs, ids.cuda(), w.cuda(), residual=rs, out=xs)
    assert torch.equal(xs, want)


@pytest.mark.parametrize("tokens,k", [(257, 2), (300, 8), (70, 32)])
def test_more_tokens_than_a_launch_takes(tokens, k):
    host, x, ids, w, r = _setup(tokens, 64, 48, 40, k)
    ex = nv.Experts(*_cuda(host))
    ws = nv.moe_workspace(ex, tokens, k)
    y = nv.moe(ex, x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda(), workspace=ws)
    _check(host, x, ids, w, "silu", r, y)


def test_one_expert_for_everybody():
    """256 pairs of one expert: eight jobs of the same rows."""
    host, x, ids, w, r = _setup(256, 96, 64, 3, 2)
    ids[:] = 1
    y = nv.moe(nv.Experts(*_cuda(host)), x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda())
    _check(host, x, ids, w, "silu", r, y)


def test_workspaces_may_hold_anything_and_results_repeat():
    host, x, ids, w, r = _setup(40, 512, 384, 12, 4)
    ex = nv.Experts(*_cuda(host))
    args = (ex, x.cuda(), ids.cuda(), w.cuda())
    want = nv.moe(*args)
    ws = nv.moe_workspace(ex, 64, 4)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        assert torch.equal(nv.moe(*args, workspace=ws), want)
    for _ in range(50):
        assert torch.equal(nv.moe(*args, workspace=ws), want)
    # fewer tokens in the same workspace
    assert torch.equal(nv.moe(ex, args[1][:7], args[2][:7], args[3][:7], workspace=ws),
                       nv.moe(ex, args[1][:7], args[2][:7], args[3][:7]))


def test_a_token_that_is_not_finite_stays_alone():
    host, x, ids, w, r = _setup()
    ex = nv.Experts(*_cuda(host))
    want = nv.moe(ex, x.cuda(), ids.cuda(), w.cuda(), residual=r.cuda())
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[4, 100] = bad
        got = nv.moe(ex, x2.cuda(), ids.cuda(), w.cuda(), residual=r.cuda())
        others = [i for i in range(9) if i != 4]
        assert torch.equal(got[others], want[others]) and not bool(got[4].isfinite().any())


def test_vectors_of_any_size():
    """Entries from 2^-120 to 2^100 in one batch, a token of zeros among them."""
    host, x, ids, w, _ = _setup(12, 128, 64, 4, 2)
    up, down, gate = host
    host = ((up[0], up[1], up[2] * 2.0 ** -30), (down[0], down[1], down[2] * 2.0 ** -60), (gate[0], gate[1], gate[2] * 2.0 ** -90))
    x = (x.double() * torch.tensor([2.0 ** e for e in (-120, -60, -30, -10, 0, 1, 10, 30, 60, 80, 100, 0)])[:, None]).to(torch.bfloat16)
    x[11] = 0.0
    y = nv.moe(nv.Experts(*_cuda(host)), x.cuda(), ids.cuda(), w.cuda(), activation="relu")
    _check(host, x, ids, w, "relu", None, y)
    assert bool((y[11] == 0).all())


def test_streams_graphs_and_two_calls_at_once():
    host, x, ids, w, r = _setup(33, 512, 256, 8, 2)
    ex = nv.Experts(*_cuda(host))
    router = torch.randn((8, 512), device="cuda").to(torch.bfloat16)
    xc, rc = x.cuda(), r.cuda()

    def layer(x, ws, stream=None):
        i, v = nv.moe_route(x, router, 2, stream=stream)
        return nv.moe(ex, x, i, v, residual=rc, workspace=ws, stream=stream)

    want = layer(xc, None)
    streams, spaces = [torch.cuda.Stream() for _ in range(3)], [nv.moe_workspace(ex, 33, 2) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = [layer(xc, ws, s) for s, ws in zip(streams, spaces)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(xc, spaces[0])
    other = x.flip(0).cuda()
    want2 = layer(other, None)
    for src, expected in ((x, want), (x.flip(0), want2), (x, want)):
        xc.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, expected)


def test_experts_quantized_together():
    g = torch.Generator(device="cuda").manual_seed(3)
    w = [(torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16) for s in ((5, 96, 128), (5, 128, 96), (5, 96, 128))]
    ex = nv.Experts.quantize(*w, mode=nv.FOUR_OVER_SIX)
    for m, t in zip(ex.tensors, w):
        for e in range(5):
            for a, b in zip(m, nv.quantize(t[e].contiguous(), nv.FOUR_OVER_SIX)):
                assert torch.equal(a[e].flatten(), b.flatten())
    assert (ex.experts, ex.hidden, ex.inner) == (5, 128, 96)
    plain = nv.Experts.quantize(w[0], w[1])
    assert plain.tensors[2] is None
    x, ids, wt, _ = _inputs(4, 128, 5, 2, 1)
    for e, host in ((ex, ex.tensors), (plain, plain.tensors)):
        host = [None if m is None else tuple(t.cpu() for t in m) for m in host]
        _check(host, x, ids, wt, "silu", None, nv.moe(e, x.cuda(), ids.cuda(), wt.cuda()))


def test_refusals():
    host, x, ids, w, r = _setup()
    up, down, gate = _cuda(host)
    ex = nv.Experts(up, down, gate)
    xc, ic, wc = x.cuda(), ids.cuda(), w.cuda()
    ok = nv.moe(ex, xc, ic, wc)
    assert nv.moe(ex, xc[:0], ic[:0], wc[:0]).shape == (0, 256)
    for bad in (lambda: nv.moe(ex, xc[:8], ic, wc), lambda: nv.moe(ex, xc.float(), ic, wc), lambda: nv.moe(ex, xc, ic.long(), wc),
                lambda: nv.moe(ex, xc, ic, wc.double()), lambda: nv.moe(ex, xc, ic, wc[:, :2]), lambda: nv.moe(ex, xc, ids, wc),
                lambda: nv.moe(ex, xc, ic, wc, activation="tanh"), lambda: nv.moe(ex, xc[:, :128], ic, wc),
                lambda: nv.moe(ex, xc, ic, wc, residual=r), lambda: nv.moe(ex, xc, ic, wc, out=ok.float()),
                lambda: nv.moe(ex, xc, ic, wc, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                lambda: nv.Experts(up, gate, gate), lambda: nv.Experts(up, down, down), lambda: nv.Experts(host[0], down),
                lambda: nv.Experts((up[0], up[1], up[2].double()), down), lambda: nv.Experts((up[0], up[1], up[2][:5]), down),
                lambda: nv.Experts((up[0], up[1].cpu(), up[2]), down), lambda: nv.Experts((up[0][:, ::2], up[1][:, ::2], up[2]), down),
                lambda: nv.moe_route(xc, torch.zeros((4, 128), device="cuda"), 2),
                lambda: nv.moe_route(xc, torch.zeros((4, 256), device="cuda").half(), 2),
                lambda: nv.moe_route(xc, torch.zeros((4, 256), device="cuda"), 2, "tanh"),
                lambda: nv.moe_route(xc, torch.zeros((4, 256), device="cuda"), 2, bias=torch.zeros(4, device="cuda")),
                lambda: nv.moe_route(xc, torch.zeros((4, 256), device="cuda"), 2, "sigmoid", bias=torch.zeros(5, device="cuda")),
                lambda: nv.sample(xc.half(), torch.zeros(9, device="cuda")), lambda: nv.sample(xc, torch.zeros(8, device="cuda")),
                lambda: nv.sample(xc, torch.zeros(9)), lambda: nv.sample(xc, torch.zeros(9, device="cuda"), top_k=wc[:, 0]),
                lambda: nv.sample(xc, torch.zeros(9, device="cuda"), top_p=torch.zeros(9)),
                lambda: nv.sample(xc.t(), torch.zeros(256, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.moe(ex, xc, ic, wc, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")),
                lambda: nv.moe_route(xc, torch.zeros((4, 256), device="cuda"), 5)):
        with pytest.raises(nv.Nvfp4Error) as e:
            bad()
        assert e.value.status == INVALID
    with pytest.raises(ValueError):
        nv.moe_workspace(ex, 4, 33)
    assert torch.equal(nv.moe(ex, xc, ic, wc), ok)


def test_allocation_failure_enqueues_nothing():
    host, x, ids, w, _ = _setup()
    ex = nv.Experts(*_cuda(host))
    y = torch.full((9, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    assert nv.nvfp4_test_fail_allocations(1) == 0
    try:
        with pytest.raises(nv.Nvfp4Error) as e:
            nv.moe(ex, x.cuda(), ids.cuda(), w.cuda(), out=y)
    finally:
        nv.nvfp4_test_fail_allocations(0)
    assert e.value.status == OOM
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())


def test_the_tracer_names_them():
    host, x, ids, w, _ = _setup()
    ex = nv.Experts(*_cuda(host))
    args = (x.cuda(), ids.cuda(), w.cuda())
    nv.nvfp4_profiler_reset()
    nv.nvfp4_profiler_enable(1)
    try:
        nv.moe(ex, *args)
        nv.moe_route(args[0], torch.randn((6, 256), device="cuda"), 2)
        nv.sample(args[0], torch.rand(9, device="cuda"))
    finally:
        nv.nvfp4_profiler_enable(0)
    names = nv.profiler_report()
    nv.nvfp4_profiler_reset()
    assert all(names[n][0] == 1 for n in ("k_moe", "k_moe_route", "k_sample"))


def test_outputs_of_a_stream_are_its_own():
    """As for the other operators: memory that the current stream gave up and
    still writes is not what a call on another stream gets."""
    host, x, ids, w, _ = _setup()
    ex = nv.Experts(*_cuda(host))
    xc, ic, wc = x.cuda(), ids.cuda(), w.cuda()
    router, u = torch.randn((6, 256), device="cuda").to(torch.bfloat16), torch.rand(9, device="cuda")
    calls = (lambda s: [nv.moe(ex, xc, ic, wc, stream=s)], lambda s: nv.moe_route(xc, router, 2, stream=s),
             lambda s: nv.sample(xc, u, return_logprob=True, stream=s))
    for call in calls:
        want = [t.clone() for t in call(None)]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        freed = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(2_000_000)
        for t in freed:
            t.fill_(1)
        del freed, t
        got = call(s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("shape", [(256, 128, 8, 2), (512, 384, 24, 6)])
def test_a_step_of_them_together(shape):
    import moe_layer
    hidden, inner, experts, k = shape
    worst, tokens, want, us = moe_layer.run(hidden, inner, experts, k, vocabulary=3001, batch=7, steps=3)
    # every tensor between two operators is rounded to bf16, as in the decoder layer's test; the tokens follow from the
    # logits that the plain layer gets too, but for those roundings: see moe_layer.run
    assert worst <= 2.0 ** -6 and tokens == want and us > 0


def test_clusters_of_eight():
    """As on a device that places none of sixteen: the same tokens and experts, and weights within what a sum's order moves."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((3, 2048), generator=g, device="cuda").to(torch.bfloat16)
    router = 0.03 * torch.randn((128, 2048), generator=g, device="cuda")
    u = torch.rand(3, generator=g, device="cuda")
    logits = [(2.5 * torch.randn((3, v), generator=g, device="cuda")).to(kind) for v in (32000, 262144, 1 << 20)
              for kind in (torch.bfloat16, torch.float32)]
    settings = (dict(), dict(top_k=40), dict(top_k=2000, top_p=0.9), dict(top_p=0.9, temperature=1.5), dict(min_p=0.05))

    def calls():
        routed = [nv.moe_route(x, r, 8, s) for r in (router, router.to(torch.bfloat16)) for s in ("softmax", "sigmoid")]
        return routed, [nv.sample(t, u, return_logprob=True, **s) for t in logits for s in settings]

    routed, sampled = calls()
    assert nv.nvfp4_test_small_clusters(1) == 0
    try:
        routed8, sampled8 = calls()
    finally:
        nv.nvfp4_test_small_clusters(0)
    for a, b in zip(sampled, sampled8):  # (sums of whole numbers)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for (i, w), (i8, w8) in zip(routed, routed8):
        # logits to 2^-46 of |x| |r| (at most 2^7) become weights with the same few fp32 roundings
        assert torch.equal(i, i8) and bool(((w - w8).abs() <= 2.0 ** -20 * w).all())
