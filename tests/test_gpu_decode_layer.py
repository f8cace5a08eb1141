"""The decode-step operators together: the example's decoder layer, captured in
a CUDA graph and replayed over growing sequences, against the same layer in
plain fp32; and the operators' failure paths, driven through the test hooks."""
import os
import sys

import pytest
import torch

import nvfp4_block_scale_gb300 as nv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_layer  # noqa: E402

pytestmark = pytest.mark.gpu
OOM, INVALID = 5, 1


# Every tensor between two operators is rounded to bf16 (2^-8 of its size at
# most, half of that on average), ten times along a layer, and the residual
# keeps the sum near its inputs: 2^-6 of the output's norm is far above what
# such roundings add up to and far below any mistake.  An E4M3 cache rounds new
# keys and values to 2^-4 of their size; they are one token among many but in
# the shortest sequence (one prompt token), where half of the attention's
# output is theirs: 2^-4 of an output that the residual dominates.
@pytest.mark.parametrize("kind,bound", [(torch.bfloat16, 2.0 ** -6), (torch.float8_e4m3fn, 2.0 ** -4)])
@pytest.mark.parametrize("shape", [(512, 1024, 8, 2, 64, 8), (1024, 2816, 8, 8, 128, 32)])
def test_decoder_layer(kind, bound, shape):
    hidden, inner, hq, hk, dim, page = shape
    worst, us = decode_layer.run(hidden, inner, hq, hk, dim, page, prompts=(300, 1, 17, 64), steps=3, kind=kind)
    assert worst <= bound and us > 0


def _small():
    w = nv.quantize(torch.randn((4096, 4096), device="cuda").to(torch.bfloat16), nv.MAX)
    cache = nv.KVCache.empty(64, 2, 16, 64)
    cache.k.normal_()
    cache.v.normal_()
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(2, 32)
    return w, cache, q, table, torch.tensor([500, 0], dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("batch", [8, 64, 200])
def test_allocation_failure_enqueues_nothing(batch):
    w, cache, q, table, n = _small()
    x = torch.randn((batch, 4096), device="cuda").to(torch.bfloat16)
    y = torch.full((batch, 4096), 7.0, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 7.0)
    for call in (lambda: nv.linear(*w, 4096, 4096, x, out=y), lambda: nv.paged_attention(cache, q, table, n, out=o)):
        assert nv.nvfp4_test_fail_allocations(1) == 0
        try:
            with pytest.raises(nv.Nvfp4Error) as e:
                call()
        finally:
            nv.nvfp4_test_fail_allocations(0)
        assert e.value.status == OOM
    torch.cuda.synchronize()
    assert bool((y == 7.0).all()) and bool((o == 7.0).all())


def test_a_workspace_too_small_is_refused():
    w, cache, q, table, n = _small()
    x = torch.randn((64, 4096), device="cuda").to(torch.bfloat16)
    for call, need in ((lambda s: nv.linear(*w, 4096, 4096, x, workspace=s), nv.linear_workspace(4096, 4096, 64)),
                       (lambda s: nv.paged_attention(cache, q, table, n, workspace=s), nv.attention_workspace(cache, 4))):
        with pytest.raises(nv.Nvfp4Error) as e:
            call(need[:-256])
        assert e.value.status == INVALID
        need.fill_(0xFF)  # whatever it holds
        assert torch.equal(call(need), call(None))


@pytest.mark.parametrize("batch", [64, 100, 200])
def test_a_wait_that_gives_up_gives_nan(batch):
    """The first bounded wait of every CTA gives up at once: outputs are NaN,
    the copies and products in flight finish, and the next call is right."""
    w, cache, q, table, n = _small()
    x = torch.randn((batch, 4096), device="cuda").to(torch.bfloat16)
    y, o = nv.linear(*w, 4096, 4096, x), nv.paged_attention(cache, q, table, n)
    try:
        assert nv.nvfp4_test_first_wait_tries(0) == 0
        bad_y, bad_o = nv.linear(*w, 4096, 4096, x), nv.paged_attention(cache, q, table, n)
        torch.cuda.synchronize()
    finally:
        nv.nvfp4_test_first_wait_tries(-1)
    assert bool(torch.isnan(bad_y).all())
    assert bool(torch.isnan(bad_o[0]).all()) and bool((bad_o[1] == 0).all())
    assert torch.equal(y, nv.linear(*w, 4096, 4096, x)) and torch.equal(o, nv.paged_attention(cache, q, table, n))
