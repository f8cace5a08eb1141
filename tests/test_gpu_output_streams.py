"""Outputs that a call on an explicit stream makes: their memory comes from
that stream, so nothing that still runs on the current one can hold it."""
import pytest
import torch

import nvfp4_block_scale_gb300 as nv
import synthetic
from gpu_util import to_device

pytestmark = pytest.mark.gpu


def _calls():
    """{name: call on a stream -> outputs}, every operand made beforehand."""
    rows, cols = 256, 1024
    w = to_device(synthetic.gaussian(rows, cols, 0.02, 900))
    q = nv.quantize(w)
    x = to_device(synthetic.gaussian(6, cols, 1.0, 901))
    v = torch.randn(4096, device="cuda")
    cache = nv.KVCache.empty(8, 2, 16, 64)
    cache.k.normal_()
    cache.v.normal_()
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    qkv = torch.randn((3, 8 * 64), device="cuda").to(torch.bfloat16)
    heads = torch.randn((3, 4, 64), device="cuda").to(torch.bfloat16)
    seq, pos, table, n = i([0, 1, 2]), i([20, 3, 40]), i([[1, 2, 3], [4, 4, 4], [5, 6, 7]]), i([20, 0, 40])
    return {
        "quantize": lambda s: nv.quantize(w, nv.FOUR_OVER_SIX, stream=s),
        "quantize_grouped": lambda s: [t for o in nv.quantize_grouped([w, w[:128]], nv.MAX, stream=s) for t in o],
        "dequantize": lambda s: [nv.dequantize(*q, rows, cols, stream=s)],
        "gemv": lambda s: [nv.gemv(*q, rows, cols, x, stream=s)],
        "gemm": lambda s: [nv.gemm(*q, rows, cols, x, stream=s)],
        "linear": lambda s: [nv.linear(*q, rows, cols, x, stream=s)],
        "kv_append": lambda s: [nv.kv_append(cache, qkv, 4, seq, pos, table, stream=s)],
        "paged_attention": lambda s: nv.paged_attention(cache, heads, table, n, return_lse=True, stream=s),
        "swizzle_scales": lambda s: [nv.swizzle_scales(q[1], rows, cols, stream=s)],
        "encode_e2m1": lambda s: [nv.encode_e2m1(v, stream=s)],
        "encode_e4m3": lambda s: [nv.encode_e4m3(v, stream=s)],
    }


NAMES = ["quantize", "quantize_grouped", "dequantize", "gemv", "gemm", "linear", "kv_append", "paged_attention",
         "swizzle_scales", "encode_e2m1", "encode_e4m3"]


def _pool_stream(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


@pytest.mark.parametrize("name", NAMES)
def test_memory_comes_from_the_calls_own_stream(name):
    call, side = _calls()[name], torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = call(side)
    torch.cuda.synchronize()
    assert [_pool_stream(t) for t in outs] == [side.cuda_stream] * len(outs)


@pytest.mark.parametrize("name", NAMES)
def test_work_pending_on_the_current_stream_leaves_outputs_alone(name):
    """The current stream gives up tensors of the outputs' sizes that a kernel
    of its own, still pending, writes."""
    call, side = _calls()[name], torch.cuda.Stream()
    torch.cuda.synchronize()
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    held = [torch.empty_like(t) for t in want for _ in range(3)]
    torch.cuda._sleep(50_000_000)
    for t in held:
        t.view(torch.uint8).fill_(0x55)
    del held, t
    outs = call(side)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
