"""nvfp4_linear, the W4A16 product with its epilogue, against the same in 64
bits.  Every output has to lie within the derived bound of decode_ref.linear."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import nvfp4_block_scale_gb300 as nv
import synthetic
from gpu_util import to_device

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, std=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((std * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16).cuda()


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _weights(rows, cols, seed, mode=None):
    w = synthetic.student_t(rows, cols, 4.0, 0.02, seed)
    return nv.quantize(to_device(w), nv.FOUR_OVER_SIX if mode is None else mode)


def _check(y, w, x, **ep):
    c, s, a = w
    host = {k: _f64(v) if isinstance(v, torch.Tensor) else v for k, v in ep.items()}
    v, bound = ref.linear(c.cpu().numpy(), s.cpu().numpy(), a.item(), _f64(x), **host)
    got = _f64(y)
    assert y.dtype == torch.bfloat16 and np.all(np.isfinite(got))
    assert ref.within(got, v, bound)


SHAPES = [(1, 16, 1), (3, 48, 2), (16, 256, 1), (17, 272, 9), (128, 128, 8), (129, 1040, 16), (300, 2064, 17),
          (1000, 512, 33), (64, 4096, 64), (257, 1536, 100), (130, 28672, 5), (96, 640, 256), (5000, 64, 3),
          (2048, 4096, 24)]


@pytest.mark.parametrize("rows,cols,batch", SHAPES)
def test_product_alone(rows, cols, batch):
    w, x = _weights(rows, cols, rows + cols), _bf16((batch, cols), batch)
    _check(nv.linear(*w, rows, cols, x), w, x)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("batch", [1, 7, 40])
def test_whole_epilogue(act, batch):
    rows, cols = 208, 1040
    w, x = _weights(rows, cols, 7), _bf16((batch, cols), 8, 2.0)
    ep = dict(bias=_bf16((rows,), 9), gate=_bf16((batch, rows), 10), residual=_bf16((batch, rows), 11))
    _check(nv.linear(*w, rows, cols, x, activation=act, **ep), w, x, act=act, **ep)


@pytest.mark.parametrize("mode", [nv.MAX, nv.CJSO])
def test_every_part_alone_and_repeats(mode):
    rows, cols, batch = 160, 512, 12
    w, x = _weights(rows, cols, 20, mode), _bf16((batch, cols), 21)
    for ep in (dict(bias=_bf16((rows,), 22)), dict(gate=_bf16((batch, rows), 23)),
               dict(residual=_bf16((batch, rows), 24))):
        y = nv.linear(*w, rows, cols, x, **ep)
        _check(y, w, x, **ep)
        assert torch.equal(y, nv.linear(*w, rows, cols, x, **ep))


@pytest.mark.parametrize("batch", [3, 20, 80])
def test_strided_rows_and_residual_in_place(batch):
    rows, cols = 120, 528
    w = _weights(rows, cols, 30)
    wide = _bf16((batch, 2 * cols + 8), 31)
    x = wide[:, 8:8 + cols]  # 16-byte aligned, rows further apart
    both = _bf16((batch, 2 * rows + 1), 32)  # odd stride: 2-byte alignment only
    gate, res = both[:, 1:1 + rows], both[:, 1 + rows:]
    keep = both.clone()
    y = nv.linear(*w, rows, cols, x, gate=gate, residual=res, out=res)
    assert y.data_ptr() == res.data_ptr()
    _check(y, w, x, gate=keep[:, 1:1 + rows], residual=keep[:, 1 + rows:])
    assert torch.equal(both[:, :1 + rows], keep[:, :1 + rows])


@pytest.mark.parametrize("batch", [1, 12, 64])
def test_codes_and_scales_off_their_natural_alignment(batch):
    rows, cols = 130, 2048
    c, s, a = _weights(rows, cols, 40)
    cb, sb = torch.zeros(c.numel() + 16, dtype=torch.uint8, device="cuda"), torch.zeros(s.numel() + 16, dtype=torch.uint8, device="cuda")
    c8, s1 = cb[8:8 + c.numel()].view_as(c), sb[1:1 + s.numel()].view_as(s)
    c8.copy_(c)
    s1.copy_(s)
    x = _bf16((batch, cols), 41)
    _check(nv.linear(c8, s1, a, rows, cols, x), (c, s, a), x)


@pytest.mark.parametrize("rows,cols", [(301, 32), (301, 96), (130, 160), (301, 416), (129, 1056), (301, 2112), (200, 4224),
                                       (70, 9632), (20500, 288), (39000, 32), (20500, 1056)])
@pytest.mark.parametrize("batch,offset", [(24, 0), (33, 1), (70, 8), (130, 3)])
def test_rows_of_scales_of_any_length(rows, cols, batch, offset):
    """Rows of scales that begin at any byte, partial last steps, tiles shared
    and whole; NaN bytes on both sides of the scales, where nothing may look."""
    w, x = _weights(rows, cols, rows + cols + offset), _bf16((batch, cols), batch)
    n = rows * cols // 16
    around = torch.full((offset + n + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    around[offset:offset + n] = w[1].view(torch.uint8).flatten()
    w = (w[0], around[offset:offset + n].view(rows, cols // 16), w[2])
    bias = _bf16((rows,), 5)
    y = nv.linear(*w, rows, cols, x, bias=bias)
    _check(y, w, x, bias=bias)
    assert torch.equal(y, nv.linear(*w, rows, cols, x, bias=bias))


def test_more_vectors_than_one_slice():
    rows, cols, batch = 136, 256, 600
    w, x, res = _weights(rows, cols, 50), _bf16((batch, cols), 51), _bf16((batch, rows), 52)
    ws = nv.linear_workspace(rows, cols, batch)
    _check(nv.linear(*w, rows, cols, x, residual=res, workspace=ws), w, x, residual=res)


def test_extreme_vectors_and_zero_weights():
    """Vectors of very different sizes side by side (each is bounded by its own
    entries), a zero vector, entries far below their vector's largest, and
    weights of whole zero blocks."""
    rows, cols = 144, 1024
    w = synthetic.bits_to_f32(synthetic.gaussian(rows, cols, 0.02, 60))
    w[:, 256:512] = 0.0
    w[7] = 0.0
    c, s, a = nv.quantize(to_device(synthetic.to_bf16_bits(w)), nv.MAX)
    for batch in (5, 24):
        x = _bf16((batch, cols), 61)
        x[0] *= 2.0 ** 60
        x[1] *= 2.0 ** -70
        x[2] = 0.0
        x[3, ::7] *= 2.0 ** 20
        x[4, 5] = 3.0e4
        _check(nv.linear(c, s, a, rows, cols, x), (c, s, a), x)


def test_no_columns_no_vectors_no_rows():
    e = torch.empty(0, dtype=torch.uint8, device="cuda")
    a = torch.zeros(1, device="cuda")
    bias, res = _bf16((24,), 70), _bf16((3, 24), 71)
    y = nv.linear(e, e, a, 24, 0, torch.empty((3, 0), dtype=torch.bfloat16, device="cuda"), bias=bias,
                  activation="relu", residual=res)
    want = (torch.relu(bias.float()) + res.float()).to(torch.bfloat16)
    assert torch.equal(y, want)
    w = _weights(16, 32, 72)
    assert nv.linear(*w, 16, 32, torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")).shape == (0, 16)
    assert nv.linear(e, e, a, 0, 32, _bf16((4, 32), 73)).shape == (4, 0)


def test_workspace_serves_calls_of_several_shapes_and_capture():
    big = nv.linear_workspace(1024, 4096, 64)
    cases = [(1024, 4096, 64), (512, 4096, 1), (1024, 1024, 20), (130, 2064, 8)]
    side = torch.cuda.Stream()
    plain = []
    for rows, cols, batch in cases:
        w, x = _weights(rows, cols, 80 + batch), _bf16((batch, cols), 81)
        need = nv.nvfp4_linear_workspace_bytes(rows, cols, batch)
        ws = big if need <= big.numel() else nv.linear_workspace(rows, cols, batch)
        y = nv.linear(*w, rows, cols, x)
        side.wait_stream(torch.cuda.current_stream())
        z = [nv.linear(*w, rows, cols, x, workspace=ws, stream=side) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(y, t) for t in z)
        plain.append((w, x, ws, y))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [nv.linear(*w, rows, cols, x, workspace=ws)
                for (rows, cols, batch), (w, x, ws, _) in zip(cases, plain)] + \
               [nv.linear(*w, rows, cols, x) for (rows, cols, batch), (w, x, _, _) in zip(cases, plain)]
    for o in outs:
        o.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, p[3]) for o, p in zip(outs, plain + plain))


@pytest.mark.parametrize("rows,cols,largest", [(1024, 4096, 64), (2048, 2048, 32), (1024, 28672, 64), (4096, 1024, 20),
                                               (300, 2064, 300), (8192, 8192, 129), (28672, 8192, 256)])
def test_a_workspace_for_the_largest_batch_serves_every_smaller_one(rows, cols, largest):
    space = nv.linear_workspace(rows, cols, largest)
    w = _weights(rows, cols, 90)
    x = _bf16((largest, cols), 91)
    need = [nv.nvfp4_linear_workspace_bytes(rows, cols, b) for b in range(largest + 1)]
    assert need == sorted(need) and need[-1] <= space.numel()
    for batch in range(1, largest + 1):
        y = nv.linear(*w, rows, cols, x[:batch], workspace=space)
        if batch in (1, 9, 17, largest // 2, largest):
            assert torch.equal(y, nv.linear(*w, rows, cols, x[:batch]))


WRONG_TYPES = {
    "fp64 alpha": lambda c, s, a: (c, s, a.double()),
    "16-bit alpha": lambda c, s, a: (c, s, a.half()),
    "no alpha": lambda c, s, a: (c, s, a[:0]),
    "wide codes": lambda c, s, a: (c.int(), s, a),
    "fp32 scales": lambda c, s, a: (c, s.view(torch.float8_e4m3fn).float(), a),
}
ON_THE_HOST = {
    "codes": lambda c, s, a: (c.cpu(), s, a),
    "scales": lambda c, s, a: (c, s.cpu(), a),
    "alpha": lambda c, s, a: (c, s, a.cpu()),
}


@pytest.mark.parametrize("case", [*WRONG_TYPES, *ON_THE_HOST])
def test_weights_of_another_type_or_on_the_host_are_refused(case):
    w, x = _weights(32, 64, 92), _bf16((3, 64), 93)
    with pytest.raises(ValueError):
        nv.linear(*(WRONG_TYPES | ON_THE_HOST)[case](*w), 32, 64, x)


def test_weights_under_other_names_for_bytes_are_taken():
    (c, s, a), x = _weights(32, 64, 94), _bf16((3, 64), 95)
    y = nv.linear(c, s, a, 32, 64, x)
    assert torch.equal(y, nv.linear(c.flatten().view(torch.int8), s.view(torch.float8_e4m3fn), a[0], 32, 64, x))


def test_a_workspace_on_the_host_is_refused():
    w, x = _weights(32, 64, 96), _bf16((3, 64), 97)
    with pytest.raises(ValueError):
        nv.linear(*w, 32, 64, x, workspace=torch.empty(1 << 20, dtype=torch.uint8))
