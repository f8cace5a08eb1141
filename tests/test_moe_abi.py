"""The entry points of the mixture-of-experts layer and of sampling on the
host: what they refuse, with which status, before touching the device."""
import ctypes
import os
import re

import pytest
import torch

import nvfp4_block_scale_gb300 as nv

INVALID, MISALIGNED = 1, 2
A = 0x100000  # fake, aligned device address: never dereferenced on these paths


def _matrix(**kw):
    d = dict(codes=A, scales=A, alpha=A, code_stride=32 * 64 // 2, scale_stride=32 * 4, alpha_stride=1)
    d.update(kw)
    return nv.nvfp4_expert_matrix(*d.values())


def _experts(**kw):
    d = dict(gate=_matrix(), up=_matrix(), down=_matrix(), hidden=64, inner=32, experts=4)
    d.update(kw)
    return nv.nvfp4_experts(*d.values())


def _moe(**kw):
    d = dict(experts=_experts(), x=A, x_stride=64, tokens=3, top_k=2, ids=A, weights=A, activation=nv.ACT_SILU, residual=None,
             residual_stride=0, y=A, y_stride=64, workspace=None, workspace_bytes=0, stream=None)
    d.update(kw)
    return nv.nvfp4_moe(*d.values())


BAD_EXPERTS = [dict(hidden=0), dict(hidden=24), dict(inner=0), dict(inner=40), dict(inner=-16), dict(experts=0),
               dict(experts=1025), dict(up=_matrix(codes=None)), dict(down=_matrix(codes=None)), dict(up=_matrix(scales=None)),
               dict(down=_matrix(alpha=None)), dict(gate=_matrix(scales=None)), dict(up=_matrix(code_stride=-8)),
               dict(gate=_matrix(scale_stride=-1)), dict(down=_matrix(alpha_stride=1 << 41)), dict(hidden=1 << 20),
               dict(inner=1 << 20)]
ODD_EXPERTS = [dict(up=_matrix(codes=A + 4)), dict(gate=_matrix(codes=A + 2)), dict(down=_matrix(alpha=A + 2)),
               dict(up=_matrix(code_stride=36))]


@pytest.mark.parametrize("kw", BAD_EXPERTS)
def test_bad_experts(kw):
    assert _moe(experts=_experts(**kw), x_stride=1 << 20, y_stride=1 << 20) == INVALID
    assert nv.nvfp4_moe_workspace_bytes(_experts(**kw), 3, 2) == -1


@pytest.mark.parametrize("kw", ODD_EXPERTS)
def test_misaligned_experts(kw):
    assert _moe(experts=_experts(**kw)) == MISALIGNED


@pytest.mark.parametrize("kw", [
    dict(experts=None), dict(x=None), dict(ids=None), dict(weights=None), dict(y=None), dict(tokens=-1), dict(top_k=0),
    dict(top_k=33), dict(x_stride=56), dict(y_stride=63), dict(residual=A, residual_stride=63), dict(activation=5),
    dict(activation=-1), dict(tokens=1 << 62)])
def test_moe_invalid(kw):
    assert _moe(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(x=A + 8), dict(x_stride=68), dict(ids=A + 2), dict(weights=A + 1), dict(y=A + 1), dict(residual=A + 1, residual_stride=64),
    dict(workspace=A + 128)])
def test_moe_misaligned(kw):
    assert _moe(**kw) == MISALIGNED


def _route(**kw):
    d = dict(x=A, x_stride=64, tokens=3, router=A, router_dtype=nv.DTYPE_BF16, router_stride=64, hidden=64, experts=8,
             bias=None, scoring=nv.SCORE_SOFTMAX, renormalize=1, scale=1.0, top_k=2, ids=A, weights=A, stream=None)
    d.update(kw)
    return nv.nvfp4_moe_route(*d.values())


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(router=None), dict(ids=None), dict(weights=None), dict(tokens=-1), dict(tokens=1 << 31), dict(hidden=0),
    dict(hidden=60), dict(experts=0), dict(experts=1025), dict(top_k=0), dict(top_k=9), dict(experts=64, top_k=33),
    dict(x_stride=56), dict(router_stride=56), dict(router_dtype=nv.DTYPE_E4M3), dict(scoring=2), dict(renormalize=2),
    dict(scale=float("inf")), dict(scale=float("nan")), dict(bias=A)])
def test_route_invalid(kw):
    assert _route(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(x=A + 2), dict(x_stride=68), dict(router=A + 8), dict(router_stride=68), dict(ids=A + 2), dict(weights=A + 2),
    dict(bias=A + 2, scoring=nv.SCORE_SIGMOID), dict(router_dtype=nv.DTYPE_FP32, router_stride=66)])
def test_route_misaligned(kw):
    assert _route(**kw) == MISALIGNED


def _sampling(**kw):
    d = dict(temperature=None, top_k=None, top_p=None, min_p=None, temperature_all=1.0, top_k_all=0, top_p_all=1.0, min_p_all=0.0)
    d.update(kw)
    return nv.nvfp4_sampling(*d.values())


def _sample(**kw):
    d = dict(logits=A, dtype=nv.DTYPE_BF16, stride=100, rows=3, vocabulary=100, sampling=_sampling(), uniform=A, token=A,
             logprob=None, stream=None)
    d.update(kw)
    return nv.nvfp4_sample(*d.values())


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(uniform=None), dict(token=None), dict(dtype=nv.DTYPE_E4M3), dict(rows=-1), dict(rows=(1 << 27) + 1),
    dict(vocabulary=-1), dict(vocabulary=(1 << 20) + 1, stride=1 << 21), dict(stride=99), dict(stride=1 << 41)])
def test_sample_invalid(kw):
    assert _sample(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(logits=A + 1), dict(logits=A + 2, dtype=nv.DTYPE_FP32), dict(uniform=A + 2), dict(token=A + 1), dict(logprob=A + 2),
    dict(sampling=_sampling(temperature=A + 2)), dict(sampling=_sampling(top_k=A + 2)), dict(sampling=_sampling(top_p=A + 1)),
    dict(sampling=_sampling(min_p=A + 3))])
def test_sample_misaligned(kw):
    assert _sample(**kw) == MISALIGNED


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(nv.nvfp4_expert_matrix) == 48
    assert ctypes.sizeof(nv.nvfp4_experts) == 3 * 48 + 24
    assert ctypes.sizeof(nv.nvfp4_sampling) == 48


class _Elsewhere:
    """What the binding looks at of a tensor on a device that this machine need not have."""
    is_cuda = True

    def __init__(self, shape, dtype, device):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


@pytest.mark.parametrize("what", ["x", "residual", "out", "ids", "weights"])
def test_moe_refuses_operands_on_another_device(what):
    experts = nv.Experts.__new__(nv.Experts)
    experts.experts, experts.hidden, experts.inner, experts.device = 4, 64, 64, torch.device("cuda:0")
    on = {n: "cuda:1" if n == what else "cuda:0" for n in ("x", "residual", "out", "ids", "weights")}
    t = {n: _Elsewhere((2, 64), torch.bfloat16, on[n]) for n in ("x", "residual", "out")}
    t["ids"], t["weights"] = _Elsewhere((2, 2), torch.int32, on["ids"]), _Elsewhere((2, 2), torch.float32, on["weights"])
    with pytest.raises(ValueError, match="experts' device"):
        nv.moe(experts, t["x"], t["ids"], t["weights"], residual=t["residual"], out=t["out"])


def test_bindings_refuse_host_tensors():
    cpu = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nv.moe_route(cpu, cpu, 1)
    with pytest.raises(ValueError):
        nv.sample(cpu, torch.zeros(2))
    with pytest.raises(ValueError):
        nv.Experts(*(tuple(torch.zeros((2, 32, n), dtype=torch.uint8) for n in (32, 4)) + (torch.ones(2),) for _ in range(2)))


def test_what_a_device_places_is_kept_by_device():
    """No kernel file holds a variable of its own (of one device's, another's call would read it, and threads race for it)."""
    csrc = os.path.join(os.path.dirname(nv.__file__), "csrc")
    for name in ("nvfp4_route.cu", "nvfp4_sample.cu", "nvfp4_moe.cu"):
        text = open(os.path.join(csrc, name)).read()
        assert re.findall(r"^(?:static )?(?:std::\w+<\w+>|int|bool|size_t|int64_t|uint\w+_t) \w+ *(?:=|\{[^}]*\};|;|\[)", text, re.M) == []


def test_small_clusters_are_asked_for_by_a_truth_value():
    assert nv.nvfp4_test_small_clusters(2) == INVALID and nv.nvfp4_test_small_clusters(-1) == INVALID
    assert nv.nvfp4_test_small_clusters(1) == 0 and nv.nvfp4_test_small_clusters(0) == 0


def test_sample_refuses_rows_past_every_address():
    for rows, stride in ((1 << 27, 1 << 39), (1 << 27, 1 << 35), (1 << 24, 1 << 38)):
        assert _sample(rows=rows, stride=stride) == INVALID
