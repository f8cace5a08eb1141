"""The decode-step operators' entry points on the host: what they refuse,
with which status, before touching the device."""
import ctypes
import os
import subprocess
import sys

import pytest

import nvfp4_block_scale_gb300 as nv

OK, INVALID, MISALIGNED = 0, 1, 2
A = 0x100000  # fake, aligned device address: never dereferenced on these paths


def _linear(**kw):
    d = dict(codes=A, scales=A, alpha=A, rows=4, cols=32, x=A, x_stride=32, batch=2, epilogue=None, y=A, y_stride=4,
             workspace=None, workspace_bytes=0, stream=None)
    d.update(kw)
    return nv.nvfp4_linear(*d.values())


def _ep(**kw):
    return nv.nvfp4_epilogue(**kw)


@pytest.mark.parametrize("kw", [
    dict(cols=24), dict(rows=-1), dict(batch=-1), dict(codes=None), dict(scales=None), dict(alpha=None), dict(x=None),
    dict(y=None), dict(x_stride=24), dict(y_stride=3), dict(epilogue=_ep(activation=5)), dict(epilogue=_ep(activation=-1)),
    dict(epilogue=_ep(gate=A, gate_stride=3)), dict(epilogue=_ep(residual=A, residual_stride=0)),
    dict(rows=1 << 25, cols=1 << 16, x_stride=1 << 16, y_stride=1 << 25)])
def test_linear_invalid(kw):
    assert _linear(**kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(codes=A + 4), dict(alpha=A + 2), dict(x=A + 8), dict(x_stride=36), dict(y=A + 1), dict(workspace=A + 16),
    dict(epilogue=_ep(bias=A + 1)), dict(epilogue=_ep(gate=A + 1, gate_stride=4)),
    dict(epilogue=_ep(residual=A + 1, residual_stride=4))])
def test_linear_misaligned(kw):
    assert _linear(**kw) == MISALIGNED


def _cache(**kw):
    d = dict(k=A, v=A, k_page_stride=2 * 16 * 64, v_page_stride=2 * 16 * 64, pages=4, page_size=16, kv_heads=2,
             head_dim=64, dtype=nv.DTYPE_BF16, k_scale=None, v_scale=None)
    d.update(kw)
    return nv.nvfp4_kv_cache(*d.values())


BAD_CACHES = [dict(head_dim=96), dict(head_dim=0), dict(page_size=24), dict(page_size=4), dict(page_size=1 << 17),
              dict(kv_heads=0), dict(pages=-1), dict(pages=1 << 31), dict(k=None), dict(v=None), dict(dtype=1),
              dict(dtype=3), dict(k_scale=A), dict(v_scale=A), dict(k_page_stride=2 * 16 * 64 - 8), dict(v_page_stride=0),
              dict(k_page_stride=1 << 61), dict(kv_heads=1 << 28)]
ODD_CACHES = [dict(k=A + 8), dict(v=A + 2), dict(k_page_stride=2 * 16 * 64 + 4),
              dict(dtype=nv.DTYPE_E4M3, v_page_stride=2 * 16 * 64 + 8), dict(dtype=nv.DTYPE_E4M3, k_scale=A + 2)]


def _append(**kw):
    d = dict(cache=_cache(), qkv=A, qkv_dtype=nv.DTYPE_BF16, qkv_stride=8 * 64, tokens=3, q_heads=4, seq=A, pos=A,
             table=A, sequences=2, table_width=4, table_stride=4, cos_sin=A, positions=100, rotary_dim=64,
             interleaved=0, q_out=A, stream=None)
    d.update(kw)
    return nv.nvfp4_kv_append(*d.values())


def _attend(**kw):
    d = dict(cache=_cache(), q=A, q_stride=4 * 64, sequences=2, q_heads=4, lengths=A, table=A, table_width=4,
             table_stride=4, scale=0.125, window=0, out=A, lse=A, workspace=None, workspace_bytes=0, stream=None)
    d.update(kw)
    return nv.nvfp4_paged_attention(*d.values())


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_cache(kw):
    assert _append(cache=_cache(**kw)) == INVALID
    assert _attend(cache=_cache(**kw)) == INVALID
    assert nv.nvfp4_paged_attention_workspace_bytes(_cache(**kw), 4) == -1


@pytest.mark.parametrize("kw", ODD_CACHES)
def test_misaligned_cache(kw):
    assert _append(cache=_cache(**kw)) == MISALIGNED
    assert _attend(cache=_cache(**kw)) == MISALIGNED


@pytest.mark.parametrize("kw", [
    dict(cache=None), dict(qkv=None), dict(seq=None), dict(pos=None), dict(q_out=None), dict(cos_sin=None),
    dict(table=None), dict(qkv_dtype=2), dict(qkv_stride=8 * 64 - 8), dict(tokens=-1), dict(q_heads=-1),
    dict(sequences=-1), dict(table_width=-1), dict(table_stride=3), dict(positions=-1), dict(rotary_dim=24),
    dict(rotary_dim=80), dict(rotary_dim=-16), dict(interleaved=2)])
def test_append_invalid(kw):
    assert _append(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(qkv=A + 8), dict(qkv_stride=8 * 64 + 4), dict(q_out=A + 4), dict(cos_sin=A + 8),
                                dict(seq=A + 2), dict(pos=A + 1), dict(table=A + 2),
                                dict(qkv_dtype=nv.DTYPE_FP32, qkv_stride=8 * 64 + 2)])
def test_append_misaligned(kw):
    assert _append(**kw) == MISALIGNED


@pytest.mark.parametrize("kw", [
    dict(cache=None), dict(q=None), dict(lengths=None), dict(out=None), dict(table=None), dict(q_heads=3),
    dict(q_heads=0), dict(q_heads=2048), dict(sequences=-1), dict(sequences=65536), dict(q_stride=4 * 64 - 8),
    dict(window=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(table_width=1 << 28, table_stride=1 << 28)])
def test_attention_invalid(kw):
    assert _attend(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(q=A + 8), dict(q_stride=4 * 64 + 4), dict(out=A + 8), dict(lse=A + 2),
                                dict(lengths=A + 2), dict(table=A + 1), dict(workspace=A + 64)])
def test_attention_misaligned(kw):
    assert _attend(**kw) == MISALIGNED


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(nv.nvfp4_epilogue) == 48
    assert ctypes.sizeof(nv.nvfp4_kv_cache) == 72
    assert nv.nvfp4_linear_workspace_bytes(4, 24, 1) == -1
    assert nv.nvfp4_linear_workspace_bytes(4, 32, -1) == -1


def test_loading_the_library_does_not_load_torch():
    code = "import sys, nvfp4_block_scale_gb300 as nv; nv.load(); assert nv.nvfp4_status_string(0) == 'ok'; " \
           "sys.exit('torch' in sys.modules)"
    root = os.path.dirname(os.path.dirname(os.path.abspath(nv.__file__)))
    assert subprocess.run([sys.executable, "-c", code], cwd=root).returncode == 0
