"""nvfp4_kv_append against the same rotation and rounding in elementary fp32
steps: queries, stored keys and values are equal bit for bit, and every other
slot of the cache keeps what it held."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import nvfp4_block_scale_gb300 as nv

pytestmark = pytest.mark.gpu
KINDS = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _cache(pages, heads, page, dim, kind, scaled=True, gap=0):
    n = heads * page * dim
    flat = [torch.full((pages, n + gap), 0x3C, dtype=torch.uint8, device="cuda") if kind == "e4m3" else
            torch.full((pages, n + gap), 0.5, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = (t[:, :n].view(KINDS[kind]).view(pages, heads, page, dim) for t in flat)
    sc = [torch.rand(heads, device="cuda") * 0.02 + 0.01 for _ in range(2)] if kind == "e4m3" and scaled else [None, None]
    return nv.KVCache(k, v, *sc), flat


def _expect(cache, qkv, hq, seq, pos, table, cos_sin, interleaved):
    """Elementary fp32 steps on the host; the cache's contents before the call are taken as they are."""
    hk, dim, page = cache.kv_heads, cache.head_dim, cache.page_size
    x = qkv.float().cpu().numpy().reshape(len(seq), hq + 2 * hk, dim)
    kb, vb = (t.view(torch.uint8).cpu().clone() if t.dtype != torch.bfloat16 else t.cpu().clone()
              for t in (cache.k, cache.v))
    q = torch.zeros((len(seq), hq, dim), dtype=torch.bfloat16)
    for t, (s, p) in enumerate(zip(seq, pos)):
        entry = p // page
        if not (0 <= s < table.shape[0] and 0 <= p and entry < table.shape[1]):
            continue
        if cos_sin is not None and p >= len(cos_sin):
            continue
        at = table[s, entry]
        if not 0 <= at < cache.pages:
            continue
        qk = x[t:t + 1, :hq + hk]
        if cos_sin is not None:
            qk = ref.rotate(qk, cos_sin, np.array([p]), interleaved)
        q[t] = torch.from_numpy(qk[0, :hq].copy()).to(torch.bfloat16)
        for buf, val, sc in ((kb, qk[0, hq:], cache.k_scale), (vb, x[t, hq + hk:], cache.v_scale)):
            val = torch.from_numpy(np.ascontiguousarray(val))
            if buf.dtype == torch.uint8:
                if sc is not None:
                    val = val * (1.0 / sc.cpu())[:, None]
                val = val.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                val = val.to(torch.bfloat16)
            buf[at, :, p % page] = val
    return q, kb, vb


def _run(cache, qkv, hq, seq, pos, table, cos_sin, interleaved):
    dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    want = _expect(cache, qkv, hq, seq, pos, table, cos_sin, interleaved)
    cs = None if cos_sin is None else torch.from_numpy(cos_sin).cuda()
    q = nv.kv_append(cache, qkv, hq, dev(seq), dev(pos), dev(table), cs, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(q.cpu(), want[0])
    for got, buf in ((cache.k, want[1]), (cache.v, want[2])):
        got = got.view(torch.uint8) if got.dtype != torch.bfloat16 else got
        assert torch.equal(got.cpu(), buf)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("inp", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dim,rotary,interleaved,hq,hk,page", [
    (64, 64, False, 8, 2, 16), (64, 16, True, 5, 5, 8), (128, 128, False, 32, 8, 32), (128, 96, True, 7, 1, 64),
    (256, 128, False, 3, 1, 8), (256, 256, True, 16, 16, 16), (128, 0, False, 0, 3, 128)])
def test_matches_elementary_steps(kind, inp, dim, rotary, interleaved, hq, hk, page):
    rng = np.random.default_rng(dim + hq)
    lens, start = [1, 5, 40, 0, 17], [0, 13, 3, 0, 2 * page - 1]
    ends = [s + n for s, n in zip(start, lens)]
    cache, _ = _cache(sum(-(-e // page) for e in ends) + 2, hk, page, dim, kind)
    table = ref.page_table(ends, page, cache.pages, 5)
    seq = np.repeat(np.arange(5), lens)
    pos = np.concatenate([np.arange(s, s + n) for s, n in zip(start, lens)])
    order = rng.permutation(len(seq))
    qkv = torch.from_numpy((3.0 * rng.standard_normal((len(seq), (hq + 2 * hk) * dim))).astype(np.float32)).to(inp).cuda()
    cos_sin = ref.angles(max(ends), rotary) if rotary else None
    _run(cache, qkv, hq, seq[order], pos[order], table, cos_sin, interleaved)


@pytest.mark.parametrize("tokens", [1, 2500])
def test_one_token_and_many(tokens):
    rng = np.random.default_rng(tokens)
    cache, _ = _cache(-(-(tokens + 9) // 64) + 1, 8, 64, 128, "bf16")
    table = ref.page_table([tokens + 9], 64, cache.pages, 6)
    qkv = torch.from_numpy(rng.standard_normal((tokens, 48 * 128)).astype(np.float32)).to(torch.bfloat16).cuda()
    _run(cache, qkv, 32, np.zeros(tokens, int), np.arange(9, 9 + tokens), table, ref.angles(tokens + 9, 128), False)


def test_tokens_that_are_skipped_leave_the_cache_alone():
    cache, _ = _cache(4, 2, 8, 64, "bf16")
    table = np.array([[2, 7], [-1, 0], [1, 3]], np.int32)  # page 7 does not exist, -1 is no page
    seq = [0, 0, 0, 1, 1, -1, 3, 2, 2, 2, 1 << 30]
    pos = [3, -1, 9, 2, 10, 0, 0, 16, 15, -2 ** 31, 2 ** 31 - 1]  # 16 is past the table's width
    rng = np.random.default_rng(1)
    qkv = torch.from_numpy(rng.standard_normal((len(seq), 6 * 64)).astype(np.float32)).cuda()
    _run(cache, qkv, 2, seq, pos, table, ref.angles(12, 64), False)  # position 15 has no angle
    _run(cache, qkv, 2, seq, pos, table, None, False)


def test_strided_pages_rows_and_tables():
    cache, flat = _cache(6, 3, 8, 64, "e4m3", gap=48)
    table = ref.page_table([20, 9], 8, 6, 7, spare=2)
    wide = torch.full((2, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = torch.from_numpy(table)
    rng = np.random.default_rng(2)
    big = torch.from_numpy(rng.standard_normal((4, 8 * 64 + 32)).astype(np.float32)).to(torch.bfloat16).cuda()
    qkv = big[:, 16:16 + 8 * 64]
    seq, pos = [0, 1, 0, 1], [19, 0, 7, 8]
    want = _expect(cache, qkv, 2, seq, pos, table, None, False)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    q = nv.kv_append(cache, qkv, 2, dev(seq), dev(pos), wide[:, :table.shape[1]])
    assert torch.equal(q.cpu(), want[0]) and torch.equal(cache.k.view(torch.uint8).cpu(), want[1])
    assert torch.equal(cache.v.view(torch.uint8).cpu(), want[2])
    assert bool((flat[0][:, -48:] == 0x3C).all()) and bool((flat[1][:, -48:] == 0x3C).all())


@pytest.mark.parametrize("scaled", [False, True])
def test_8_bit_values_saturate_and_keep_nan(scaled):
    cache, _ = _cache(2, 1, 8, 64, "e4m3", scaled=scaled)
    v = np.array([0.0, -0.0, 1e9, -1e9, np.inf, -np.inf, 448.0, 449.0, 2.0 ** -10, 2.0 ** -9, 2.0 ** -11, 1.0625, 1.1875] +
                 [300.0] * 51, np.float32)
    qkv = torch.from_numpy(np.concatenate((v, -v))[None]).cuda()
    _run(cache, qkv, 0, [0], [4], np.array([[1]], np.int32), None, False)
    qkv[0, 5] = float("nan")
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    nv.kv_append(cache, qkv, 0, i([0]), i([5]), i([[1]]))
    row = cache.k[1, 0, 5].float()
    assert bool(torch.isnan(row[5])) and int(torch.isnan(row).sum()) == 1


def test_capture_and_another_stream():
    cache, _ = _cache(8, 2, 16, 128, "bf16")
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    qkv = torch.randn(3, 8 * 128, device="cuda").to(torch.bfloat16)
    seq, pos, table = i([0, 1, 1]), i([17, 2, 3]), i([[3, 5], [0, 1]])
    cs = torch.from_numpy(ref.angles(32, 128)).cuda()
    q = nv.kv_append(cache, qkv, 4, seq, pos, table, cs)
    k, v = cache.k.clone(), cache.v.clone()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    for run in ("stream", "graph"):
        cache.k.fill_(0.5)
        cache.v.fill_(0.5)
        if run == "stream":
            side.wait_stream(torch.cuda.current_stream())
            r = nv.kv_append(cache, qkv, 4, seq, pos, table, cs, stream=side)
            torch.cuda.current_stream().wait_stream(side)
        else:
            with torch.cuda.graph(g):
                r = nv.kv_append(cache, qkv, 4, seq, pos, table, cs)
            g.replay()
        assert torch.equal(r, q) and torch.equal(cache.k, k) and torch.equal(cache.v, v)
