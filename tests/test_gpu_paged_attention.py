"""nvfp4_paged_attention against the same in 64 bits, head group by head
group, within the derived bounds of decode_ref.attend.  Pages lie scattered;
what a sequence does not reach (other pages, the tail of its last one) holds
NaN in every test but the ones on larger caches."""
import numpy as np
import pytest
import torch

import decode_ref as ref
import nvfp4_block_scale_gb300 as nv

pytestmark = pytest.mark.gpu


def _setup(lengths, hq, hk, dim, page, kind, seed, scaled=True, spare_pages=2):
    rng = np.random.default_rng(seed)
    pages = sum(-(-max(0, int(n)) // page) for n in lengths) + spare_pages
    table = ref.page_table([max(0, int(n)) for n in lengths], page, pages, seed)
    shape = (pages, hk, page, dim)
    vals = [rng.standard_normal(shape).astype(np.float32) for _ in range(2)]
    mask = np.ones((pages, page), bool)  # slots that no sequence reaches
    for i, n in enumerate(lengths):
        for j in range(-(-max(0, int(n)) // page)):
            mask[table[i, j], :max(0, min(page, int(n) - j * page))] = False
    sc = [None, None]
    if kind == "e4m3":
        if scaled:
            sc = [torch.from_numpy((0.01 + 0.02 * rng.random(hk)).astype(np.float32)).cuda() for _ in range(2)]
            vals = [v * 60.0 for v in vals]
    kt = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    kv = []
    for v in vals:
        v[np.broadcast_to(mask[:, None, :, None], shape)] = np.nan
        kv.append(torch.from_numpy(v).to(kt).cuda())
    q = torch.from_numpy((1.5 * rng.standard_normal((len(lengths), hq, dim))).astype(np.float32)).to(torch.bfloat16).cuda()
    return nv.KVCache(kv[0], kv[1], *sc), q, torch.from_numpy(table).cuda(), \
        torch.tensor([int(n) for n in lengths], dtype=torch.int32, device="cuda")


def _check(cache, q, table, lengths, out, lse, scale=None, window=0, which=None):
    hk, dim, g = cache.kv_heads, cache.head_dim, q.shape[1] // cache.kv_heads
    scale = dim ** -0.5 if scale is None else scale
    qh, o, ls = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i, n in enumerate(lengths.tolist()):
        if which is not None and i not in which:
            continue
        n = max(0, min(n, table.shape[1] * cache.page_size))
        ids = table[i, :-(-n // cache.page_size)].long()
        for h in range(hk):
            k, v = (np.asarray(t.view(torch.uint8)[ids, h].view(torch.float8_e4m3fn).double().cpu()
                               if t.dtype != torch.bfloat16 else t[ids, h].double().cpu()).reshape(-1, dim)[:n]
                    for t in (cache.k, cache.v))
            if cache.k_scale is not None:
                k, v = k * cache.k_scale[h].item(), v * cache.v_scale[h].item()
            ro, rl, bo, bl = ref.attend(qh[i, h * g:(h + 1) * g], k, v, scale, window)
            go, gl = o[i, h * g:(h + 1) * g], ls[i, h * g:(h + 1) * g]
            assert ref.within(go, ro, bo), (i, h)
            if n == 0:
                assert np.all(np.isneginf(gl)) and np.all(go == 0)
            else:
                assert np.all(np.abs(gl - rl) <= bl), (i, h, float((np.abs(gl - rl) / bl).max()))


HEADS = [(8, 8), (32, 8), (6, 2), (7, 1), (8, 1), (12, 1), (16, 1), (18, 2), (40, 1), (64, 2), (71, 1)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk", HEADS)
def test_head_groups(kind, hq, hk):
    cache, q, table, n = _setup([1, 33, 0, 250], hq, hk, 128, 16, kind, hq * 100 + hk)
    _check(cache, q, table, n, *nv.paged_attention(cache, q, table, n, return_lse=True))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 256])
def test_dims_and_pages(kind, dim, page):
    cache, q, table, n = _setup([0, 1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 130, 300], 8, 2, dim, page,
                                kind, dim + page, scaled=page != 16)
    _check(cache, q, table, n, *nv.paged_attention(cache, q, table, n, return_lse=True))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 5000])
def test_windows(kind, window):
    cache, q, table, n = _setup([0, 1, 16, 17, 99, 100, 101, 640], 8, 4, 64, 32, kind, window)
    _check(cache, q, table, n, *nv.paged_attention(cache, q, table, n, window=window, return_lse=True), window=window)


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 1, 2 ** 31, 2 ** 62, 2 ** 63 - 33, 2 ** 63 - 1])
@pytest.mark.parametrize("hq,hk,dim,count", [(8, 8, 64, 601), (16, 2, 128, 81), (24, 1, 256, 7)])
def test_windows_wider_than_any_context(hq, hk, dim, count, window):
    """Any window >= 0 is accepted, and one that holds every token is none."""
    lengths = np.random.default_rng(count).integers(0, 200, count)
    cache, q, table, n = _setup(lengths, hq, hk, dim, 32, "bf16", 41)
    want = nv.paged_attention(cache, q, table, n, return_lse=True)
    got = nv.paged_attention(cache, q, table, n, window=window, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", [(32, 8, 128), (4, 4, 64), (24, 1, 256)])
def test_long_and_short_together(kind, hq, hk, dim):
    """Lengths for which one sequence is cut over many CTAs while others are not."""
    lengths = [20011, 3, 0, 4096, 1, 777]
    cache, q, table, n = _setup(lengths, hq, hk, dim, 64, kind, 11)
    out = nv.paged_attention(cache, q, table, n, return_lse=True)
    _check(cache, q, table, n, *out)
    again = nv.paged_attention(cache, q, table, n, return_lse=True)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,hk,dim", [(8, 1, 128), (24, 1, 256), (16, 1, 256), (48, 1, 128), (32, 1, 64), (6, 2, 64)])
def test_short_items_between_long_ones(kind, hq, hk, dim):
    """CTAs that hold several short items, each one warp's, between parts of
    long ones: the queries of one must not reach another."""
    rng = np.random.default_rng(hq)
    lengths = []
    for i in range(24):
        lengths += [int(rng.integers(2500, 6000))] + [int(n) for n in rng.integers(0, 40, int(rng.integers(1, 9)))]
    cache, q, table, n = _setup(lengths, hq, hk, dim, 64, kind, 21)
    out = nv.paged_attention(cache, q, table, n, return_lse=True)
    _check(cache, q, table, n, *out, which={i for i, m in enumerate(lengths) if m < 40} | {0, len(lengths) - 1})
    again = nv.paged_attention(cache, q, table, n, return_lse=True)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("hk,dim,kind", [(3, 128, "bf16"), (8, 128, "bf16"), (5, 64, "bf16"), (8, 128, "e4m3")])
def test_short_contexts_repeat_over_many_calls(hk, dim, kind):
    """Tiles that follow one another quickly in the same shared memory: what a
    warp still reads must not be the next tile (which took one call in 300)."""
    rng = np.random.default_rng(hk)
    lengths = rng.integers(0, 80, 330).tolist()
    cache, q, table, n = _setup(lengths, hk, hk, dim, 64, kind, 31)
    first = nv.paged_attention(cache, q, table, n, return_lse=True)
    _check(cache, q, table, n, *first, which=set(range(0, 330, 11)))
    wrong = torch.zeros(2, dtype=torch.int64, device="cuda")
    space = nv.attention_workspace(cache, hk)
    for _ in range(2000):
        out, lse = nv.paged_attention(cache, q, table, n, return_lse=True, workspace=space)
        wrong[0] += (out != first[0]).any()
        wrong[1] += (lse != first[1]).any()
    assert wrong.tolist() == [0, 0]


@pytest.mark.parametrize("kind,bits", [("bf16", 16), ("e4m3", 11)])
@pytest.mark.parametrize("hq,hk,dim", [(4, 2, 64), (8, 1, 128), (3, 1, 256), (12, 1, 64), (24, 1, 128), (16, 1, 256)])
def test_weights_keep_their_bits(kind, bits, hq, hk, dim):
    """Scores so small that their own error is far below a weight's rounding:
    decode_ref.attend's bound with 2^-bits in place of 2^-8 for the weights (half
    a unit of as many bits; two bf16 numbers hold a weight to 2^-16)."""
    lengths = [2, 3, 5, 9, 16, 33, 70, 130, 300]
    cache, q, table, n = _setup(lengths, hq, hk, dim, 16, kind, 43, scaled=False)
    q.mul_(2.0 ** -5 if kind == "bf16" else 2.0 ** -11)
    out, lse = nv.paged_attention(cache, q, table, n, return_lse=True)
    g = hq // hk
    for i, m in enumerate(lengths):
        ids = table[i, :-(-m // 16)].long()
        for h in range(hk):
            k, v = (t.float()[ids, h].double().cpu().numpy().reshape(-1, dim)[:m] for t in (cache.k, cache.v))
            qh = q[i, h * g:(h + 1) * g].double().cpu().numpy()
            ro, rl, bo, bl = ref.attend(qh, k, v, dim ** -0.5)
            mag = ref.attend(qh, k, np.abs(v), dim ** -0.5)[0]
            assert ref.within(out[i, h * g:(h + 1) * g].double().cpu().numpy(), ro, bo - (2.0 ** -8 - 2.0 ** -bits) * mag), (i, h)
            assert np.all(np.abs(lse[i, h * g:(h + 1) * g].double().cpu().numpy() - rl) <= bl)


def test_many_sequences():
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 60, 1500)
    lengths[::9] = 0
    cache, q, table, n = _setup(lengths, 4, 2, 64, 16, "bf16", 12)
    out, lse = nv.paged_attention(cache, q, table, n, return_lse=True)
    _check(cache, q, table, n, out, lse, which=set(range(0, 1500, 37)) | {1499})
    assert bool((out[n == 0] == 0).all()) and bool(torch.isneginf(lse[n == 0]).all())
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse[n > 0]).all())


def test_all_rows_empty_and_no_sequence():
    cache, q, table, n = _setup([0, 0, 0], 8, 2, 128, 16, "bf16", 13)
    n[1] = -5
    out, lse = nv.paged_attention(cache, q, table, n, return_lse=True)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
    o = nv.paged_attention(cache, q[:0], table[:0], n[:0])
    assert o.shape == (0, 8, 128)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_large_scores_of_both_signs(kind):
    """Scores far apart: rising, falling, and one key that takes all of the weight."""
    cache, q, table, n = _setup([200, 200, 200], 8, 2, 64, 16, kind, 14)
    for i, ramp in enumerate((torch.arange(200.0) / 8, 25.0 - torch.arange(200.0) / 8)):
        for t in range(200):
            at = cache.k[table[i, t // 16].item(), :, t % 16]
            at.copy_((ramp[t] * torch.ones_like(at, dtype=torch.float32)).to(at.dtype))
    cache.k[table[2, 5].item(), :, 3].copy_((torch.full((2, 64), 200.0, device="cuda")).to(cache.k.dtype))
    q.copy_(q.abs())
    scale = 0.5
    _check(cache, q, table, n, *nv.paged_attention(cache, q, table, n, scale=scale, return_lse=True), scale=scale)
    q.neg_()
    _check(cache, q, table, n, *nv.paged_attention(cache, q, table, n, scale=scale, return_lse=True), scale=scale)


def test_queries_of_extreme_size():
    """Each query row keeps its own precision: 8-bit keys take queries as small as 2^-40 or as large as 2^20."""
    for kind in ("bf16", "e4m3"):
        cache, q, table, n = _setup([150, 70], 8, 1, 128, 16, kind, 15)
        q[0, 0] *= 2.0 ** 20
        q[0, 1] *= 2.0 ** -40
        q[0, 2] = 0.0
        q[1, 3, ::5] *= 2.0 ** 18
        for scale in (2.0 ** -20, 0.05):
            out, lse = nv.paged_attention(cache, q, table, n, scale=scale, return_lse=True)
            keep = torch.isfinite(lse)
            assert bool(keep.all())
            _check(cache, q, table, n, out, lse, scale=scale)


def test_infinite_scores():
    """A key of -inf weighs nothing; a row of such keys alone counts as empty; a NaN key spoils its row only."""
    cache, q, table, n = _setup([40, 3, 40], 4, 1, 64, 8, "bf16", 16)
    q.copy_(q.abs() + 0.1)
    cache.k[table[0, 0].item(), 0, :] = -float("inf")  # the sequence's first 8 keys
    cache.k[table[1, 0].item(), 0, :3] = -float("inf")
    cache.k[table[2, 1].item(), 0, 2] = float("nan")
    out, lse = nv.paged_attention(cache, q, table, n, return_lse=True)
    short = table[:1, 1:].contiguous()
    o, ls = nv.paged_attention(cache, q[:1], short, n[:1] - 8, return_lse=True)
    assert torch.allclose(out[:1].float(), o.float(), rtol=2 ** -7, atol=2 ** -7) and torch.allclose(lse[:1], ls, rtol=1e-5)
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    assert bool(torch.isnan(out[2].float()).all()) and bool(torch.isnan(lse[2]).all())


def test_page_numbers_outside_the_cache_read_as_zeros():
    cache, q, table, n = _setup([64, 64], 8, 2, 64, 16, "bf16", 17)
    bad = table.clone()
    bad[0, 1], bad[0, 2], bad[1, 3] = -1, cache.pages, 2 ** 31 - 1
    out, lse = nv.paged_attention(cache, q, bad, n, return_lse=True)
    k, v = cache.k.clone(), cache.v.clone()
    for i, j in ((0, 1), (0, 2), (1, 3)):
        k[table[i, j].item()] = 0
        v[table[i, j].item()] = 0
    o, ls = nv.paged_attention(nv.KVCache(k, v), q, table, n, return_lse=True)
    assert torch.equal(out, o) and torch.equal(lse, ls)


def test_strided_pages_queries_and_tables():
    cache, q, table, n = _setup([90, 5, 33], 8, 2, 64, 16, "bf16", 18)
    want = nv.paged_attention(cache, q, table, n, return_lse=True)
    both = torch.stack((cache.k, cache.v), 1).contiguous()  # keys and values of a page side by side
    wide_q = torch.zeros((3, 12 * 64), dtype=torch.bfloat16, device="cuda")
    wide_q[:, 64:9 * 64] = q.flatten(1)
    wide_t = torch.full((3, table.shape[1] + 5), 3, dtype=torch.int32, device="cuda")
    wide_t[:, 2:2 + table.shape[1]] = table
    got = nv.paged_attention(nv.KVCache(both[:, 0], both[:, 1]), wide_q.as_strided((3, 8, 64), (12 * 64, 64, 1), 64),
                             wide_t[:, 2:2 + table.shape[1]], n,
                             return_lse=True)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("count,n0,hq,hk,dim,page", [(1, 517, 32, 8, 128, 16), (1, 300, 8, 8, 64, 16), (3, 150, 8, 2, 128, 16),
                                                     (2, 900, 16, 2, 256, 32), (5, 64, 8, 8, 128, 16), (40, 20, 8, 8, 128, 16),
                                                     (1, 8192, 40, 1, 64, 64)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 100])
def test_results_do_not_depend_on_the_tables_width(count, n0, hq, hk, dim, page, kind, window):
    """The order of the additions goes by the lengths and the device only."""
    cache, q, table, n = _setup([n0] * count, hq, hk, dim, page, kind, 42)
    want = nv.paged_attention(cache, q, table[:, :-(-n0 // page)], n, window=window, return_lse=True)
    for more in (1, 7, 60, 5000):
        wide = torch.full((count, -(-n0 // page) + more), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
        got = nv.paged_attention(cache, q, wide, n, window=window, return_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_lengths_beyond_the_table_are_clipped():
    cache, q, table, n = _setup([32, 32], 4, 2, 64, 16, "bf16", 19)
    cut = table[:, :2].contiguous()
    a = nv.paged_attention(cache, q, cut, n, return_lse=True)
    b = nv.paged_attention(cache, q, cut, n + 1000000, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_workspace_streams_and_capture():
    cache, q, table, n = _setup([9000, 17, 0, 700], 16, 2, 128, 32, "bf16", 20)
    ws = nv.attention_workspace(cache, 16)
    want = nv.paged_attention(cache, q, table, n, return_lse=True)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    got = [nv.paged_attention(cache, q, table, n, return_lse=True, workspace=ws, stream=side) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        got += [nv.paged_attention(cache, q, table, n, return_lse=True, workspace=w) for w in (ws, None)]
    for o, ls in got[4:]:
        o.zero_()
        ls.zero_()
    n.copy_(torch.tensor([100, 20, 5, 8]))  # other lengths through the same graph, then the first ones again
    g.replay()
    n.copy_(torch.tensor([9000, 17, 0, 700]))
    g.replay()
    for o, ls in got:
        assert torch.equal(o, want[0]) and torch.equal(ls, want[1])


def test_a_cache_past_two_to_the_32_elements():
    """Pages whose elements lie beyond 2^32 elements (8 GiB) into the keys and values."""
    pages = (1 << 32) // (8 * 64 * 128) + 9
    k = torch.empty((pages, 8, 64, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    used = [pages - 1, pages - 3, 0, pages // 2, pages - 8]
    for p in used:
        k[p].normal_()
        v[p].normal_()
    cache = nv.KVCache(k, v)
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    n = torch.tensor([5 * 64 - 30], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 32, 128), device="cuda").to(torch.bfloat16)
    _check(cache, q, table, n, *nv.paged_attention(cache, q, table, n, return_lse=True))
    qkv = torch.randn((1, 48 * 128), device="cuda").to(torch.bfloat16)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    nv.kv_append(cache, qkv, 32, i([0]), i([5 * 64 - 30]), table)
    assert torch.equal(k[pages - 8, :, 34].flatten(), qkv[0, 32 * 128:40 * 128])
    assert torch.equal(v[pages - 8, :, 34].flatten(), qkv[0, 40 * 128:])
