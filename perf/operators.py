"""Cases of the decode-step operators: linear (the W4A16 product with its
epilogue), kv_append (rotation and paged cache write) and paged_attention
(one new token per sequence over that cache).

`run` computes an operator either in plain torch operations (own = False) or
through the framework's entry points (own = True) on what `prepare` made;
`exact` computes the same outputs in 64 bits.
"""
import math

import torch

if torch.cuda.is_available():
    DEVICE = torch.device("cuda")
else:
    DEVICE = torch.device("cpu")

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
CACHE_TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
INPUT_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def _append(name, tokens, sequences, history, q_heads, kv_heads, head_dim, page, cache, inp, rotary, interleaved):
    return {"name": name, "op": "append", "tokens": tokens, "sequences": sequences, "history": history,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "cache": cache,
            "input": inp, "rotary": rotary, "interleaved": interleaved}


def _attend(name, sequences, length, ragged, q_heads, kv_heads, head_dim, page, cache, window):
    return {"name": name, "op": "attend", "sequences": sequences, "length": length, "ragged": ragged,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "cache": cache,
            "window": window}


def _linear(name, batch, rows, cols, bias, act, gate, residual):
    return {"name": name, "op": "linear", "batch": batch, "rows": rows, "cols": cols, "bias": bias, "act": act,
            "gate": gate, "residual": residual}


def listed():
    return [
        # one user's next token: the whole cost is latency
        _append("append 1 token", 1, 1, 1000, 32, 8, 128, 16, "bf16", "bf16", 128, False),
        # a decode batch of odd size: rotated quarter of the head in interleaved pairs, fp32 products as they leave
        # nvfp4_gemm, 8-bit cache
        _append("append 129 fp32 to e4m3", 129, 129, 700, 40, 8, 64, 32, "e4m3", "fp32", 16, True),
        # prompts of five users taken in at once, wide heads
        _append("append 3001 D256", 3001, 5, 900, 16, 4, 256, 64, "bf16", "bf16", 128, False),
        # a long prompt into the 8-bit cache: the largest write
        _append("append 8192 to e4m3", 8192, 2, 0, 64, 8, 128, 64, "e4m3", "bf16", 128, False),
        # one user, short context: latency
        _attend("attend 1 x 517", 1, 517, False, 32, 8, 128, 16, "bf16", 0),
        # an ordinary decode batch, ragged lengths, odd count
        _attend("attend 61 x 2048 ragged", 61, 2048, True, 32, 8, 128, 16, "bf16", 0),
        # many short sequences (some without any token), one query head per cache head, sliding window, 8-bit cache
        _attend("attend 256 x 300 window e4m3", 256, 300, True, 16, 16, 64, 32, "e4m3", 128),
        # few long contexts in the 8-bit cache: the work has to be split over the length
        _attend("attend 3 x 65536 e4m3", 3, 65536, False, 64, 8, 128, 64, "e4m3", 0),
        # long contexts in bf16: the largest read
        _attend("attend 16 x 32768", 16, 32768, False, 64, 8, 128, 64, "bf16", 0),
        # one user's attention output projection with the residual stream
        _linear("linear 1 4096x4096", 1, 4096, 4096, False, "none", False, True),
        # an odd decode batch through the gated half of an MLP
        _linear("linear 13 14336x4096 silu", 13, 14336, 4096, False, "silu", True, False),
        # the largest decode batch through the benchmark's 8192 x 28672 tensor
        _linear("linear 256 8192x28672", 256, 8192, 28672, True, "gelu_tanh", False, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _draw_heads(rng):
    kv = rng.choice((1, 2, 4, 5, 8, 16))
    return min(96, kv * rng.choice((1, 2, 3, 4, 7, 8, 12, 16))) // kv * kv, kv


def draw(rng):
    kind = rng.choice(("append", "attend", "attend", "linear", "linear"))
    q_heads, kv_heads = _draw_heads(rng)
    head_dim, page = rng.choice((64, 128, 256)), rng.choice((8, 16, 32, 64, 128, 256))
    cache = rng.choice(("bf16", "e4m3"))
    if kind == "append":
        tokens = _log_int(rng, 1, 8192)
        while tokens * (q_heads + 2 * kv_heads) * head_dim > 8192 * 80 * 128:
            tokens = _log_int(rng, 1, 8192)
        sequences = tokens if tokens <= 256 and rng.random() < 0.6 else rng.randint(1, min(tokens, 16))
        c = _append("", tokens, sequences, _log_int(rng, 1, 1500), q_heads, kv_heads, head_dim, page, cache,
                    rng.choice(("bf16", "fp32")), 16 * rng.randint(1, head_dim // 16), rng.random() < 0.5)
    elif kind == "attend":
        size = {"bf16": 2, "e4m3": 1}[cache]
        while True:
            sequences, length = _log_int(rng, 1, 256), _log_int(rng, 1, 65536)
            n = sequences * length * head_dim
            if n * kv_heads * size < 1.0e9 and n * q_heads < 4.0e9 and n * kv_heads < 5.0e8:
                break
        c = _attend("", sequences, length, rng.random() < 0.6, q_heads, kv_heads, head_dim, page, cache,
                    rng.choice((0, 0, _log_int(rng, 1, 8192))))
    else:
        while True:
            batch, rows, cols = _log_int(rng, 1, 256), _log_int(rng, 32, 28672), 16 * _log_int(rng, 4, 1792)
            if rows * cols <= 8192 * 28672:
                break
        c = _linear("", batch, rows, cols, rng.random() < 0.5, rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                    rng.random() < 0.3, rng.random() < 0.5)
    del c["name"]
    return c


def _spread(n, top):
    """n whole numbers in 0..top, evenly spread in a scattered order (the golden ratio's multiples); the first is top."""
    return [top if i == 0 else int((0.5 + i * 0.6180339887498949) % 1.0 * (top + 1)) for i in range(n)]


def _lengths(case):
    return _spread(case["sequences"], case["length"]) if case["ragged"] else [case["length"]] * case["sequences"]


def _tokens(case):
    """(sequence, position) of every appended token: each sequence continues behind its history."""
    n, s = case["tokens"], case["sequences"]
    seq, pos = [], []
    for i, start in enumerate(_spread(s, case["history"])):
        count = n // s + (1 if i < n % s else 0)
        seq += [i] * count
        pos += range(start, start + count)
    return seq, pos


# ------------------------------------------------------------------ inputs

def _table(lengths, page, g):
    """A page table whose pages lie scattered over the cache, -1 behind each sequence's last; and the page count."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + 1
    perm = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    width = max(need) + 1
    at = torch.arange(width, device=DEVICE)
    n = torch.tensor(need, device=DEVICE)
    first = torch.cumsum(n, 0) - n
    index = (first[:, None] + at[None, :]).clamp(max=pages - 1)
    return torch.where(at[None, :] < n[:, None], perm[index], torch.full_like(perm[index], -1)).contiguous(), pages


def _prepare_cache(case, s, pages, g):
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    kind = CACHE_TYPES[case["cache"]]
    s["k"] = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16).to(kind)
    s["v"] = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16).to(kind)
    if case["cache"] == "e4m3":  # the value of a unit of each head's keys and values
        s["k_scale"] = 0.02 + 0.03 * torch.rand(case["kv_heads"], generator=g, device=DEVICE)
        s["v_scale"] = 0.02 + 0.03 * torch.rand(case["kv_heads"], generator=g, device=DEVICE)
    else:
        s["k_scale"] = s["v_scale"] = None
    if case["op"] == "attend" and case["cache"] == "e4m3":  # fill the type's range as written keys and values do
        s["k"] = (s["k"].to(torch.bfloat16) * 40).to(kind)
        s["v"] = (s["v"].to(torch.bfloat16) * 40).to(kind)


def _prepare_append(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    seq, pos = _tokens(case)
    ends = [0] * case["sequences"]
    for i, p in zip(seq, pos):
        ends[i] = max(ends[i], p + 1)
    s = {"case": case}
    s["table"], pages = _table(ends, case["page"], g)
    _prepare_cache(case, s, pages, g)
    s["seq"] = torch.tensor(seq, dtype=torch.int32, device=DEVICE)
    s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEVICE)
    width = (case["q_heads"] + 2 * case["kv_heads"]) * case["head_dim"]
    s["qkv"] = torch.randn((case["tokens"], width), generator=g, device=DEVICE).to(INPUT_TYPES[case["input"]])
    half = case["rotary"] // 2
    angle = torch.arange(max(ends), device=DEVICE, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)[None, :]
    s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
    return s


def _prepare_attend(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"case": case}
    lengths = _lengths(case)
    s["table"], pages = _table(lengths, case["page"], g)
    _prepare_cache(case, s, pages, g)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEVICE)
    s["q"] = (1.5 * torch.randn((case["sequences"], case["q_heads"], case["head_dim"]), generator=g,
                                device=DEVICE)).to(torch.bfloat16)
    s["scale"] = case["head_dim"] ** -0.5
    return s


def _prepare_linear(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    rows, cols, batch = case["rows"], case["cols"], case["batch"]
    s = {"case": case}
    w = 0.02 * torch.randn((rows, cols // 16, 16), generator=g, device=DEVICE)
    top = w.abs().amax(2, keepdim=True)
    s["alpha"] = (w.abs().max() / 2688.0).reshape(1)
    scale = (top / (6.0 * s["alpha"])).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = (scale.float() * s["alpha"]).clamp(min=1e-30)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
    code = (torch.bucketize(w.abs() / unit, edges, out_int32=True) + 8 * (w < 0).int()).to(torch.uint8).view(rows, cols)
    s["codes"] = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    s["scales"] = scale.view(torch.uint8).view(rows, cols // 16).contiguous()
    del w, top, scale, unit, code
    s["x"] = torch.randn((batch, cols), generator=g, device=DEVICE).to(torch.bfloat16)
    s["bias"] = torch.randn(rows, generator=g, device=DEVICE).to(torch.bfloat16) if case["bias"] else None
    s["gate"] = torch.randn((batch, rows), generator=g, device=DEVICE).to(torch.bfloat16) if case["gate"] else None
    s["residual"] = torch.randn((batch, rows), generator=g, device=DEVICE).to(torch.bfloat16) if case["residual"] else None
    return s


def prepare(case, seed):
    s = {"append": _prepare_append, "attend": _prepare_attend, "linear": _prepare_linear}[case["op"]](case, seed)
    if own:  # the cache's handle and the workspace that a serving program keeps from step to step
        import nvfp4_block_scale_gb300 as nv
        s["nv"] = nv
        if case["op"] != "linear":
            s["handle"] = nv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] == "attend":
            s["workspace"] = nv.attention_workspace(s["handle"], case["q_heads"])
        if case["op"] == "linear":
            s["workspace"] = nv.linear_workspace(case["rows"], case["cols"], case["batch"])
    return s


# ---------------------------------------------------------------- plain form

def _plain_append(s):
    c = s["case"]
    hq, hk, d, r = c["q_heads"], c["kv_heads"], c["head_dim"], c["rotary"]
    x = s["qkv"].float().view(-1, hq + 2 * hk, d)
    pos, seq = s["pos"].long(), s["seq"].long()
    cos, sin = s["cos_sin"][pos][:, None, :r // 2], s["cos_sin"][pos][:, None, r // 2:]
    qk = x[:, :hq + hk]
    rot = qk[..., :r]
    if c["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = rot[..., :r // 2], rot[..., r // 2:]
        rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    qk = torch.cat((rot, qk[..., r:]), -1)
    k, v = qk[:, hq:], x[:, hq + hk:]
    page, row = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    if c["cache"] == "e4m3":
        k = (k * (1.0 / s["k_scale"])[:, None]).clamp(-448.0, 448.0)
        v = (v * (1.0 / s["v_scale"])[:, None]).clamp(-448.0, 448.0)
        s["k"].view(torch.uint8)[page, :, row] = k.to(torch.float8_e4m3fn).view(torch.uint8)
        s["v"].view(torch.uint8)[page, :, row] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        s["k"][page, :, row] = k.to(torch.bfloat16)
        s["v"][page, :, row] = v.to(torch.bfloat16)
    return {"q": qk[:, :hq].to(torch.bfloat16), "k": s["k"], "v": s["v"]}


def _gathered(cache, table, scale):
    x = cache[table].float()  # [sequences, pages, heads, page, dim]
    x = x.transpose(1, 2).flatten(2, 3)
    return x if scale is None else x * scale[None, :, None, None]


def _plain_attend(s):
    c = s["case"]
    n, hk, g = c["sequences"], c["kv_heads"], c["q_heads"] // c["kv_heads"]
    table = s["table"].clamp(min=0).long()
    q = s["q"].float().view(n, hk, g, -1)
    score = torch.matmul(q, _gathered(s["k"], table, s["k_scale"]).transpose(2, 3)) * s["scale"]
    at = torch.arange(score.shape[3], device=score.device)
    length = s["lengths"].long()[:, None]
    seen = at < length
    if c["window"]:
        seen = seen & (at >= length - c["window"])
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    m = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, _gathered(s["v"], table, s["v_scale"]))
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return {"out": out.reshape(n, hk * g, -1).to(torch.bfloat16),
            "lse": (m + torch.log(total)).reshape(n, hk * g)}


def _activate(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _plain_linear(s):
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=s["codes"].device)
    rows, half = s["codes"].shape
    q = torch.stack((value[(s["codes"] & 15).int()], value[(s["codes"] >> 4).int()]), -1).view(rows, half // 8, 16)
    w = (q * s["scales"].view(torch.float8_e4m3fn).float()[..., None]).view(rows, 2 * half)
    v = torch.matmul(s["x"].float(), w.t()) * s["alpha"]
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _activate(v, s["case"]["act"])
    if s["gate"] is not None:
        v = v * s["gate"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(torch.bfloat16)


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "linear": _plain_linear}[c["op"]](s)
    nv = s["nv"]
    if c["op"] == "append":
        q = nv.kv_append(s["handle"], s["qkv"], c["q_heads"], s["seq"], s["pos"], s["table"], s["cos_sin"],
                         interleaved=c["interleaved"])
        return {"q": q, "k": s["k"], "v": s["v"]}
    if c["op"] == "attend":
        out, lse = nv.paged_attention(s["handle"], s["q"], s["table"], s["lengths"], scale=s["scale"],
                                      window=c["window"], return_lse=True, workspace=s["workspace"])
        return {"out": out, "lse": lse}
    return nv.linear(s["codes"], s["scales"], s["alpha"], c["rows"], c["cols"], s["x"], bias=s["bias"],
                     activation=c["act"], gate=s["gate"], residual=s["residual"], workspace=s["workspace"])


# --------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "linear":
        n, out = c["rows"] * c["cols"], c["batch"] * c["rows"]
        extra = 2 * c["rows"] * bool(c["bias"]) + 2 * out * (bool(c["gate"]) + bool(c["residual"]))
        return {"bytes": n // 2 + n // 16 + 2 * c["batch"] * c["cols"] + 2 * out + extra,
                "flops": 2.0 * n * c["batch"]}
    size = 2 if c["cache"] == "bf16" else 1
    if c["op"] == "append":
        t, hq, hk, d = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
        distinct = len(set(_tokens(c)[1]))
        return {"bytes": t * (hq + 2 * hk) * d * (2 if c["input"] == "bf16" else 4) + t * hq * d * 2 +
                t * 2 * hk * d * size + distinct * c["rotary"] * 4 + t * 12,
                "flops": 3.0 * t * (hq + hk) * c["rotary"]}
    seen = sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
    q = c["sequences"] * c["q_heads"] * c["head_dim"]
    return {"bytes": 2 * seen * c["kv_heads"] * c["head_dim"] * size + 4 * q + 4 * c["sequences"] * c["q_heads"],
            "flops": 4.0 * seen * c["q_heads"] * c["head_dim"]}


# -------------------------------------------------------------------- exact

def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    hq, hk, d, r = case["q_heads"], case["kv_heads"], case["head_dim"], case["rotary"]
    heads = s["qkv"].double().reshape(case["tokens"], hq + 2 * hk, d)
    turned = heads.clone()
    first = torch.arange(r // 2, device=heads.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else r // 2)
    angle = s["cos_sin"].double().index_select(0, s["pos"].long()).unsqueeze(1)
    z = torch.complex(heads[:, :hq + hk, first], heads[:, :hq + hk, second]) * \
        torch.complex(angle[..., :r // 2], angle[..., r // 2:])
    turned[:, :hq + hk, first], turned[:, :hq + hk, second] = z.real, z.imag
    where = s["table"].long().gather(0, s["seq"].long()[:, None].expand(-1, s["table"].shape[1]))
    slot = where.gather(1, (s["pos"].long() // case["page"])[:, None])[:, 0] * case["page"] + s["pos"].long() % case["page"]
    result = {"q": turned[:, :hq]}
    for name, part in (("k", turned[:, hq:hq + hk]), ("v", turned[:, hq + hk:])):
        flat = s[name].double().transpose(1, 2).reshape(-1, hk, d)
        if case["cache"] == "e4m3":
            part = torch.clamp(part / s[name + "_scale"].double()[None, :, None], -448, 448)
        flat.index_copy_(0, slot, part)
        result[name] = flat.view(-1, case["page"], hk, d).transpose(1, 2)
    return result


def _exact_attend(case, seed):
    if work(case)["flops"] > 7e12:
        return None
    s = _prepare_attend(case, seed)
    hk, g, d = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["head_dim"]
    outs, sums = [], []
    for i, n in enumerate(_lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            outs.append(torch.zeros(hk * g, d, dtype=torch.float64, device=DEVICE))
            sums.append(torch.full((hk * g,), -math.inf, dtype=torch.float64, device=DEVICE))
            continue
        p0 = lo // case["page"]
        ids = s["table"][i, p0:-(-n // case["page"])].long()
        kv = []
        for name in ("k", "v"):
            x = s[name].index_select(0, ids) if case["cache"] == "bf16" else \
                s[name].view(torch.uint8).index_select(0, ids).view(torch.float8_e4m3fn)
            x = x.permute(1, 0, 2, 3).reshape(hk, -1, d)[:, lo - p0 * case["page"]:n - p0 * case["page"]].double()
            kv.append(x if s[name + "_scale"] is None else x * s[name + "_scale"].double()[:, None, None])
        score = torch.bmm(s["q"][i].double().view(hk, g, d), kv[0].transpose(1, 2)) * s["scale"]
        sums.append(torch.logsumexp(score, 2).view(-1))
        outs.append(torch.bmm(torch.softmax(score, 2), kv[1]).view(hk * g, d))
    return {"out": torch.stack(outs), "lse": torch.stack(sums)}


def _exact_linear(case, seed):
    s = _prepare_linear(case, seed)
    rows, cols = case["rows"], case["cols"]
    nib = torch.empty((rows, cols), dtype=torch.uint8, device=DEVICE)
    nib[:, 0::2], nib[:, 1::2] = s["codes"] % 16, s["codes"] // 16
    mag = nib % 8
    e, f = (mag // 2).double(), (mag % 2).double()
    w = torch.where(e > 0, torch.exp2(e - 1) * (1 + f / 2), f / 2) * (1 - 2 * (nib // 8).double())
    del nib, mag, e, f
    w = w * s["scales"].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * s["alpha"].double()
    v = s["x"].double() @ w.T
    if case["bias"]:
        v += s["bias"].double()
    f = torch.nn.functional
    v = {"none": lambda t: t, "relu": torch.relu, "gelu": f.gelu, "silu": f.silu,
         "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[case["act"]](v)
    if case["gate"]:
        v = v * s["gate"].double()
    return v + s["residual"].double() if case["residual"] else v


def exact(case, seed):
    return {"append": _exact_append, "attend": _exact_attend, "linear": _exact_linear}[case["op"]](case, seed)
