"""Cases of what follows attention in a decode step: moe_route (the router of a
mixture-of-experts layer), moe (its experts' products on NVFP4 weights) and
sample (the next token from logits).

`run` computes an operator either in plain torch operations (own = False) or
through the framework's entry points (own = True) on what `prepare` made;
`exact` computes the same outputs in 64 bits.
"""
import math
import random

import torch

if torch.cuda.is_available():
    DEVICE = torch.device("cuda")
else:
    DEVICE = torch.device("cpu")

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def _route(name, tokens, hidden, experts, top_k, scoring, renormalize, router):
    return {"name": name, "op": "route", "tokens": tokens, "hidden": hidden, "experts": experts, "top_k": top_k,
            "scoring": scoring, "renormalize": renormalize, "router": router}


def _moe(name, tokens, padding, hidden, inner, experts, top_k, act, gated, residual):
    return {"name": name, "op": "moe", "tokens": tokens, "padding": padding, "hidden": hidden, "inner": inner,
            "experts": experts, "top_k": top_k, "act": act, "gated": gated, "residual": residual}


def _sample(name, rows, vocabulary, dtype, temperature, top_k, top_p, min_p, masked, mixed):
    return {"name": name, "op": "sample", "rows": rows, "vocabulary": vocabulary, "dtype": dtype,
            "temperature": temperature, "top_k": top_k, "top_p": top_p, "min_p": min_p, "masked": masked,
            "mixed": mixed}


def listed():
    return [
        # one user's token among many small experts: latency
        _route("route 1 x 2048, 8 of 128", 1, 2048, 128, 8, "softmax", True, "bf16"),
        # an odd decode batch over few large experts, the softmax over all of them
        _route("route 61 x 4096, 2 of 8", 61, 4096, 8, 2, "softmax", False, "fp32"),
        # the largest decode batch over the most experts, sigmoid scores with a selection bias
        _route("route 256 x 7168, 8 of 256 sigmoid", 256, 7168, 256, 8, "sigmoid", True, "bf16"),
        # one user's token: eight small experts out of 128, latency
        _moe("moe 1 x 2048 x 768, 8 of 128", 1, 0, 2048, 768, 128, 8, "silu", True, False),
        # a handful of users, two of eight large experts, with the residual stream
        _moe("moe 5 x 4096 x 14336, 2 of 8", 5, 0, 4096, 14336, 8, 2, "silu", True, True),
        # an odd decode batch padded to its captured size: nearly every expert has a few tokens
        _moe("moe 61 x 2048 x 768, 8 of 128", 61, 3, 2048, 768, 128, 8, "silu", True, True),
        # the largest decode batch, experts without a gate, sizes that no tile divides
        _moe("moe 256 x 2064 x 1424, 6 of 60 gelu", 256, 0, 2064, 1424, 60, 6, "gelu", False, False),
        # the largest weights: most of 256 wide experts named by some token
        _moe("moe 33 x 7168 x 2048, 8 of 256", 33, 0, 7168, 2048, 256, 8, "silu", True, False),
        # one user, the usual settings together: latency
        _sample("sample 1 x 32000 bf16", 1, 32000, "bf16", 0.8, 50, 0.9, 0.0, 0.0, False),
        # an odd batch of users with settings of their own, greedy ones among them, some tokens masked by a grammar
        _sample("sample 61 x 128256 bf16 mixed", 61, 128256, "bf16", 1.0, 100, 0.95, 0.05, 0.5, True),
        # few rows of a large vocabulary in fp32, top-p alone: the mass of every token counts
        _sample("sample 7 x 262144 fp32 top-p", 7, 262144, "fp32", 1.0, 0, 0.9, 0.0, 0.0, False),
        # the largest batch, an odd vocabulary, every token a candidate
        _sample("sample 256 x 151003 fp32", 256, 151003, "fp32", 1.3, 0, 1.0, 0.02, 0.1, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(("route", "moe", "moe", "sample", "sample"))
    experts = rng.choice((4, 8, 16, 32, 60, 64, 128, 256))
    top_k = min(experts, rng.choice((1, 2, 4, 6, 8, 8)))
    if kind == "route":
        c = _route("", _log_int(rng, 1, 256), 16 * _log_int(rng, 16, 448), experts, top_k,
                   rng.choice(("softmax", "sigmoid")), rng.random() < 0.6, rng.choice(("bf16", "fp32")))
    elif kind == "moe":
        while True:
            tokens, hidden, inner = _log_int(rng, 1, 256), 16 * _log_int(rng, 16, 448), 16 * _log_int(rng, 8, 896)
            if experts * hidden * inner <= 256 * 7168 * 2048 and tokens * top_k * hidden * inner <= 264 * 7168 * 2048:
                break
        c = _moe("", tokens, rng.choice((0, 0, tokens // 9)), hidden, inner, experts, top_k,
                 rng.choice(("silu", "silu", "relu", "gelu", "gelu_tanh")), rng.random() < 0.8, rng.random() < 0.5)
    else:
        while True:
            rows, vocabulary = _log_int(rng, 1, 256), _log_int(rng, 1000, 262144)
            if rows * vocabulary <= 256 * 151003:
                break
        c = _sample("", rows, vocabulary, rng.choice(("bf16", "fp32")), rng.choice((0.0, 0.5, 0.8, 1.0, 1.3)),
                    rng.choice((0, 0, _log_int(rng, 1, 1000))), rng.choice((1.0, 0.95, 0.9, 0.5)),
                    rng.choice((0.0, 0.0, 0.02, 0.1)), rng.choice((0.0, 0.1, 0.9)), rng.random() < 0.5)
    del c["name"]
    return c


def _assignment(case):
    """The experts of every token: distinct ones, some experts more popular than others; -1 in padding tokens."""
    rng = random.Random(case["tokens"] * 1000003 + case["experts"] * 1009 + case["top_k"])
    weight = [math.exp(0.7 * rng.gauss(0.0, 1.0)) for _ in range(case["experts"])]
    out = []
    for t in range(case["tokens"]):
        key = [(-math.log(1.0 - rng.random()) / w, e) for e, w in enumerate(weight)]
        out.append([e for _, e in sorted(key)[:case["top_k"]]])
    for t in range(case["tokens"] - case["padding"], case["tokens"]):
        out[t] = [-1] * case["top_k"]
    return out


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEVICE)


def _prepare_route(case, seed):
    g = _generator(seed)
    h, e = case["hidden"], case["experts"]
    s = {"case": case}
    s["x"] = _randn(g, case["tokens"], h).to(torch.bfloat16)
    s["router"] = (1.5 * h ** -0.5 * _randn(g, e, h)).to(TYPES[case["router"]])
    s["bias"] = 0.1 * _randn(g, e) if case["scoring"] == "sigmoid" else None
    s["scale"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
    return s


def _matrices(g, experts, rows, cols):
    """Codes, scales and alphas of `experts` matrices whose entries have a variance of about 1 / cols."""
    codes = torch.randint(0, 256, (experts, rows, cols // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    scales = torch.randint(80, 112, (experts, rows, cols // 16), generator=g, device=DEVICE, dtype=torch.uint8)
    alpha = (0.8 + 0.4 * torch.rand(experts, generator=g, device=DEVICE)) * cols ** -0.5 / 170.0
    return codes, scales, alpha


def _prepare_moe(case, seed):
    g = _generator(seed)
    t, h, i, e, k = case["tokens"], case["hidden"], case["inner"], case["experts"], case["top_k"]
    s = {"case": case}
    s["gate"] = _matrices(g, e, i, h) if case["gated"] else None
    s["up"] = _matrices(g, e, i, h)
    s["down"] = _matrices(g, e, h, i)
    s["x"] = _randn(g, t, h).to(torch.bfloat16)
    label = torch.randperm(e, generator=g, device=DEVICE).to(torch.int32)
    ids = torch.tensor(_assignment(case), dtype=torch.int32, device=DEVICE).view(t, k)
    s["ids"] = torch.where(ids < 0, ids, label[ids.clamp(min=0).long()])
    w = 0.2 + torch.rand((t, k), generator=g, device=DEVICE)
    s["weights"] = w / w.sum(1, keepdim=True)
    s["residual"] = _randn(g, t, h).to(torch.bfloat16) if case["residual"] else None
    return s


def _prepare_sample(case, seed):
    g = _generator(seed)
    b, v = case["rows"], case["vocabulary"]
    s = {"case": case}
    logits = 2.0 * _randn(g, b, v)
    # the tokens that fit the context stand out by a few units, fewer the further
    at = torch.randint(0, v, (b, 60), generator=g, device=DEVICE)
    logits.scatter_add_(1, at, 4.0 - 3.0 * torch.log(torch.rand((b, 60), generator=g, device=DEVICE).clamp(min=1e-3)))
    if case["masked"] > 0:
        hidden = torch.rand((b, v), generator=g, device=DEVICE) < case["masked"]
        logits = torch.where(hidden, torch.full_like(logits, -math.inf), logits)
        if b > 2:
            logits[b // 2] = -math.inf  # a row that the mask leaves empty
    s["logits"] = logits.to(TYPES[case["dtype"]])
    s["uniform"] = torch.rand(b, generator=g, device=DEVICE)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        s[name] = case[name]
    if case["mixed"]:  # every user's own settings; some decode greedily, some leave a filter out
        r = torch.rand((4, b), generator=g, device=DEVICE)
        s["temperature"] = torch.where(r[0] < 0.15, torch.zeros_like(r[0]), case["temperature"] * (0.5 + r[0]))
        if case["top_k"]:
            s["top_k"] = torch.where(r[1] < 0.2, torch.zeros_like(r[1]), 1 + r[1] * 2 * case["top_k"]).to(torch.int32)
        if case["top_p"] < 1.0:
            s["top_p"] = torch.where(r[2] < 0.2, torch.ones_like(r[2]), 1.0 - 2 * (1.0 - case["top_p"]) * r[2])
        if case["min_p"]:
            s["min_p"] = torch.where(r[3] < 0.2, torch.zeros_like(r[3]), 2 * case["min_p"] * r[3])
    return s


def prepare(case, seed):
    s = {"route": _prepare_route, "moe": _prepare_moe, "sample": _prepare_sample}[case["op"]](case, seed)
    if own:  # the experts' handle and the workspace that a serving program keeps from step to step
        import nvfp4_block_scale_gb300 as nv
        s["nv"] = nv
        if case["op"] == "moe":
            s["experts"] = nv.Experts(s["up"], s["down"], s["gate"])
            s["workspace"] = nv.moe_workspace(s["experts"], case["tokens"], case["top_k"])
    return s


# ---------------------------------------------------------------- plain form

def _plain_route(s):
    c = s["case"]
    # 64 bits: two experts' scores may lie closer than 32 bits tell apart
    logit = torch.matmul(s["x"].double(), s["router"].double().t())
    if c["scoring"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-logit))
        score = p + s["bias"].double()
    else:
        e = torch.exp(logit - logit.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        score = logit
    order = torch.sort(score, dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = torch.gather(p, 1, order)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": order.to(torch.int32), "weights": (w * s["scale"]).float()}


def _activate(v, act):
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v / (1.0 + torch.exp(-v))


def _expert(weights, e, value):
    codes, scales, alpha = (w[e] for w in weights)
    rows, half = codes.shape
    q = torch.stack((value[(codes & 15).int()], value[(codes >> 4).int()]), -1).view(rows, half // 8, 16)
    return (q * scales.view(torch.float8_e4m3fn).float()[..., None]).view(rows, 2 * half), alpha


def _plain_moe(s):
    c = s["case"]
    value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=s["x"].device)
    x, k = s["x"].float(), c["top_k"]
    part = torch.zeros((c["tokens"] * k, c["hidden"]), device=x.device)
    named = s["ids"].flatten().tolist()
    for e in sorted(set(named)):
        if e < 0:
            continue
        pairs = torch.tensor([i for i, n in enumerate(named) if n == e], device=x.device)
        xe = x[pairs // k]
        w, a = _expert(s["up"], e, value)
        h = torch.matmul(xe, w.t()) * a
        if s["gate"] is not None:
            w, a = _expert(s["gate"], e, value)
            h = _activate(torch.matmul(xe, w.t()) * a, c["act"]) * h
        else:
            h = _activate(h, c["act"])
        w, a = _expert(s["down"], e, value)
        part[pairs] = torch.matmul(h, w.t()) * a
    y = (part.view(c["tokens"], k, -1) * s["weights"][..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _column(v, rows, device, kind):
    if isinstance(v, torch.Tensor):
        return v.to(kind)[:, None]
    return torch.full((rows, 1), v, dtype=kind, device=device)


def _plain_sample(s):
    x = s["logits"]
    b, v = x.shape
    t, p, low = (_column(s[n] if isinstance(s[n], torch.Tensor) else torch.tensor(s[n], dtype=torch.float32).item(),
                         b, x.device, torch.float64) for n in ("temperature", "top_p", "min_p"))
    k = _column(s["top_k"], b, x.device, torch.int64)
    x, order = torch.sort(x.float(), dim=1, descending=True, stable=True)
    top = x[:, :1].double()
    alive = x > -math.inf
    # sums over a vocabulary, and values next to a cut: 64 bits
    w = torch.where(alive, torch.exp((x.double() - top) / torch.where(t > 0, t, torch.ones_like(t))), 0.0)
    keep = alive & ((k <= 0) | (torch.arange(v, device=x.device) < k))
    w = torch.where(keep, w, 0.0)
    upto = torch.cumsum(w, 1)
    before = torch.cat((torch.zeros_like(upto[:, :1]), upto[:, :-1]), 1)
    keep = keep & ((p >= 1) | (before < p * upto[:, -1:])) & (w >= low)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    upto = torch.cumsum(w, 1)
    goal = s["uniform"].double()[:, None] * upto[:, -1:]
    token = torch.where((upto > goal) & (w > 0), torch.arange(v, device=x.device), v).amin(1).clamp(max=v - 1)
    token = torch.where(t[:, 0] > 0, token, order[:, 0])
    chance = torch.gather(w, 1, token[:, None])[:, 0] / upto[:, -1]
    chance = torch.where(t[:, 0] > 0, chance, torch.ones_like(chance))
    return {"token": torch.where(alive[:, 0], token, -1).to(torch.int32),
            "logprob": torch.log(torch.where(alive[:, 0], chance, 0.0)).float()}


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"route": _plain_route, "moe": _plain_moe, "sample": _plain_sample}[c["op"]](s)
    nv = s["nv"]
    if c["op"] == "route":
        ids, weights = nv.moe_route(s["x"], s["router"], c["top_k"], scoring=c["scoring"], renormalize=c["renormalize"],
                                    bias=s["bias"], scale=s["scale"])
        return {"ids": ids, "weights": weights}
    if c["op"] == "moe":
        return nv.moe(s["experts"], s["x"], s["ids"], s["weights"], activation=c["act"], residual=s["residual"],
                      workspace=s["workspace"])
    token, logprob = nv.sample(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                               top_p=s["top_p"], min_p=s["min_p"], return_logprob=True)
    return {"token": token, "logprob": logprob}


# --------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "route":
        t, h, e = c["tokens"], c["hidden"], c["experts"]
        return {"bytes": 2 * t * h + (2 if c["router"] == "bf16" else 4) * e * h + 8 * t * c["top_k"] +
                4 * e * (c["scoring"] == "sigmoid"), "flops": 2.0 * t * e * h}
    if c["op"] == "moe":
        named = [e for token in _assignment(c) for e in token if e >= 0]
        n = (3 if c["gated"] else 2) * c["hidden"] * c["inner"]
        t = c["tokens"] - c["padding"]
        out = c["tokens"] * c["hidden"]
        return {"bytes": len(set(named)) * (n // 2 + n // 16 + 4) + 2 * t * c["hidden"] +
                (4 if c["residual"] else 2) * out + 8 * c["tokens"] * c["top_k"], "flops": 2.0 * n * len(named)}
    n = c["rows"] * c["vocabulary"]
    return {"bytes": (2 if c["dtype"] == "bf16" else 4) * n + (28 if c["mixed"] else 12) * c["rows"], "flops": 5.0 * n}


# -------------------------------------------------------------------- exact

def _exact_route(case, seed):
    s = _prepare_route(case, seed)
    ids, weights = [], []
    r = s["router"].double()
    for row in s["x"].double():
        logit = (r * row).sum(1)
        score = torch.sigmoid(logit) + s["bias"].double() if case["scoring"] == "sigmoid" else logit
        score = score.tolist()
        best = sorted(range(case["experts"]), key=lambda e: (-score[e], e))[:case["top_k"]]
        p = torch.sigmoid(logit) if case["scoring"] == "sigmoid" else torch.softmax(logit, 0)
        w = p[best]
        ids.append(torch.tensor(best, dtype=torch.int32, device=DEVICE))
        weights.append(s["scale"] * (w / w.sum() if case["renormalize"] else w))
    return {"ids": torch.stack(ids), "weights": torch.stack(weights)}


def _exact_matrix(codes, scales, alpha):
    nib = torch.stack((codes % 16, codes // 16), -1).flatten(1)
    mag = nib % 8
    e, f = (mag // 2).double(), (mag % 2).double()
    w = torch.where(e > 0, torch.exp2(e - 1) * (1 + f / 2), f / 2) * (1 - 2 * (nib // 8).double())
    return w * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * alpha.double()


def _exact_moe(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = _prepare_moe(case, seed)
    f = torch.nn.functional
    act = {"relu": torch.relu, "gelu": f.gelu, "silu": f.silu, "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[case["act"]]
    x = s["x"].double()
    y = s["residual"].double() if case["residual"] else torch.zeros_like(x)
    for e in range(case["experts"]):
        token, slot = torch.where(s["ids"] == e)
        if len(token) == 0:
            continue
        u = x[token] @ _exact_matrix(*(w[e] for w in s["up"])).T
        h = act(x[token] @ _exact_matrix(*(w[e] for w in s["gate"])).T) * u if case["gated"] else act(u)
        o = h @ _exact_matrix(*(w[e] for w in s["down"])).T
        y.index_add_(0, token, o * s["weights"][token, slot].double()[:, None])
    return y


def _exact_sample(case, seed):
    s = _prepare_sample(case, seed)
    b = case["rows"]
    single = {n: torch.as_tensor(s[n], device=DEVICE).float().expand(b).tolist() for n in ("temperature", "top_p", "min_p")}
    top_k = torch.as_tensor(s["top_k"], device=DEVICE).expand(b).tolist()
    uniform, tokens, chances = s["uniform"].tolist(), [], []
    for i in range(b):
        x = s["logits"][i].double()
        at = torch.nonzero(x > -math.inf)[:, 0]
        x = x[at]
        if len(at) == 0:
            tokens.append(-1)
            chances.append(-math.inf)
            continue
        if single["temperature"][i] <= 0:
            tokens.append(int(at[x == x.max()][0]))
            chances.append(0.0)
            continue
        w = ((x - x.max()) / single["temperature"][i]).exp()
        place = torch.argsort(x, descending=True, stable=True)
        if top_k[i] > 0:
            place = place[:top_k[i]]
        mass = w[place].cumsum(0)
        n = len(place)
        if single["top_p"][i] < 1.0:  # the first tokens up to the one that reaches top_p
            n = min(n, 1 + int((mass < single["top_p"][i] * mass[-1]).sum()))
        place = place[:n]
        place = torch.sort(place[w[place] >= single["min_p"][i]])[0]
        mass = w[place].cumsum(0)
        j = min(int((mass <= uniform[i] * mass[-1]).sum()), len(place) - 1)
        tokens.append(int(at[place[j]]))
        chances.append(float(w[place[j]].log() - mass[-1].log()))
    return {"token": torch.tensor(tokens, dtype=torch.int32, device=DEVICE),
            "logprob": torch.tensor(chances, dtype=torch.float64, device=DEVICE)}


def exact(case, seed):
    return {"route": _exact_route, "moe": _exact_moe, "sample": _exact_sample}[case["op"]](case, seed)
