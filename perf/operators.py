"""The decoder-block operators next to ShortConv, as a serving program calls them: the residual
stream's addition with RMSNorm (and its 8-bit output), the expert router, and the experts'
products.

Each case is one call. ``run`` computes it in plain torch, or through
``encoder_free_audio_b200.dmel`` where ``own`` is set; ``exact`` evaluates the definition in
64 bits.
"""
import torch

own = False

DEV = "cuda"
_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------- cases

def _norm(name, rows, dim, dtype, out, block=0, residual=True):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "out": out, "block": block,
            "residual": residual}


def _route(name, tokens, experts, shared, top_k, scoring, dtype="f32", bias=True, groups=1, topk_groups=1,
           renormalise=True, scale=1.0):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "shared": shared, "top_k": top_k,
            "scoring": scoring, "dtype": dtype, "bias": bias, "groups": groups, "topk_groups": topk_groups,
            "renormalise": renormalise, "scale": scale}


def _experts(name, tokens, slots, experts, dim, hidden):
    return {"name": name, "op": "experts", "tokens": tokens, "slots": slots, "experts": experts, "dim": dim,
            "hidden": hidden}


def listed():
    return [
        # a decode step of 8 requests at the model width: latency
        _norm("norm_step8", 8, 6144, "bf16", "bf16"),
        # a 20-minute clip's 24,000 frames as one prompt: the largest stream
        _norm("norm_long20min", 24000, 6144, "bf16", "bf16"),
        # the 64 x 10 s batch (12,800 frames) normed into e4m3 rows for an 8-bit product
        _norm("norm_batch64_e4m3", 12800, 6144, "bf16", "e4m3", block=128),
        # fp32 stream, odd sizes: a last block of 104 columns
        _norm("norm_f32_odd", 1601, 5992, "f32", "e4m3", block=128),
        # a decode step of 64 requests: 256 routed experts and 2 shared, top 6 (the pages' router)
        _route("route_step64", 64, 256, 2, 6, "sigmoid"),
        # the 20-minute prompt through the same router
        _route("route_long20min", 24000, 256, 2, 6, "sigmoid"),
        # group-limited softmax routing of bf16 logits on the 12,800-frame batch
        _route("route_groups", 12800, 256, 0, 8, "softmax", dtype="bf16", groups=8, topk_groups=4, scale=2.5),
        # few experts, an odd number of tokens, weights as the softmax gives them
        _route("route_odd", 4097, 60, 0, 4, "softmax", bias=False, renormalise=False),
        # one token through 6 of 32 experts at the model width: bound by the experts' weights
        _experts("experts_token", 1, 6, 32, 6144, 1024),
        # a decode step of 64 requests: every expert is read, with a few tokens each
        _experts("experts_step64", 64, 6, 32, 6144, 1024),
        # a prompt of 4,096 tokens: bound by the products
        _experts("experts_prompt", 4096, 6, 32, 6144, 1024),
        # odd sizes: nothing a multiple of a tile
        _experts("experts_odd", 777, 3, 7, 2056, 520),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "route", "experts"])
    if op == "norm":
        dim = 8 * _between(rng, 8, 1024)
        out = rng.choice(["f32", "bf16", "e4m3", "e4m3"])
        case = _norm("", _between(rng, 1, min(24000, 24000 * 6144 // dim)), dim, rng.choice(["f32", "bf16", "bf16"]), out,
                     block=rng.choice([0, 32, 64, 128]) if out == "e4m3" else 0, residual=rng.random() < 0.75)
        if case["dtype"] == "f32":
            case["rows"] = max(1, case["rows"] // 2)
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _between(rng, 4, 256 // groups)
        experts = groups * per
        topk_groups = rng.randint(1, groups)
        case = _route("", _between(rng, 1, 24000), experts, rng.choice([0, 0, 1, 2, 3]),
                      rng.randint(1, min(12, topk_groups * per)), rng.choice(["softmax", "sigmoid"]),
                      dtype=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.6, groups=groups, topk_groups=topk_groups,
                      renormalise=rng.random() < 0.75, scale=rng.choice([1.0, 2.5]))
    else:
        experts = _between(rng, 2, 32)
        dim, hidden = 8 * _between(rng, 32, 768), 8 * _between(rng, 16, 128)
        slots = rng.randint(1, min(8, experts))
        case = _experts("", 1, slots, experts, dim, hidden)
        case["tokens"] = _between(rng, 1, min(4096, int(4096 * 6 * 6144 * 1024 / (slots * dim * hidden))))
    del case["name"]
    return case


def work(case):
    if case["op"] == "norm":
        n, es = case["rows"] * case["dim"], {"f32": 4, "bf16": 2, "e4m3": 1}
        blocks = case["rows"] * (-(-case["dim"] // case["block"]) if case["block"] else 1) if case["out"] == "e4m3" else 0
        streams = es[case["dtype"]] * (3 if case["residual"] else 1) + es[case["out"]]
        return {"bytes": n * streams + 4 * blocks + case["dim"] * es[case["dtype"]], "flops": 6 * n}
    if case["op"] == "route":
        cols, slots = case["experts"] + case["shared"], case["top_k"] + case["shared"]
        return {"bytes": case["tokens"] * (cols * (4 if case["dtype"] == "f32" else 2) + 8 * slots) + 4 * case["experts"],
                "flops": case["tokens"] * cols * 8}
    rows = case["tokens"] * case["slots"]
    # the experts that any slot chose, at most; each one's weights read once
    used = case["experts"] * (1.0 - (1.0 - case["slots"] / case["experts"]) ** case["tokens"])
    weights = used * 3 * case["dim"] * case["hidden"] * 2
    return {"bytes": weights + case["tokens"] * case["dim"] * 4 + rows * 8, "flops": 6 * rows * case["dim"] * case["hidden"]}


# ------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=g)

    s = dict(case)
    if case["op"] == "norm":
        n, d, dt = case["rows"], case["dim"], _DT[case["dtype"]]
        # branch outputs smaller than the stream, whose rows differ in size; a few large channels
        s["x"] = (0.3 * normal(n, d)).to(dt)
        s["r"] = (normal(n, d) * torch.exp(normal(n, 1)) * torch.exp(0.5 * normal(1, d))).to(dt) if case["residual"] else None
        s["w"] = (1.0 + normal(d, scale=0.1)).to(dt)
        s["r_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["out"] = torch.empty((n, d), dtype=_DT[case["out"]], device=DEV)
        blocks = -(-d // case["block"]) if case["block"] else 1
        s["scales"] = torch.empty((n, blocks), dtype=torch.float32, device=DEV) if case["out"] == "e4m3" else None
    elif case["op"] == "route":
        n, e, k = case["tokens"], case["experts"], case["top_k"] + case["shared"]
        s["logits"] = (1.5 * normal(n, e + case["shared"]) + 0.5 * normal(1, e + case["shared"])).to(_DT[case["dtype"]])
        s["bias"] = normal(e, scale=0.05) if case["bias"] else None
        s["ids"] = torch.empty((n, k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((n, k), dtype=torch.float32, device=DEV)
    else:
        n, k, e, d, h = case["tokens"], case["slots"], case["experts"], case["dim"], case["hidden"]
        s["x"] = normal(n, d, dtype=torch.bfloat16)
        s["w_in"] = normal(e, d, 2 * h, scale=d ** -0.5, dtype=torch.bfloat16)
        s["w_out"] = normal(e, h, d, scale=h ** -0.5, dtype=torch.bfloat16)
        # some experts are liked more than others; a token's experts differ
        top = torch.topk(normal(n, e) + 0.5 * normal(1, e), k, dim=1)
        s["ids"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(top.values, dim=1)
        s["out"] = torch.empty((n, d), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------------------------- passes

def run(state):
    s = state
    if own:
        return _RUN_OWN[s["op"]](s)
    return _RUN_PLAIN[s["op"]](s)


def _own_norm(s):
    from encoder_free_audio_b200 import dmel
    dmel.dmel_add_rmsnorm(s["x"], s["w"], s["out"], residual=s["r"], residual_out=s["r_out"], eps=1e-6,
                          scales=s["scales"], scale_block=s["block"])
    return {"stream": s["r_out"], "out": s["out"], "scales": s["scales"]}


def _own_route(s):
    from encoder_free_audio_b200 import dmel
    scoring = dmel.DMEL_ROUTE_SIGMOID if s["scoring"] == "sigmoid" else dmel.DMEL_ROUTE_SOFTMAX
    dmel.dmel_route(s["logits"], s["ids"], s["weights"], n_shared=s["shared"], bias=s["bias"], scoring=scoring,
                    n_groups=s["groups"], topk_groups=s["topk_groups"], renormalise=s["renormalise"], scale=s["scale"])
    return {"ids": s["ids"], "weights": s["weights"]}


def _own_experts(s):
    from encoder_free_audio_b200 import dmel
    if "workspace" not in s:  # kept beside the buffers, as a serving program does
        n = dmel.dmel_experts_workspace_size(s["tokens"], s["slots"], s["experts"], s["dim"], s["hidden"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    dmel.dmel_experts(s["x"], s["ids"], s["weights"], s["w_in"], s["w_out"], s["out"], s["workspace"])
    return {"out": s["out"]}


def _plain_norm(s):
    v = s["x"].float()
    stream = None
    if s["r"] is not None:
        v = v + s["r"].float()
        stream = v.to(s["x"].dtype)
    y = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + 1e-6) * s["w"].float()
    if s["out"].dtype != torch.float8_e4m3fn:
        return {"stream": stream, "out": y.to(s["out"].dtype), "scales": None}
    n, d = y.shape
    block = s["block"] or d
    blocks = -(-d // block)
    padded = torch.zeros((n, blocks * block), dtype=torch.float32, device=y.device)
    padded[:, :d] = y
    padded = padded.view(n, blocks, block)
    scales = padded.abs().amax(dim=2).clamp(min=1e-30) / 448.0
    q = (padded / scales.unsqueeze(2)).view(n, blocks * block)[:, :d].clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return {"stream": stream, "out": q, "scales": scales}


def _plain_route(s):
    # in 64 bits: experts next to the border between chosen and not are as far apart as they are
    e, k = s["experts"], s["top_k"]
    logits = torch.nan_to_num(s["logits"].double(), nan=-torch.inf, posinf=torch.finfo(torch.float32).max, neginf=-torch.inf)
    if s["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-logits))
    else:
        top = logits.amax(dim=1, keepdim=True)
        score = torch.exp(logits - torch.where(top > -torch.inf, top, 0.0))
        score = score / score.sum(dim=1, keepdim=True).clamp(min=1e-300)
    routed = logits[:, :e]
    choice = score[:, :e] if s["bias"] is None else score[:, :e] + s["bias"].double()
    choice = torch.where(routed > -torch.inf, choice, -torch.inf)
    key = torch.where(routed > -torch.inf, routed, -torch.inf) if s["bias"] is None else choice
    if s["groups"] > 1:
        n, groups = choice.shape[0], s["groups"]
        two = torch.sort(choice.view(n, groups, e // groups), dim=2, descending=True).values[:, :, :2]
        rated = torch.where(two > -torch.inf, two, 0.0).sum(dim=2)
        rated = torch.where(two[:, :, 0] > -torch.inf, rated, -torch.inf)
        best = torch.sort(rated, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        kept = torch.zeros((n, groups), dtype=torch.bool, device=key.device).scatter_(1, best, True)
        key = torch.where(kept.repeat_interleave(e // groups, dim=1), key, -torch.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids, there = order.indices[:, :k], order.values[:, :k] > -torch.inf
    weights = torch.where(there, score.gather(1, ids), 0.0)
    ids = torch.where(there, ids, -1)
    if s["shared"]:
        shared = torch.arange(e, e + s["shared"], device=ids.device).expand(ids.shape[0], -1)
        ids = torch.cat([ids, torch.where(logits[:, e:] > -torch.inf, shared, -1)], dim=1)
        weights = torch.cat([weights, score[:, e:]], dim=1)
    if s["renormalise"]:
        weights = weights / weights.sum(dim=1, keepdim=True).clamp(min=1e-300)
    return {"ids": ids.to(torch.int32), "weights": (weights * s["scale"]).float()}


def _plain_experts(s):
    # the chosen experts' rows padded to the longest expert, two batched products in 32 bits
    n, k = s["ids"].shape
    d = s["x"].shape[1]
    used, which, counts = torch.unique(s["ids"].flatten(), return_inverse=True, return_counts=True)
    longest = int(counts.max())
    order = torch.argsort(which, stable=True)
    first = torch.cumsum(counts, 0) - counts
    place = torch.empty_like(which)
    place[order] = torch.arange(n * k, device=which.device) - first[which[order]] + which[order] * longest
    rows = torch.zeros((used.numel() * longest, d), dtype=torch.float32, device=which.device)
    rows[place] = s["x"].float().repeat_interleave(k, dim=0)
    used = used.long()
    hidden = torch.bmm(rows.view(used.numel(), longest, d), s["w_in"][used].float())
    gate, up = hidden.chunk(2, dim=2)
    y = torch.bmm(gate / (1.0 + torch.exp(-gate)) * up, s["w_out"][used].float()).view(-1, d)[place]
    y = (y.view(n, k, d) * s["weights"].unsqueeze(2)).sum(dim=1)
    return {"out": y.to(torch.bfloat16)}


_RUN_OWN = {"norm": _own_norm, "route": _own_route, "experts": _own_experts}
_RUN_PLAIN = {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts}


# ------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "experts": _exact_experts}[case["op"]](s)


def _exact_norm(s):
    n, d = s["x"].shape
    outs, scales, streams = [], [], []
    for a in range(0, n, 4096):
        v = s["x"][a:a + 4096].double()
        if s["r"] is not None:
            v = v + s["r"][a:a + 4096].double()
            streams.append(v)
        y = v * s["w"].double() * (v.square().sum(1, keepdim=True) / d + 1e-6) ** -0.5
        if s["scales"] is not None:
            step = s["block"] or d
            parts = [y[:, c:c + step] for c in range(0, d, step)]
            sc = [p.abs().max(1, keepdim=True).values.clamp(min=1e-30) / 448.0 for p in parts]
            y = torch.cat([p / q for p, q in zip(parts, sc)], 1)
            scales.append(torch.cat(sc, 1))
        outs.append(y)
    return {"stream": torch.cat(streams) if streams else None, "out": torch.cat(outs),
            "scales": torch.cat(scales) if scales else None}


def _exact_route(s):
    # every expert's place is the number of experts that come before it
    n, e, k, groups = s["logits"].shape[0], s["experts"], s["top_k"], s["groups"]
    found = []
    for a in range(0, n, 1024):
        l = s["logits"][a:a + 1024].double()
        log_score = -torch.log1p(torch.exp(-l)) if s["scoring"] == "sigmoid" else l - torch.logsumexp(l, 1, keepdim=True)
        c = log_score[:, :e].exp() + (0.0 if s["bias"] is None else s["bias"].double())
        lower = torch.arange(e, device=l.device)

        def place(v, index):
            before = (v.unsqueeze(1) > v.unsqueeze(2)) | ((v.unsqueeze(1) == v.unsqueeze(2)) & (index[None, :] < index[:, None]))
            return before.sum(2)

        if groups > 1:
            rated = torch.topk(c.view(-1, groups, e // groups), min(2, e // groups), dim=2).values.sum(2)
            kept = place(rated, lower[:groups]) < s["topk_groups"]
            c = c.masked_fill(~kept.repeat_interleave(e // groups, 1), -torch.inf)
        at = place(c, lower)
        chosen = torch.stack([(at == j).to(torch.int8).argmax(1) for j in range(k)], 1)
        lw = log_score.gather(1, chosen)
        lw = torch.cat([lw, log_score[:, e:]], 1)
        if s["renormalise"]:
            lw = lw - torch.logsumexp(lw, 1, keepdim=True)
        found.append(lw.exp() * s["scale"])
    return {"ids": None, "weights": torch.cat(found)}


def _exact_experts(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    h = s["hidden"]
    for e in range(s["experts"]):
        token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if token.numel() == 0:
            continue
        a = s["x"][token].double() @ s["w_in"][e].double()
        y = (a[:, :h] * torch.sigmoid(a[:, :h]) * a[:, h:]) @ s["w_out"][e].double()
        out.index_add_(0, token, y * s["weights"][token, slot].double().unsqueeze(1))
    return {"out": out}
