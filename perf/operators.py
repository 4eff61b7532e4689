"""The operators around and inside the MoE layer that serving needs: their cases, inputs and plain forms.

Five operators:

* "route":   routing with a balance bias -- scores (sigmoid or softmax) plus a bias choose groups and experts,
             the scores alone give the gates;
* "norm":    the RMS norm of the residual stream in front of the layer;
* "product": int8 matrix product with a scale per token and per output channel over the experts' row groups,
             from the activations as the model holds them (quantised inside the call, after the norm where the
             case has one);
* "ffn":     the grouped SwiGLU FFN on int8 codes;
* "after":   the end of the block -- gate-weighted combine, norm, gate and scaled residual.

run() takes the plain torch form, or with `own` the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------------------------


def listed():
    return [
        # one decoded token through the router of a 256-expert layer with group-limited routing: pure latency
        dict(name="route 1 token, 256 experts, groups", op="route", tokens=1, experts=256, groups=8, keep=4, topn=2,
             k=8, score="sigmoid", renorm=True, scale=2.5, k_varies=False, offline=0),
        # a prefill batch of the same layer
        dict(name="route 8192 tokens, 256 experts, groups", op="route", tokens=8192, experts=256, groups=8, keep=4,
             topn=2, k=8, score="sigmoid", renorm=True, scale=2.5, k_varies=False, offline=0),
        # an odd-sized batch of a softmax router, k per request, three experts taken offline
        dict(name="route 16381 tokens, 128 experts, softmax", op="route", tokens=16381, experts=128, groups=1, keep=1,
             topn=1, k=8, score="softmax", renorm=True, scale=1.0, k_varies=True, offline=3),
        # a decode step's norm in front of the layer
        dict(name="norm 64 x 4096", op="norm", rows=64, hidden=4096, stream="bf16"),
        # a prefill chunk's norm, the residual stream held in fp32
        dict(name="norm 8192 x 7168, fp32 stream", op="norm", rows=8192, hidden=7168, stream="f32"),
        # a dense int8 projection of an odd decode batch straight after the norm
        dict(name="product 17 x 14336 x 4096 after the norm", op="product", rows=17, n=14336, k=4096, experts=1,
             norm=True, out="bf16"),
        # the down projection of a prefill chunk over eight experts
        dict(name="product 8192 x 4096 x 14336, 8 experts", op="product", rows=8192, n=4096, k=14336, experts=8,
             norm=False, out="f32"),
        # one decoded token through eight of 128 small experts
        dict(name="ffn 1 token, 128 experts", op="ffn", tokens=1, hidden=2048, inter=768, experts=128, k=8, out="f16"),
        # a decode step over eight large experts: their weights are read once
        dict(name="ffn 64 tokens, 8 experts", op="ffn", tokens=64, hidden=4096, inter=14336, experts=8, k=2,
             out="f16"),
        # a prefill chunk over 256 experts
        dict(name="ffn 8192 tokens, 256 experts", op="ffn", tokens=8192, hidden=7168, inter=2048, experts=256, k=8,
             out="f16"),
        # the end of a decode step's block: an odd batch, a learned gate per channel
        dict(name="after 33 x 4096, top 2", op="after", tokens=33, hidden=4096, k=2, y="f16", stream="bf16",
             shared=False, gate="channel", dropped=0.0, scale=1.0),
        # the end of a prefill chunk's block, shared expert, a gate per token and channel, a few dropped slots
        dict(name="after 8192 x 7168, top 8 and shared", op="after", tokens=8192, hidden=7168, k=8, y="f16",
             stream="bf16", shared=True, gate="both", dropped=0.02, scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "product", "ffn", "after"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log(rng, 4, 512 // groups)
        keep = rng.randint((groups + 1) // 2, groups)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=groups * size, groups=groups, keep=keep,
                    topn=rng.randint(1, min(3, size)), k=rng.randint(1, min(10, keep * size)),
                    score=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), k_varies=rng.random() < 0.3,
                    offline=rng.choice([0, 0, 1, 2]) if size > 8 else 0)
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 8192), hidden=64 * _log(rng, 4, 112), stream=rng.choice(["bf16", "f32"]))
    if op == "product":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 8192), n=16 * _log(rng, 16, 896), k=128 * _log(rng, 2, 112),
                     experts=_log(rng, 1, 64), norm=rng.random() < 0.4, out=rng.choice(["f32", "bf16", "f16"]))
            if c["experts"] * c["n"] * c["k"] <= 1 << 30 and c["rows"] * c["n"] * c["k"] <= 8192 * 4096 * 14336:
                c["out"] = "bf16" if c["norm"] and c["out"] == "f32" else c["out"]
                return c
    if op == "ffn":
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 8192), hidden=128 * _log(rng, 4, 56), inter=128 * _log(rng, 2, 112),
                     experts=_log(rng, 4, 256), k=rng.randint(1, 8), out="f16")
            c["k"] = min(c["k"], c["experts"] // 2)
            weights, rows = c["experts"] * c["hidden"] * c["inter"], c["tokens"] * c["k"]
            if weights <= 1 << 30 and rows * c["hidden"] * c["inter"] <= 32768 * 7168 * 2048:
                return c
    return dict(op=op, tokens=_log(rng, 1, 8192), hidden=64 * _log(rng, 4, 112), k=rng.randint(1, 8),
                y=rng.choice(["f32", "f16", "bf16"]), stream=rng.choice(["bf16", "f32"]), shared=rng.random() < 0.5,
                gate=rng.choice(["none", "channel", "token", "both"]), dropped=rng.choice([0.0, 0.02, 0.3]),
                scale=rng.choice([1.0, 0.5, 0.0]))


# ---- inputs ----------------------------------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _codes(gen, experts, n, k):
    """Weight codes as a per-channel quantisation of normal weights leaves them, and their scales."""
    w = torch.empty(experts, n, k, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for e in range(0, experts, step):
        part = w[e:e + step]
        part.copy_(_randn(gen, *part.shape).mul_(32.0).round_().clamp_(-127, 127))
    scales = (1 + 0.2 * torch.rand(experts, n, generator=gen, device="cuda")) / (32.0 * math.sqrt(k))
    return w, scales


def _row_groups(gen, tokens, k, experts):
    """Rows per expert of a routed batch with a mild skew: offsets [E + 1], and the largest group."""
    pull = 0.4 * _randn(gen, experts) - torch.log(-torch.log(torch.rand(tokens, experts, generator=gen, device="cuda")
                                                             .clamp_(1e-7, 1 - 1e-7)))
    ids = pull.topk(k, dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c, s = case, {"case": case}
    if c["op"] == "route":
        T, E = c["tokens"], c["experts"]
        s["logits"] = _randn(gen, T, E) + 0.5 * _randn(gen, E)
        s["bias"] = (0.05 if c["score"] == "sigmoid" else 0.3 / E) * _randn(gen, E)
        if c["offline"]:
            s["bias"][torch.randperm(E, generator=gen, device="cuda")[:c["offline"]]] = -math.inf
        s["k"] = (torch.randint(1, c["k"] + 1, (T,), generator=gen, device="cuda", dtype=torch.int32)
                  if c["k_varies"] else None)
    elif c["op"] == "norm":
        x = _randn(gen, c["rows"], c["hidden"]) * torch.exp(0.5 * _randn(gen, c["rows"], 1))
        s["x"] = x.to(DTYPES[c["stream"]])
        s["weight"] = 1 + 0.1 * _randn(gen, c["hidden"])
    elif c["op"] == "product":
        s["x"] = _randn(gen, c["rows"], c["k"]).to(torch.bfloat16)
        s["weight"] = 1 + 0.1 * _randn(gen, c["k"])
        s["w"], s["w_scales"] = _codes(gen, c["experts"], c["n"], c["k"])
        s["offsets"], s["most"] = _row_groups(gen, c["rows"], 1, c["experts"])
    elif c["op"] == "ffn":
        H, I, E, rows = c["hidden"], c["inter"], c["experts"], c["tokens"] * c["k"]
        s["x"] = (_randn(gen, rows, H) * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["x_scales"] = (1 + 0.2 * torch.rand(rows, generator=gen, device="cuda")) / 32
        s["gate"], s["gate_scales"] = _codes(gen, E, I, H)
        s["up"], s["up_scales"] = _codes(gen, E, I, H)
        s["down"], s["down_scales"] = _codes(gen, E, H, I)
        s["offsets"], s["most"] = _row_groups(gen, c["tokens"], c["k"], E)
    else:
        T, H, k = c["tokens"], c["hidden"], c["k"]
        s["y"] = _randn(gen, T * k, H).to(DTYPES[c["y"]])
        s["shared"] = _randn(gen, T, H).to(DTYPES[c["y"]]) if c["shared"] else None
        rows = torch.randperm(T * k, generator=gen, device="cuda", dtype=torch.int32).view(T, k)
        gone = torch.rand(T, k, generator=gen, device="cuda") < c["dropped"]
        s["rows"] = torch.where(gone, torch.full_like(rows, -1), rows)
        gates = torch.rand(T, k, generator=gen, device="cuda") + 0.05
        s["gates"] = gates / gates.sum(1, keepdim=True)
        s["weight"] = 1 + 0.1 * _randn(gen, H)
        s["residual"] = _randn(gen, T, H).to(DTYPES[c["stream"]])
        shape = {"none": None, "channel": (1, H), "token": (T, 1), "both": (T, H)}[c["gate"]]
        s["gate"] = None if shape is None else _randn(gen, *shape).to(torch.bfloat16)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its data: the shape, output buffers and the workspace."""
    from expert_serving_amd import abi

    c = s["case"]
    code = {"f32": abi.MOE_F32, "bf16": abi.MOE_BF16, "f16": abi.MOE_F16}
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s["abi"] = abi
    if c["op"] == "route":
        T, E = c["tokens"], c["experts"]
        s["shape"] = abi.make_shape(
            num_tokens=T, hidden=64, num_experts=E, intermediate=64, top_k=c["k"],
            score=abi.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else abi.MOE_SCORE_SOFTMAX,
            renormalize=int(c["renorm"]), routed_scale=c["scale"], num_groups=c["groups"], topk_groups=c["keep"],
            group_topn=c["topn"])
        s["ws"] = empty(abi.moe_workspace_size(s["shape"]), dtype=torch.uint8)
        s["ids"], s["out_gates"] = empty(T, c["k"], dtype=torch.int32), empty(T, c["k"], dtype=torch.float32)
    elif c["op"] == "norm":
        s["out"] = empty(c["rows"], c["hidden"], dtype=torch.bfloat16)
        s["stream"] = code[c["stream"]]
    elif c["op"] == "product":
        s["codes"], s["scales"] = empty(c["rows"], c["k"], dtype=torch.int8), empty(c["rows"], dtype=torch.float32)
        s["out"], s["code"] = empty(c["rows"], c["n"], dtype=DTYPES[c["out"]]), code[c["out"]]
        s["ws"] = empty(abi.moe_workspace_size_gemm_int8(c["rows"], c["n"], c["k"], c["experts"]), dtype=torch.uint8)
    elif c["op"] == "ffn":
        s["shape"] = abi.make_shape(num_tokens=c["tokens"], hidden=c["hidden"], num_experts=c["experts"],
                                    intermediate=c["inter"], top_k=c["k"])
        s["out"] = empty(c["tokens"] * c["k"], c["hidden"], dtype=DTYPES[c["out"]])
        s["code"] = code[c["out"]]
        s["weights"] = abi.int8_ffn((s["gate"], s["gate_scales"]), (s["up"], s["up_scales"]),
                                    (s["down"], s["down_scales"]))
        s["ws"] = empty(abi.moe_workspace_size_int8(s["shape"]), dtype=torch.uint8)
    else:
        s["shape"] = abi.make_shape(num_tokens=c["tokens"], hidden=c["hidden"], num_experts=max(8, c["k"]),
                                    intermediate=64, top_k=c["k"])
        g = s["gate"]
        s["block"] = abi.make_block(
            post_norm=s["weight"], eps=EPS, gate=g, residual_scale=c["scale"], stream_dtype=code[c["stream"]])
        s["code"] = code[c["y"]]
        s["out"] = empty(c["tokens"], c["hidden"], dtype=DTYPES[c["stream"]])


# ---- one pass --------------------------------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return {"route": _route, "norm": _norm, "product": _product, "ffn": _ffn, "after": _after}[s["case"]["op"]](s)


def _run_own(s):
    c, abi = s["case"], s["abi"]
    if c["op"] == "route":
        abi.moe_route_biased(s["shape"], None, None, None, s["bias"], s["logits"], None, s["k"], s["ids"],
                             s["out_gates"], s["ws"])
        return {"ids": s["ids"], "gates": s["out_gates"]}
    if c["op"] == "norm":
        abi.moe_norm(c["rows"], c["hidden"], s["stream"], s["x"], s["weight"], EPS, abi.MOE_BF16, s["out"], None, None)
        return {"out": s["out"]}
    if c["op"] == "product":
        if c["norm"]:
            abi.moe_norm(c["rows"], c["k"], abi.MOE_BF16, s["x"], s["weight"], EPS, abi.MOE_BF16, None, s["codes"],
                         s["scales"])
        else:
            abi.moe_quantize_int8(c["rows"], c["k"], abi.MOE_BF16, s["x"], s["codes"], s["scales"])
        abi.moe_grouped_gemm_int8(c["rows"], c["n"], c["k"], c["experts"], s["codes"], s["scales"], s["offsets"],
                                  s["w"], s["w_scales"], s["code"], s["out"], s["ws"])
        return {"scales": s["scales"], "out": s["out"]}
    if c["op"] == "ffn":
        abi.moe_grouped_ffn_int8(s["shape"], s["x"], s["x_scales"], s["offsets"], s["weights"], s["code"], s["out"],
                                 s["ws"])
        return {"out": s["out"]}
    abi.moe_combine_norm(s["shape"], s["block"], s["code"], s["y"], s["rows"], s["gates"], s["shared"],
                         s["residual"], s["out"])
    return {"out": s["out"]}


def _route(s):
    c, T, E, G, k = s["case"], s["case"]["tokens"], s["case"]["experts"], s["case"]["groups"], s["case"]["k"]
    logits, bias = s["logits"].double(), s["bias"].double()
    out = (bias == -math.inf).expand(T, E)
    low = torch.tensor(-math.inf, dtype=torch.float64, device=logits.device)
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        e = torch.where(out, 0.0, torch.exp(logits - torch.where(out, low, logits).amax(1, keepdim=True)))
        score = e / e.sum(1, keepdim=True)
    key = torch.where(out, low, score + bias)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :c["topn"]]
        group = torch.where(best == low, 0.0, best).sum(2)
        group = torch.where((best == low).all(2), low, group)
        order = group.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, order, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, low)
    best, ids = key.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    used = best > low
    if s["k"] is not None:
        used = used & (torch.arange(k, device=logits.device) < s["k"].unsqueeze(1))
    gates = torch.where(used, score.gather(1, ids), 0.0)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    return {"ids": torch.where(used, ids, -1).int(), "gates": (gates * c["scale"]).float()}


def _rms(x, weight):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


def _norm(s):
    return {"out": _rms(s["x"].float(), s["weight"]).to(torch.bfloat16)}


def _quantise(x):
    top = x.abs().amax(1, keepdim=True)
    return torch.where(top > 0, torch.round(127 * x / top), 0.0), top / 127  # half of the top is a tie: 63.5


def _grouped(a, weights, offsets, most):
    """a [rows, K] times the transposed weights [E, N, K] of each row's expert; all in 32 bits."""
    rows, experts = a.shape[0], weights.shape[0]
    at = torch.arange(rows, device=a.device, dtype=torch.int32)
    e = torch.searchsorted(offsets, at, right=True) - 1
    if rows <= experts:  # few rows: the weights of each row
        return torch.matmul(weights[e].float(), a.unsqueeze(2)).squeeze(2), e
    place = at - offsets[e]
    padded = torch.zeros(experts, most, a.shape[1], dtype=a.dtype, device=a.device)
    padded[e, place] = a
    return torch.matmul(padded, weights.float().transpose(1, 2))[e, place], e


def _product(s):
    x = s["x"].float()
    codes, scale = _quantise(_rms(x, s["weight"]) if s["case"]["norm"] else x)
    y, e = _grouped(codes, s["w"], s["offsets"], s["most"])
    return {"scales": scale.squeeze(1), "out": (y * scale * s["w_scales"][e]).to(DTYPES[s["case"]["out"]])}


def _ffn(s):
    x, scale = s["x"].float(), s["x_scales"].unsqueeze(1)
    g, e = _grouped(x, s["gate"], s["offsets"], s["most"])
    u, _ = _grouped(x, s["up"], s["offsets"], s["most"])
    g, u = g * scale * s["gate_scales"][e], u * scale * s["up_scales"][e]
    h = (g / (1 + torch.exp(-g)) * u).clamp(-65504, 65504).half().float()
    codes, scale = _quantise(h)
    y, _ = _grouped(codes, s["down"], s["offsets"], s["most"])
    return {"out": (y * scale * s["down_scales"][e]).to(DTYPES[s["case"]["out"]])}


def _after(s):
    c = s["case"]
    rows = s["rows"].long()
    picked = torch.where((rows >= 0).unsqueeze(2), s["y"][rows.clamp(min=0)].float(), 0.0)
    y = (picked * s["gates"].unsqueeze(2)).sum(1)
    if s["shared"] is not None:
        y = y + s["shared"].float()
    y = _rms(y, s["weight"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    return {"out": (c["scale"] * s["residual"].float() + y).to(DTYPES[c["stream"]])}


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "route":
        T, E = c["tokens"], c["experts"]
        return {"bytes": 4 * T * E + 4 * E + 8 * T * c["k"] + (4 * T if c["k_varies"] else 0), "flops": 10 * T * E}
    if c["op"] == "norm":
        n = c["rows"] * c["hidden"]
        return {"bytes": n * (size[c["stream"]] + 2) + 4 * c["hidden"], "flops": 4 * n}
    if c["op"] == "product":
        used = min(c["experts"], c["rows"])
        return {"bytes": 2 * c["rows"] * c["k"] + used * c["n"] * (c["k"] + 4) + c["rows"] * c["n"] * size[c["out"]],
                "flops": 2 * c["rows"] * c["n"] * c["k"]}
    if c["op"] == "ffn":
        H, I, rows = c["hidden"], c["inter"], c["tokens"] * c["k"]
        used = min(c["experts"], rows)
        return {"bytes": used * (3 * H * I + 8 * I + 4 * H) + rows * (H + 4 + H * size[c["out"]]),
                "flops": 6 * rows * H * I}
    T, H, k = c["tokens"], c["hidden"], c["k"]
    kept = T * k * (1 - c["dropped"])
    gate = {"none": 0, "channel": 2 * H, "token": 2 * T, "both": 2 * T * H}[c["gate"]]
    return {"bytes": kept * H * size[c["y"]] + (T * H * size[c["y"]] if c["shared"] else 0) + 8 * T * k + gate +
            2 * T * H * size[c["stream"]] + 4 * H, "flops": 2 * kept * H + 8 * T * H}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "product": _exact_product, "ffn": _exact_ffn,
            "after": _exact_after}[case["op"]](s)


def _exact_route(s):
    """Gates from the definition, expert by expert of the chosen ones; the choice by counting what ranks before."""
    c, T, E, G, k = s["case"], s["case"]["tokens"], s["case"]["experts"], s["case"]["groups"], s["case"]["k"]
    ids_all, gates_all = [], []
    index = torch.arange(E, device="cuda")
    for t0 in range(0, T, 512):
        l, b = s["logits"][t0:t0 + 512].double(), s["bias"].double()
        here = (b > -math.inf).unsqueeze(0).expand_as(l)
        if c["score"] == "sigmoid":
            score = torch.sigmoid(l)
        else:
            score = torch.softmax(l.masked_fill(~here, -math.inf), 1)
        key = (score + b).masked_fill(~here, -math.inf)
        if G > 1:
            part = key.view(len(l), G, E // G)
            total = torch.zeros(len(l), G, dtype=torch.float64, device="cuda")
            for j in range(c["topn"]):
                v, at = part.max(2)
                total += v.masked_fill(v == -math.inf, 0.0)
                part = part.scatter(2, at.unsqueeze(2), -math.inf)
            total.masked_fill_(~here.view(len(l), G, E // G).any(2), -math.inf)
            g = torch.arange(G, device="cuda")
            before = (total.unsqueeze(1) > total.unsqueeze(2)) | (
                (total.unsqueeze(1) == total.unsqueeze(2)) & (g.view(1, 1, G) < g.view(1, G, 1)))
            kept = before.sum(2) < c["keep"]
            key = key.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
        ids = torch.full((len(l), k), -1, dtype=torch.int64, device="cuda")
        gates = torch.zeros(len(l), k, dtype=torch.float64, device="cuda")
        for j in range(k):
            v = key.amax(1, keepdim=True)
            at = torch.where(key == v, index, E).amin(1)
            ok = v.squeeze(1) > -math.inf
            if s["k"] is not None:
                ok &= s["k"][t0:t0 + 512] > j
            ids[:, j] = torch.where(ok, at, -1)
            gates[:, j] = torch.where(ok, score.gather(1, at.unsqueeze(1)).squeeze(1), 0.0)
            key = key.scatter(1, at.unsqueeze(1), -math.inf)
        if c["renorm"]:
            gates = gates / gates.sum(1, keepdim=True)
        ids_all.append(ids.int())
        gates_all.append(gates * c["scale"])
    return {"ids": torch.cat(ids_all), "gates": torch.cat(gates_all)}


def _exact_rms(x, weight):
    x = x.double()
    return x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()


def _exact_norm(s):
    return {"out": _exact_rms(s["x"], s["weight"])}


def _exact_codes(x):
    top = x.abs().max(1, keepdim=True).values
    return (x * 127 / top).round().nan_to_num(0.0), top / 127


def _exact_groups(s, f):
    """f(expert, its rows) for every expert that has rows, joined."""
    at = s["offsets"].tolist()
    return torch.cat([f(e, slice(a, b)) for e, (a, b) in enumerate(zip(at, at[1:])) if b > a])


def _exact_product(s):
    x = s["x"].double()
    codes, scale = _exact_codes(_exact_rms(x, s["weight"]) if s["case"]["norm"] else x)
    y = _exact_groups(s, lambda e, r: scale[r] * (codes[r] @ s["w"][e].double().t()) * s["w_scales"][e].double())
    return {"scales": scale.squeeze(1), "out": y}


def _exact_ffn(s):
    def one(e, r):
        x, scale = s["x"][r].double(), s["x_scales"][r].double().unsqueeze(1)
        g = scale * (x @ s["gate"][e].double().t()) * s["gate_scales"][e].double()
        u = scale * (x @ s["up"][e].double().t()) * s["up_scales"][e].double()
        h = (g * torch.sigmoid(g) * u).clamp(-65504, 65504).to(torch.float16).double()
        codes, scale = _exact_codes(h)
        return scale * (codes @ s["down"][e].double().t()) * s["down_scales"][e].double()

    return {"out": _exact_groups(s, one)}


def _exact_after(s):
    c, outs = s["case"], []
    for t0 in range(0, c["tokens"], 1024):
        part = slice(t0, t0 + 1024)
        y = torch.zeros(len(s["rows"][part]), c["hidden"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            r = s["rows"][part, j].long()
            g = torch.where(r >= 0, s["gates"][part, j].double(), 0.0)
            y += g.unsqueeze(1) * s["y"][r.clamp(min=0)].double()
        if s["shared"] is not None:
            y += s["shared"][part].double()
        y = _exact_rms(y, s["weight"])
        g = s["gate"]
        if g is not None:
            y = y * (g if g.shape[0] == 1 else g[part]).double()
        outs.append(c["scale"] * s["residual"][part].double() + y)
    return {"out": torch.cat(outs)}
