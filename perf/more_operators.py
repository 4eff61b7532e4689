"""Operators of experts in 8-bit floating point and of training through the layer: cases, inputs and plain forms.

The format: E4M3 codes with an fp32 scale for each block of 128 -- 128 columns of a token row (128 consecutive
elements of the axis that a product sums over), 128 x 128 elements of a weight matrix.

Five operators:

* "sort":     token rows to expert order, times a weight per slot or quantised to codes on the way;
* "unsort":   the gradient of "sort": rows summed back to their tokens, and the weights' gradients;
* "weighted": the gradient of the gate-weighted sum back: the expert rows' and the gates';
* "product":  rows quantised and multiplied by their expert's weights;
* "ffn":      the grouped SwiGLU FFN on codes.

run() takes the plain torch form, or with `own` the library's entry points.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FP8 = torch.float8_e4m3fn
TOP = 448.0  # the largest E4M3 value
B = 128


# ---- cases -----------------------------------------------------------------------------------------------------


def listed():
    return [
        # one decoded token to the eight experts it takes: pure latency
        dict(name="sort 1 x 7168 to codes, top 8", op="sort", tokens=1, hidden=7168, k=8, type="bf16", weights=False,
             codes=True, dropped=0.0),
        # a prefill chunk of a 256-expert layer, a few slots over capacity
        dict(name="sort 8192 x 7168 to codes, top 8", op="sort", tokens=8192, hidden=7168, k=8, type="bf16",
             weights=False, codes=True, dropped=0.02),
        # an odd training batch whose experts take their rows already weighted
        dict(name="sort 4099 x 4096 weighted, top 2", op="sort", tokens=4099, hidden=4096, k=2, type="bf16",
             weights=True, codes=False, dropped=0.0),
        # a small odd batch's gradient of the same, with that of the weights
        dict(name="unsort 33 x 4096 weighted, top 2", op="unsort", tokens=33, hidden=4096, k=2, type="bf16",
             weights=True, dropped=0.0),
        # a training step's gradient of the dispatched rows
        dict(name="unsort 8192 x 7168, top 8", op="unsort", tokens=8192, hidden=7168, k=8, type="bf16", weights=False,
             dropped=0.02),
        # a short sequence's gradient of the combine, everything held in fp32
        dict(name="weighted 64 x 2048 fp32, top 8", op="weighted", tokens=64, hidden=2048, k=8, y="f32", out="f32",
             dropped=0.1),
        # a training step's, expert rows in bf16 and the residual stream's gradient in fp32
        dict(name="weighted 8192 x 7168, top 8", op="weighted", tokens=8192, hidden=7168, k=8, y="bf16", out="f32",
             dropped=0.02),
        # a dense projection of an odd decode batch
        dict(name="product 17 x 14336 x 4096", op="product", rows=17, n=14336, k=4096, experts=1, out="bf16"),
        # the down projection of a prefill chunk over eight experts
        dict(name="product 8192 x 4096 x 14336, 8 experts", op="product", rows=8192, n=4096, k=14336, experts=8,
             out="bf16"),
        # one decoded token through eight of 128 small experts
        dict(name="ffn 1 token, 128 experts", op="ffn", tokens=1, hidden=2048, inter=768, experts=128, k=8, out="bf16"),
        # a decode step over eight large experts: their weights are read once
        dict(name="ffn 64 tokens, 8 experts", op="ffn", tokens=64, hidden=4096, inter=14336, experts=8, k=2,
             out="bf16"),
        # a prefill chunk over 256 experts
        dict(name="ffn 8192 tokens, 256 experts", op="ffn", tokens=8192, hidden=7168, inter=2048, experts=256, k=8,
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sort", "unsort", "weighted", "product", "ffn"])
    if op in ("sort", "unsort"):
        codes = op == "sort" and rng.random() < 0.5
        c = dict(op=op, tokens=_log(rng, 1, 8192), hidden=(128 if codes else 64) * _log(rng, 2, 56 if codes else 112),
                 k=rng.randint(1, 8), type=rng.choice(["bf16", "bf16", "f16", "f32"]),
                 weights=not codes and rng.random() < 0.6, dropped=rng.choice([0.0, 0.02, 0.3]))
        if op == "sort":
            c["codes"] = codes
        return c
    if op == "weighted":
        y = rng.choice(["bf16", "f16", "f32"])
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=64 * _log(rng, 4, 112 if y != "f32" else 56),
                    k=rng.randint(1, 8), y=y, out=rng.choice(["bf16", "f32", "f16"]),
                    dropped=rng.choice([0.0, 0.02, 0.3]))
    if op == "product":
        while True:
            c = dict(op=op, rows=_log(rng, 1, 8192), n=16 * _log(rng, 16, 896), k=B * _log(rng, 2, 112),
                     experts=_log(rng, 1, 64), out=rng.choice(["bf16", "f16"]))
            if c["experts"] * c["n"] * c["k"] <= 1 << 30 and c["rows"] * c["n"] * c["k"] <= 8192 * 4096 * 14336:
                return c
    while True:
        c = dict(op=op, tokens=_log(rng, 1, 8192), hidden=B * _log(rng, 4, 56), inter=B * _log(rng, 2, 112),
                 experts=_log(rng, 4, 256), k=rng.randint(1, 8), out="bf16")
        c["k"] = min(c["k"], c["experts"] // 2)
        weights, rows = c["experts"] * c["hidden"] * c["inter"], c["tokens"] * c["k"]
        if weights <= 1 << 30 and rows * c["hidden"] * c["inter"] <= 32768 * 7168 * 2048:
            return c


# ---- inputs ----------------------------------------------------------------------------------------------------


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _weights(gen, experts, n, k):
    """Codes [E, N, K] as the quantisation of normal weights by 128 x 128 blocks leaves them (the largest of a block
    is four to five deviations), and scales [E, N / 128 up, K / 128]."""
    w = torch.empty(experts, n, k, dtype=FP8, device="cuda")
    step = max(1, (1 << 28) // (n * k))
    for e in range(0, experts, step):
        part = w[e:e + step]
        part.copy_(_randn(gen, *part.shape).mul_(100.0).clamp_(-TOP, TOP))
    scales = (1 + 0.2 * _rand(gen, experts, -(-n // B), k // B)) / (100.0 * math.sqrt(k))
    return w, scales


def _row_groups(gen, tokens, k, experts):
    """Rows per expert of a routed batch with a mild skew: offsets [E + 1], and the largest group."""
    pull = 0.4 * _randn(gen, experts) - torch.log(-torch.log(_rand(gen, tokens, experts).clamp_(1e-7, 1 - 1e-7)))
    counts = torch.bincount(pull.topk(k, dim=1).indices.reshape(-1), minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return offsets, int(counts.max())


def _slots(gen, tokens, k, dropped):
    """The row of each slot [T, k]: the kept slots take rows 0, 1, ... in a random order, dropped ones have -1."""
    order = torch.rand(tokens * k, generator=gen, device="cuda")
    order = torch.where(_rand(gen, tokens * k) < dropped, 2.0, order)
    rows = torch.empty(tokens * k, dtype=torch.int32, device="cuda")
    rows[order.argsort()] = torch.arange(tokens * k, dtype=torch.int32, device="cuda")
    return torch.where(order < 2.0, rows, -1).view(tokens, k)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c, s = case, {"case": case}
    if c["op"] in ("sort", "unsort", "weighted"):
        T, H, k = c["tokens"], c["hidden"], c["k"]
        s["rows"] = _slots(gen, T, k, c["dropped"])
        gates = _rand(gen, T, k) + 0.05
        s["gates"] = gates / gates.sum(1, keepdim=True)
        if c["op"] == "weighted":
            s["y"] = _randn(gen, T * k, H).to(DTYPES[c["y"]])
            s["out"] = (_randn(gen, T, H) * torch.exp(0.5 * _randn(gen, T, 1))).to(DTYPES[c["out"]])
        else:
            s["x"] = (_randn(gen, T, H) * torch.exp(0.5 * _randn(gen, T, 1))).to(DTYPES[c["type"]])
            if c["op"] == "unsort":
                s["grad"] = _randn(gen, T * k, H).to(DTYPES[c["type"]])
    elif c["op"] == "product":
        s["x"] = _randn(gen, c["rows"], c["k"]).to(torch.bfloat16)
        s["w"], s["w_scales"] = _weights(gen, c["experts"], c["n"], c["k"])
        s["offsets"], s["most"] = _row_groups(gen, c["rows"], 1, c["experts"])
    else:
        H, I, E, rows = c["hidden"], c["inter"], c["experts"], c["tokens"] * c["k"]
        s["x"] = (_randn(gen, rows, H) * 150).clamp_(-TOP, TOP).to(FP8)
        s["x_scales"] = (1 + 0.2 * _rand(gen, rows, H // B)) / 150
        s["gate"], s["gate_scales"] = _weights(gen, E, I, H)
        s["up"], s["up_scales"] = _weights(gen, E, I, H)
        s["down"], s["down_scales"] = _weights(gen, E, H, I)
        s["offsets"], s["most"] = _row_groups(gen, c["tokens"], c["k"], E)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps beside its data: the shape, output buffers and the workspace."""
    from expert_serving_amd import abi

    c = s["case"]
    code = {"f32": abi.MOE_F32, "bf16": abi.MOE_BF16, "f16": abi.MOE_F16}
    zeros = lambda *shape, dtype: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s["abi"] = abi
    if c["op"] in ("sort", "unsort", "weighted"):
        T, H, k = c["tokens"], c["hidden"], c["k"]
        s["shape"] = abi.make_shape(num_tokens=T, hidden=H, num_experts=max(8, k), intermediate=64, top_k=k)
        if c["op"] == "weighted":
            s["y_code"], s["out_code"] = code[c["y"]], code[c["out"]]
            s["dy"], s["dg"] = zeros(T * k, H, dtype=DTYPES[c["y"]]), zeros(T, k, dtype=torch.float32)
        elif c["op"] == "unsort":
            s["code"] = code[c["type"]]
            s["dx"] = zeros(T, H, dtype=DTYPES[c["type"]])
            s["dw"] = zeros(T, k, dtype=torch.float32) if c["weights"] else None
        else:
            s["code"] = code[c["type"]]
            s["perm"] = zeros(T * k, H, dtype=torch.uint8 if c["codes"] else DTYPES[c["type"]])
            s["scales"] = zeros(T * k, H // B, dtype=torch.float32) if c["codes"] else None
    elif c["op"] == "product":
        s["codes"] = zeros(c["rows"], c["k"], dtype=torch.uint8)
        s["scales"] = zeros(c["rows"], c["k"] // B, dtype=torch.float32)
        s["y"], s["code"] = zeros(c["rows"], c["n"], dtype=DTYPES[c["out"]]), code[c["out"]]
        s["ws"] = zeros(abi.moe_workspace_size_gemm_fp8(c["rows"], c["n"], c["k"], c["experts"]), dtype=torch.uint8)
    else:
        s["shape"] = abi.make_shape(num_tokens=c["tokens"], hidden=c["hidden"], num_experts=c["experts"],
                                    intermediate=c["inter"], top_k=c["k"])
        s["y"] = zeros(c["tokens"] * c["k"], c["hidden"], dtype=DTYPES[c["out"]])
        s["code"] = code[c["out"]]
        s["weights"] = abi.fp8_ffn((s["gate"], s["gate_scales"]), (s["up"], s["up_scales"]),
                                   (s["down"], s["down_scales"]))
        s["ws"] = zeros(abi.moe_workspace_size_fp8(s["shape"]), dtype=torch.uint8)


# ---- one pass --------------------------------------------------------------------------------------------------


def run(s):
    if own:
        return _run_own(s)
    return {"sort": _sort, "unsort": _unsort, "weighted": _weighted, "product": _product,
            "ffn": _ffn}[s["case"]["op"]](s)


def _run_own(s):
    c, abi = s["case"], s["abi"]
    if c["op"] == "sort":
        n = c["tokens"] * c["k"]
        if c["codes"]:
            abi.moe_dispatch_rows_fp8(s["shape"], s["code"], s["x"], s["rows"], n, s["perm"], s["scales"])
            return {"codes": s["perm"].view(FP8), "scales": s["scales"]}
        abi.moe_dispatch_rows(s["shape"], s["code"], s["x"], s["rows"], s["gates"] if c["weights"] else None, n,
                              s["perm"])
        return {"rows": s["perm"]}
    if c["op"] == "unsort":
        weighted = c["weights"]
        abi.moe_dispatch_rows_backward(s["shape"], s["code"], s["grad"], s["rows"], c["tokens"] * c["k"],
                                       s["gates"] if weighted else None, s["x"] if weighted else None, s["dx"],
                                       s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]} if weighted else {"dx": s["dx"]}
    if c["op"] == "weighted":
        abi.moe_combine_backward(s["shape"], s["out_code"], s["out"], s["y_code"], s["y"], s["rows"], s["gates"],
                                 c["tokens"] * c["k"], s["dy"], s["dg"])
        return {"dy": s["dy"], "dg": s["dg"]}
    if c["op"] == "product":
        abi.moe_quantize_fp8(c["rows"], c["k"], abi.MOE_BF16, s["x"], s["codes"], s["scales"])
        abi.moe_grouped_gemm_fp8(c["rows"], c["n"], c["k"], c["experts"], s["codes"], s["scales"], s["offsets"],
                                 s["w"], s["w_scales"], s["code"], s["y"], s["ws"])
        return {"scales": s["scales"], "out": s["y"]}
    abi.moe_grouped_ffn_fp8(s["shape"], s["x"], s["x_scales"], s["offsets"], s["weights"], s["code"], s["y"], s["ws"])
    return {"out": s["y"]}


def _quantise(x):
    """Codes of x [R, K] fp32 by blocks of 128 columns, and the scales [R, K / 128]."""
    v = x.view(x.shape[0], -1, B)
    top = v.abs().amax(2, keepdim=True)
    codes = torch.where(top > 0, TOP * v / top, 0.0).to(FP8)
    return codes.view(x.shape), (top / TOP).squeeze(2)


def _sort(s):
    c, rows = s["case"], s["rows"]
    T, H, k = c["tokens"], c["hidden"], c["k"]
    kept = rows >= 0
    to, x = rows[kept].long(), s["x"].float()
    token = torch.arange(T, device="cuda").unsqueeze(1).expand(T, k)[kept]
    if c["codes"]:
        codes, scales = _quantise(x)
        out = torch.zeros(T * k, H, dtype=torch.uint8, device="cuda")
        out[to] = codes.view(torch.uint8)[token]
        out_scales = torch.zeros(T * k, H // B, device="cuda")
        out_scales[to] = scales[token]
        return {"codes": out.view(FP8), "scales": out_scales}
    out = torch.zeros(T * k, H, dtype=s["x"].dtype, device="cuda")
    moved = x[token]
    if c["weights"]:
        moved = moved * s["gates"][kept].unsqueeze(1)
    out[to] = moved.to(out.dtype)
    return {"rows": out}


def _unsort(s):
    c, rows = s["case"], s["rows"].long()
    grad = torch.where((rows >= 0).unsqueeze(2), s["grad"][rows.clamp(min=0)].float(), 0.0)
    if not c["weights"]:
        return {"dx": grad.sum(1).to(s["x"].dtype)}
    return {"dx": (grad * s["gates"].unsqueeze(2)).sum(1).to(s["x"].dtype),
            "dw": (grad * s["x"].float().unsqueeze(1)).sum(2)}


def _weighted(s):
    c, rows = s["case"], s["rows"].long()
    kept = rows >= 0
    out = s["out"].float().unsqueeze(1)
    y = torch.where(kept.unsqueeze(2), s["y"][rows.clamp(min=0)].float(), 0.0)
    dg = (y * out).sum(2)
    dy = torch.zeros_like(s["y"])
    dy[rows[kept]] = (s["gates"].unsqueeze(2) * out)[kept].to(dy.dtype)
    return {"dy": dy, "dg": dg}


def _widen(w, scales, n):
    """Weights [E, N, K] in fp32 from their codes and the scales of their 128 x 128 blocks."""
    full = scales.repeat_interleave(B, dim=1)[:, :n]
    return (w.float().view(*w.shape[:2], -1, B) * full.unsqueeze(3)).view(w.shape)


def _grouped(a, w, scales, offsets, most):
    """a [rows, K] fp32 times the transposed weights of each row's expert; all in 32 bits."""
    rows, experts, n = a.shape[0], w.shape[0], w.shape[1]
    at = torch.arange(rows, device=a.device, dtype=torch.int32)
    e = torch.searchsorted(offsets, at, right=True) - 1
    if rows <= experts:  # few rows: the weights of each row
        return torch.matmul(_widen(w.view(torch.uint8)[e].view(FP8), scales[e], n), a.unsqueeze(2)).squeeze(2)
    place = at - offsets[e]
    padded = torch.zeros(experts, most, a.shape[1], dtype=a.dtype, device=a.device)
    padded[e, place] = a
    return torch.matmul(padded, _widen(w, scales, n).transpose(1, 2))[e, place]


def _decode(codes, scales):
    v = codes.float().view(codes.shape[0], -1, B) * scales.unsqueeze(2)
    return v.view(codes.shape)


def _product(s):
    codes, scales = _quantise(s["x"].float())
    y = _grouped(_decode(codes, scales), s["w"], s["w_scales"], s["offsets"], s["most"])
    return {"scales": scales, "out": y.to(DTYPES[s["case"]["out"]])}


def _ffn(s):
    x = _decode(s["x"], s["x_scales"])
    g = _grouped(x, s["gate"], s["gate_scales"], s["offsets"], s["most"])
    u = _grouped(x, s["up"], s["up_scales"], s["offsets"], s["most"])
    h = _decode(*_quantise(g / (1 + torch.exp(-g)) * u))
    return {"out": _grouped(h, s["down"], s["down_scales"], s["offsets"], s["most"]).to(DTYPES[s["case"]["out"]])}


# ---- what a pass cannot do without -----------------------------------------------------------------------------


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] in ("sort", "unsort", "weighted"):
        T, H, k = c["tokens"], c["hidden"], c["k"]
        kept = T * k * (1 - c["dropped"])
        if c["op"] == "weighted":
            return {"bytes": T * H * size[c["out"]] + 2 * kept * H * size[c["y"]] + 12 * T * k, "flops": 3 * kept * H}
        one = H * size[c["type"]]
        if c["op"] == "sort":
            return {"bytes": T * one + kept * (H + H // B * 4 if c["codes"] else one) + 4 * T * k +
                    (4 * T * k if c["weights"] else 0), "flops": (2 * T if c["codes"] else kept) * H}
        return {"bytes": kept * one + T * one * (2 if c["weights"] else 1) + (12 if c["weights"] else 4) * T * k,
                "flops": kept * H * (4 if c["weights"] else 1)}
    if c["op"] == "product":
        used = min(c["experts"], c["rows"])
        return {"bytes": 2 * c["rows"] * c["k"] + used * c["n"] * c["k"] + 4 * used * -(-c["n"] // B) * (c["k"] // B) +
                c["rows"] * c["n"] * size[c["out"]], "flops": 2 * c["rows"] * c["n"] * c["k"]}
    H, I, rows = c["hidden"], c["inter"], c["tokens"] * c["k"]
    used = min(c["experts"], rows)
    return {"bytes": used * 3 * H * I * (1 + 4 / (B * B)) + rows * (H + 4 * (H // B) + H * size[c["out"]]),
            "flops": 6 * rows * H * I}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"sort": _exact_sort, "unsort": _exact_unsort, "weighted": _exact_weighted, "product": _exact_product,
            "ffn": _exact_ffn}[case["op"]](s)


def _exact_codes(x):
    """The E4M3 values nearest to 448 x / amax (ties to even) of x [R, K] fp64, and the scales [R, K / 128]."""
    v = x.reshape(len(x), -1, B)
    top = v.abs().max(2, keepdim=True).values
    q = (TOP * v / top).nan_to_num(0.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)  # three bits below the first
    return ((q / step).round() * step).reshape(x.shape), (top / TOP).squeeze(2)


def _chunks(n, size):
    return [slice(a, min(a + size, n)) for a in range(0, n, size)]


def _exact_sort(s):
    c = s["case"]
    T, H, k = c["tokens"], c["hidden"], c["k"]
    wide = torch.float32 if c["codes"] else torch.float64
    out = torch.zeros(T * k, H, dtype=wide, device="cuda")
    scales = torch.zeros(T * k, H // B, dtype=torch.float64, device="cuda") if c["codes"] else None
    for part in _chunks(T, 1024):
        x = s["x"][part].double()
        if c["codes"]:
            x, sc = _exact_codes(x)
        for j in range(k):
            r = s["rows"][part, j].long()
            ok = r >= 0
            v = x * s["gates"][part, j].double().unsqueeze(1) if c["weights"] else x
            out[r[ok]] = v[ok].to(wide)  # codes are exact in fp32
            if c["codes"]:
                scales[r[ok]] = sc[ok]
    return {"codes": out, "scales": scales} if c["codes"] else {"rows": out}


def _exact_unsort(s):
    c = s["case"]
    T, H, k = c["tokens"], c["hidden"], c["k"]
    dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for part in _chunks(T, 1024):
        for j in range(k):
            r = s["rows"][part, j].long()
            g = s["grad"][r.clamp(min=0)].double() * (r >= 0).unsqueeze(1)
            dx[part] += g * s["gates"][part, j].double().unsqueeze(1) if c["weights"] else g
            dw[part, j] = torch.linalg.vecdot(g, s["x"][part].double())
    return {"dx": dx, "dw": dw} if c["weights"] else {"dx": dx}


def _exact_weighted(s):
    c = s["case"]
    T, H, k = c["tokens"], c["hidden"], c["k"]
    dy = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    dg = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for part in _chunks(T, 1024):
        o = s["out"][part].double()
        for j in range(k):
            r = s["rows"][part, j].long()
            ok = r >= 0
            dy[r[ok]] = s["gates"][part, j].double().unsqueeze(1)[ok] * o[ok]
            dg[part, j] = torch.linalg.vecdot(o, s["y"][r.clamp(min=0)].double()) * ok
    return {"dy": dy, "dg": dg}


def _exact_groups(s, f):
    """f(expert, its rows) for every expert that has rows, joined."""
    at = s["offsets"].tolist()
    return torch.cat([f(e, slice(a, b)) for e, (a, b) in enumerate(zip(at, at[1:])) if b > a])


def _exact_times(x, sx, w, sw):
    """x [R, K], sx [R, K / 128], w codes [N, K], sw [N / 128 up, K / 128]: scaled rows times scaled weights."""
    n = torch.arange(w.shape[0], device="cuda") // B
    kb = torch.arange(w.shape[1], device="cuda") // B
    return (x * sx[:, kb]) @ (w.double() * sw.double()[n][:, kb]).t()


def _exact_product(s):
    codes, scales = _exact_codes(s["x"].double())
    y = _exact_groups(s, lambda e, r: _exact_times(codes[r], scales[r], s["w"][e], s["w_scales"][e]))
    return {"scales": scales, "out": y}


def _exact_ffn(s):
    def one(e, r):
        x, sx = s["x"][r].double(), s["x_scales"][r].double()
        g = _exact_times(x, sx, s["gate"][e], s["gate_scales"][e])
        u = _exact_times(x, sx, s["up"][e], s["up_scales"][e])
        return _exact_times(*_exact_codes(g * torch.sigmoid(g) * u), s["down"][e], s["down_scales"][e])

    return {"out": _exact_groups(s, one)}
