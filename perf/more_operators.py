"""The 8-bit floating-point products of the library and the experts' layer built on them, as a
user's program calls them, each beside a plain form in elementary torch operations (32-bit
arithmetic, one rounding at the end) and its definition in 64 bits.

  quantize           X to e4m3 codes with a power-of-two scale for each block, and back to the
                     values they stand for. A block is 128 values of a row, 128 of a column, or
                     a 128 x 128 tile (weights).
  product            Y = A . W: A in 8 bits with a scale for 128 values of a row, W in 8 bits
                     with a scale for each 128 x 128 tile.
  gradients          dX = dY . W^T and dW = X^T . dY of that product: dY is taken to 8 bits
                     along both axes within the call, X was saved along its columns.
  route              top-k experts of each token from its logits, their weights, and the rows'
                     order by expert; in training the logits' gradient too.
  experts            y[t] = sum_j weights[t][j] * (x[t] . W[expert j of t]): rows gathered into
                     the experts' order and taken to 8 bits, the experts' products, the sum.
  experts_gradients  its gradients for x, W and the weights.

Codes are torch.float8_e4m3fn, rows 16-byte aligned (a view of rows padded to 16).
"""

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
BLOCK = 128
TINY = 2.0 ** -100  # blocks whose largest magnitude is below this become zeros
NIL = 1e-20         # added to the sum of the chosen scores
DEV = "cuda"


def listed():
    return [
        # The activations of a training step's tokens, along both axes.
        {"name": "quantize_both_8192", "op": "quantize", "M": 8192, "K": 8192, "kind": "both",
         "type": "bf16"},
        # A weight matrix off every boundary.
        {"name": "quantize_tiles_odd", "op": "quantize", "M": 3001, "K": 1023, "kind": "tiles",
         "type": "f16"},
        # One decoded token through a small projection: latency counts.
        {"name": "product_token_1024", "op": "product", "M": 1, "N": 1024, "K": 1024},
        # A serving batch through a wide matrix, sizes off every boundary: the weights' bytes count.
        {"name": "product_batch_33_odd", "op": "product", "M": 33, "N": 16383, "K": 8190},
        # A long prompt.
        {"name": "product_prompt_8192", "op": "product", "M": 8192, "N": 8192, "K": 8192},
        # The backward pass of a large layer: the largest case.
        {"name": "gradients_8192", "op": "gradients", "M": 8192, "N": 8192, "K": 8192,
         "type": "bf16"},
        # A small layer and batch, sizes off every boundary.
        {"name": "gradients_odd", "op": "gradients", "M": 1001, "N": 1023, "K": 515, "type": "f16"},
        # One decoded token among many experts, in groups, with a bias for balance.
        {"name": "route_token", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "align": 1, "train": False},
        # A training step's tokens, forward and backward.
        {"name": "route_train", "op": "route", "T": 16384, "E": 128, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "align": 128, "train": True},
        # A few decoded tokens through the experts: their weights' bytes count.
        {"name": "experts_decode", "op": "experts", "T": 4, "E": 64, "k": 8, "K": 4096, "N": 2048,
         "align": 1, "type": "bf16"},
        # A prompt through the experts.
        {"name": "experts_prompt", "op": "experts", "T": 8192, "E": 64, "k": 6, "K": 4096,
         "N": 2048, "align": 1, "type": "bf16"},
        # A training step's backward pass through them.
        {"name": "experts_gradients", "op": "experts_gradients", "T": 8192, "E": 32, "k": 4,
         "K": 2048, "N": 2048, "align": 128, "type": "bf16"},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of low .. high: half of them odd, half multiples of 40
    (rows on 16-byte boundaries that are no whole tiles)."""
    v = int(low * (high / low) ** rng.random())
    return v | 1 if rng.random() < 0.5 else max(40, v // 40 * 40)


def _draw_sizes(rng):
    op = rng.choice(["quantize", "product", "product", "gradients", "route", "experts",
                     "experts_gradients"])
    if op == "quantize":
        return {"op": op, "M": _size(rng, 64, 32768), "K": _size(rng, 256, 16384),
                "kind": rng.choice(["rows", "columns", "both", "tiles"]),
                "type": rng.choice(["bf16", "f16", "f32"])}
    if op == "product":
        tokens = rng.choice([1, int(128 ** rng.random()), int(16384 ** rng.random())])
        return {"op": op, "M": tokens, "N": _size(rng, 256, 32768), "K": _size(rng, 256, 16384)}
    if op == "gradients":
        return {"op": op, "M": _size(rng, 64, 32768), "N": _size(rng, 256, 16384),
                "K": _size(rng, 256, 16384), "type": rng.choice(["bf16", "f16"])}
    E = rng.choice([8, 16, 32, 64, 128, 256])
    k = rng.choice([1, 2, 3, 4, 6, 8])
    if op == "route":
        groups = rng.choice([1, 4, 8])
        top = groups if E // groups < 8 else rng.choice([1, 2, 4]) if groups > 1 else 1
        return {"op": op, "T": int(65536 ** rng.random()), "E": E, "k": k,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "top_groups": top, "align": rng.choice([1, 128]),
                "train": rng.random() < 0.5}
    case = {"op": op, "E": E, "k": k, "K": _size(rng, 256, 4096), "N": _size(rng, 256, 4096),
            "type": rng.choice(["bf16", "f16"])}
    if op == "experts":
        return {**case, "T": int(16384 ** rng.random()), "align": rng.choice([1, 128])}
    return {**case, "T": _size(rng, 64, 16384), "align": 128}


def draw(rng):
    while True:
        case = _draw_sizes(rng)
        held = case.get("E", 1) * case.get("K", 1) * case.get("N", 1)
        if work(case)["flops"] <= 1 << 40 and held <= 1 << 30:
            return case


def _gathered(case):
    """Rows of a buffer in the experts' order: each expert's part starts at a multiple of align."""
    slots = case["T"] * case["k"]
    return slots + min(case["E"], slots) * (case["align"] - 1)


def _touched(case):
    """Experts that some token chose, were all equally likely."""
    return case["E"] * (1 - (1 - case["k"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        held = 4 * T * E + 12 * T * k + 4 * _gathered(case) + 4 * (E + 1)
        return {"bytes": held + (4 * T * E + 4 * T * k if case["train"] else 0), "flops": 0}
    K = case["K"]
    if op == "quantize":
        M = case["M"]
        rows, cols = -(-M // BLOCK), -(-K // BLOCK)
        scales = {"rows": M * cols, "columns": rows * K, "tiles": rows * cols,
                  "both": M * cols + rows * K}[case["kind"]]
        size = TYPES[case["type"]].itemsize
        values = 4 * M * K * (2 if case["kind"] == "both" else 1)
        return {"bytes": M * K * size + values + 4 * scales, "flops": 0}
    N = case["N"]
    if op == "product":
        return {"bytes": case["M"] * K + K * N + 4 * case["M"] * N,
                "flops": 2 * case["M"] * N * K}
    if op == "gradients":
        M = case["M"]
        return {"bytes": M * K + 2 * M * N + K * N + 4 * M * K + 4 * K * N, "flops": 4 * M * N * K}
    T, k = case["T"], case["k"]
    if op == "experts":
        return {"bytes": 2 * T * K + int(_touched(case) * K * N) + 4 * T * N,
                "flops": 2 * T * k * K * N}
    return {"bytes": T * k * K + 2 * T * N + 4 * T * k * N + 5 * case["E"] * K * N + 4 * T * K,
            "flops": 4 * T * k * K * N}


# ------------------------------------------------------------ inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _activations(gen, rows, cols):
    """Tokens x channels with the few loud channels that activations have."""
    loud = torch.rand(cols, generator=gen, device=DEV) < 1 / 64
    return _normal(gen, rows, cols) * torch.where(loud, 8.0, 1.0)


def _padded(codes):
    """The same codes as a view of rows padded to 16 bytes."""
    K = codes.shape[-1]
    held = torch.zeros(*codes.shape[:-1], -(-K // 16) * 16, dtype=torch.uint8, device=DEV)
    held[..., :K] = codes.view(torch.uint8)
    return held.view(F8)[..., :K]


def _weight(gen, *shape):
    """A weight as a checkpoint holds it: codes, and scales that are no powers of two."""
    codes = _padded((_normal(gen, *shape) * 64).clamp(-448, 448).to(F8))
    tiles = [-(-n // BLOCK) for n in shape[-2:]]
    scales = torch.rand(*shape[:-2], *tiles, generator=gen, device=DEV) * 4e-4 + 2e-4
    return codes, scales


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op = case["op"]
    dtype = TYPES[case.get("type", "bf16")]
    if op == "quantize":
        x = _activations(gen, case["M"], case["K"])
        return {"x": (x * 0.02 if case["kind"] == "tiles" else x).to(dtype)}
    if op == "product":
        a, s = _quantize_plain(_activations(gen, case["M"], case["K"]).bfloat16(), 1, BLOCK)
        w, ws = _weight(gen, case["K"], case["N"])
        return {"a": _padded(a), "as": s, "w": w, "ws": ws}
    if op == "gradients":
        x, s = _quantize_plain(_activations(gen, case["M"], case["K"]).bfloat16(), BLOCK, 1)
        w, ws = _weight(gen, case["K"], case["N"])
        return {"x": _padded(x), "xs": s, "w": w, "ws": ws,
                "dy": (_normal(gen, case["M"], case["N"]) * 0.02).to(dtype)}
    T, E, k = case["T"], case["E"], case["k"]
    # Some experts are liked more than others.
    logits = _normal(gen, T, E) + 0.5 * _normal(gen, E)
    if op == "route":
        d = {"logits": logits}
        if case["bias"]:
            d["bias"] = _normal(gen, E) * 0.05
        if case["train"]:
            d["dweights"] = _normal(gen, T, k)
        return d
    plan = {"score": "softmax", "bias": False, "groups": 1, "top_groups": 1, **case}
    d = _route_plain(plan, logits, None)
    d["w"], d["ws"] = _weight(gen, E, case["K"], case["N"])
    if op == "experts":
        d["x"] = _activations(gen, T, case["K"]).to(dtype)
        return d
    gathered = _gather_plain(_activations(gen, T, case["K"]).to(dtype), d["rows"], k, None)
    x, d["xs"] = _quantize_plain(gathered, BLOCK, 1)
    d["x"] = _padded(x)
    d["dy"] = (_normal(gen, T, case["N"]) * 0.02).to(dtype)
    d["c"] = _normal(gen, _gathered(case), case["N"])  # the experts' products of the forward pass
    return d


def prepare(case, seed):
    """Weights, routing and saved activations as a program holds them that loaded a model or ran
    the forward pass; the plain form is told the most rows that an expert has."""
    d = _inputs(case, seed)
    if "offsets" in d:
        d["most"] = int((d["offsets"][1:] - d["offsets"][:-1]).max())
    return {"case": dict(case), **d}


# ------------------------------------------------------------ plain forms

def _blocks(x, bm, bk):
    """x as its blocks, filled up with zeros: blocks down x bm x blocks across x bk."""
    M, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % bk, 0, -M % bm))
    return x.view(x.shape[0] // bm, bm, x.shape[1] // bk, bk)


def _spread(s, bm, bk, M, K):
    """One scale for each value."""
    return s.repeat_interleave(bm, 0)[:M].repeat_interleave(bk, 1)[:, :K]


def _quantize_plain(x, bm, bk):
    """(codes, scales) with a scale 2^i for each bm x bk block, the least with max|x| <= 448 * 2^i."""
    M, K = x.shape
    g = _blocks(x.float(), bm, bk)
    top = g.abs().amax((1, 3))
    m, e = torch.frexp(top)
    s = torch.ldexp(torch.ones_like(top), e - 8 - (m <= 0.875).int())
    s = torch.where(top < TINY, torch.zeros_like(s), s)
    inv = torch.where(s == 0, s, 1 / s)
    q = (g * inv[:, None, :, None]).to(F8)
    return q.reshape(g.shape[0] * bm, -1)[:M, :K], s


def _values(codes, s, bm, bk):
    M, K = codes.shape
    return codes.float() * _spread(s, bm, bk, M, K)


def _weight_values(codes, s):
    K, N = codes.shape[-2:]
    s = s.repeat_interleave(BLOCK, -2)[..., :K, :].repeat_interleave(BLOCK, -1)[..., :N]
    return codes.float() * s


def _gather_plain(x, rows, fan, factors):
    """Row i: row rows[i] // fan of x, times factors[rows[i]]; zeros where rows[i] is -1."""
    got = x.float()[rows.clamp(min=0) // fan]
    if factors is not None:
        got = got * factors.flatten()[rows.clamp(min=0)][:, None]
    return torch.where(rows[:, None] < 0, torch.zeros_like(got), got)


def _scores(case, logits):
    z = logits.double()
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_plain(case, logits, bias):
    """Scores in 64 bits, since neighbours decide the order; a tie goes to the lowest index."""
    T, E, k = case["T"], case["E"], case["k"]
    s = _scores(case, logits)
    chosen = s if bias is None else s + bias.double()
    if case["groups"] > 1:
        g = chosen.view(T, case["groups"], -1)
        best = g.sort(-1, descending=True)[0][..., :2].sum(-1)
        keep = best.sort(dim=-1, descending=True, stable=True)[1][:, :case["top_groups"]]
        mask = torch.zeros_like(best).scatter_(1, keep, 1.0)
        chosen = torch.where(mask[..., None] > 0, g, torch.full_like(g, -torch.inf)).view(T, E)
    experts = chosen.sort(dim=-1, descending=True, stable=True)[1][:, :k]
    p = s.gather(1, experts)
    weights = (p / (p.sum(1, keepdim=True) + NIL)).float()
    # Slots t * k + j by expert, in order; each expert's part at a multiple of align.
    flat, align = experts.reshape(-1), case["align"]
    counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
    ends = counts.cumsum(0)
    parts = (counts + align - 1) // align * align
    offsets = torch.nn.functional.pad(parts.cumsum(0), (1, 0))
    order = flat.sort(dim=0, stable=True)[1]
    by = flat[order]
    at = torch.arange(T * k, device=DEV) - (ends - counts)[by] + offsets[by]
    rows = torch.full((_gathered(case),), -1, dtype=torch.int64, device=DEV)
    rows[at] = order
    slots = torch.empty_like(flat).scatter_(0, order, at)
    whole = {"experts": experts, "slots": slots.view(T, k), "rows": rows, "offsets": offsets}
    return {"weights": weights, **{n: v.int() for n, v in whole.items()}}


def _route_backward_plain(case, logits, experts, dweights):
    s, experts, dw = _scores(case, logits), experts.long(), dweights.double()
    p = s.gather(1, experts)
    total = p.sum(1, keepdim=True) + NIL
    dp = (dw - (dw * p).sum(1, keepdim=True) / total) / total
    if case["score"] == "sigmoid":
        return torch.zeros_like(s).scatter_(1, experts, dp * p * (1 - p)).float()
    ds = torch.zeros_like(s).scatter_(1, experts, dp)
    return (s * (ds - (ds * s).sum(1, keepdim=True))).float()


def _by_expert(state, x):
    """x's rows as experts x most x columns, zeros after an expert's last row; and where they go back."""
    o = state["offsets"].long()
    at = o[:-1, None] + torch.arange(state["most"], device=DEV)
    inside = at < o[1:, None]
    at = torch.where(inside, at, torch.zeros_like(at))
    return torch.where(inside[..., None], x[at], torch.zeros_like(x[:1])), inside, at


def _from_experts(y, inside, at, rows):
    """The rows of experts x most x columns back in the experts' order."""
    out = torch.zeros(rows + 1, y.shape[-1], device=DEV)
    out[torch.where(inside, at, torch.full_like(at, rows)).flatten()] = y.flatten(0, 1)
    return out[:rows]


def _run_plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "quantize":
        kinds = {"rows": [(1, BLOCK)], "columns": [(BLOCK, 1)], "tiles": [(BLOCK, BLOCK)],
                 "both": [(1, BLOCK), (BLOCK, 1)]}[case["kind"]]
        held = [(*_quantize_plain(state["x"], *b), b) for b in kinds]
        return [t for q, s, b in held for t in (_values(q, s, *b), s)]
    if op == "product":
        return {"y": _values(state["a"], state["as"], 1, BLOCK) @ _weight_values(state["w"], state["ws"])}
    if op == "gradients":
        rows, columns = ((1, BLOCK), (BLOCK, 1))
        dy = _values(*_quantize_plain(state["dy"], *rows), *rows)
        dx = dy @ _weight_values(state["w"], state["ws"]).t()
        dy = _values(*_quantize_plain(state["dy"], *columns), *columns)
        return {"dx": dx, "dw": _values(state["x"], state["xs"], *columns).t() @ dy}
    if op == "route":
        got = _route_plain(case, state["logits"], state.get("bias"))
        if case["train"]:
            got["dlogits"] = _route_backward_plain(case, state["logits"], got["experts"],
                                                   state["dweights"])
        return got
    k, R, slots = case["k"], _gathered(case), state["slots"].long()
    w = _weight_values(state["w"], state["ws"])
    if op == "experts":
        a = _gather_plain(state["x"], state["rows"], k, None)
        a = _values(*_quantize_plain(a, 1, BLOCK), 1, BLOCK)
        a, inside, at = _by_expert(state, a)
        c = _from_experts(a @ w, inside, at, R)
        return {"y": (c[slots] * state["weights"][..., None]).sum(1)}
    dc = _gather_plain(state["dy"], state["rows"], k, state["weights"])
    d, inside, at = _by_expert(state, _values(*_quantize_plain(dc, 1, BLOCK), 1, BLOCK))
    dx = _from_experts(d @ w.transpose(1, 2), inside, at, R)[slots].sum(1)
    d = _by_expert(state, _values(*_quantize_plain(dc, BLOCK, 1), BLOCK, 1))[0]
    x = _by_expert(state, _values(state["x"], state["xs"], BLOCK, 1))[0]
    dweights = (state["dy"].float()[:, None] * state["c"][slots]).sum(-1)
    return {"dx": dx, "dw": x.transpose(1, 2) @ d, "dweights": dweights}


# ------------------------------------------------------------ the library's calls

def _run_own(state):
    import register_tiled_matrix_gb300 as rtm

    case, op = state["case"], state["case"]["op"]
    if op == "quantize":
        if case["kind"] == "tiles":
            held = [(rtm.gemm_f8_quantize_tiles(state["x"]), "tiles")]
        elif case["kind"] == "both":
            q, s, qc, sc = rtm.gemm_f8_quantize(state["x"], "both")
            held = [((q, s), "rows"), ((qc, sc), "columns")]
        else:
            held = [(rtm.gemm_f8_quantize(state["x"], case["kind"]), case["kind"])]
        return [t for (q, s), kind in held
                for t in (rtm.gemm_f8_dequantize(q, s, kind, torch.float32), s)]
    if op == "product":
        return {"y": rtm.gemm_f8w8f32(state["a"], state["as"], state["w"], state["ws"])}
    if op == "gradients":
        q, s, qc, sc = rtm.gemm_f8_quantize(state["dy"], "both")
        return {"dx": rtm.gemm_f8w8tf32(q, s, state["w"], state["ws"]),
                "dw": rtm.gemm_f8tf8f32(state["x"], state["xs"], qc, sc)}
    if op == "route":
        plan = rtm.gemm_route(state["logits"], case["k"], state.get("bias"), score=case["score"],
                              groups=case["groups"], top_groups=case["top_groups"],
                              align=case["align"])
        experts, weights, slots, rows, offsets = plan
        got = {"weights": weights, "experts": experts, "slots": slots, "rows": rows,
               "offsets": offsets}
        if case["train"]:
            got["dlogits"] = rtm.gemm_route_backward(state["logits"], experts, state["dweights"],
                                                     score=case["score"])
        return got
    k, rows, slots, offsets = case["k"], state["rows"], state["slots"], state["offsets"]
    if op == "experts":
        a, s = rtm.gemm_f8_quantize(state["x"], "rows", gather=rows, fan=k)
        c = rtm.gemm_f8w8f32_experts(a, s, state["w"], state["ws"], offsets)
        return {"y": rtm.gemm_experts_join(c, slots, state["weights"])}
    q, s, qc, sc = rtm.gemm_f8_quantize(state["dy"], "both", gather=rows, fan=k,
                                        factors=state["weights"])
    dx = rtm.gemm_f8w8tf32_experts(q, s, state["w"], state["ws"], offsets)
    return {"dx": rtm.gemm_experts_join(dx, slots),
            "dw": rtm.gemm_f8tf8f32_experts(state["x"], state["xs"], qc, sc, offsets),
            "dweights": rtm.gemm_experts_join_backward(state["dy"], state["c"], slots)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ the definitions in 64 bits

def _e4m3(v):
    """The nearest value with three mantissa bits and exponents from -6, halves to even."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1]
    step = torch.exp2(e.double() - 4)
    return torch.round(v / step) * step


def _held(x, axis):
    """What is held of x (64 bits) with a scale for 128 values along `axis` (None: along both)."""
    M, K = x.shape
    r, c = (torch.arange(n, device=DEV) // BLOCK for n in (M, K))
    r = torch.arange(M, device=DEV) if axis == 1 else r
    c = torch.arange(K, device=DEV) if axis == 0 else c
    blocks = int(c[-1]) + 1
    at = (r[:, None] * blocks + c).flatten()
    top = torch.zeros((int(r[-1]) + 1) * blocks, dtype=torch.float64, device=DEV)
    top = top.scatter_reduce(0, at, x.abs().flatten(), "amax")
    m, i = torch.frexp(top / 448)  # m in [0.5, 1)
    s = torch.where(top > 0, torch.exp2(i.double() - (m == 0.5).double()), 0.0)
    v = torch.where(s[at] > 0, _e4m3(x.flatten() / s[at]) * s[at], 0.0)
    return v.view(M, K), s.view(-1, blocks)


def _tiled(codes, s):
    K, N = codes.shape
    k, n = (torch.arange(d, device=DEV) // BLOCK for d in (K, N))
    return codes.double() * s.double()[k][:, n]


def exact(case, seed):
    d, op = _inputs(case, seed), case["op"]
    if op == "quantize":
        axes = {"rows": [1], "columns": [0], "both": [1, 0], "tiles": [None]}[case["kind"]]
        return [t for a in axes for t in _held(d["x"].double(), a)]
    if op == "product":
        k = torch.arange(case["K"], device=DEV) // BLOCK
        return {"y": (d["a"].double() * d["as"].double()[:, k]) @ _tiled(d["w"], d["ws"])}
    if op == "gradients":
        m = torch.arange(case["M"], device=DEV) // BLOCK
        dy = d["dy"].double()
        return {"dx": _held(dy, 1)[0] @ _tiled(d["w"], d["ws"]).t(),
                "dw": (d["x"].double() * d["xs"].double()[m]).t() @ _held(dy, 0)[0]}
    if op == "route":
        z, T = d["logits"].double(), case["T"]
        whole = {n: None for n in ("experts", "slots", "rows", "offsets")}
        experts = _route_plain(case, d["logits"], d.get("bias"))["experts"].long()
        z.requires_grad_(case["train"])
        s = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
        p = s[torch.arange(T, device=DEV)[:, None], experts]
        w = p / (p.sum(1, keepdim=True) + NIL)
        got = {"weights": w.detach(), **whole}
        if case["train"]:
            w.backward(d["dweights"].double())
            got["dlogits"] = z.grad
        return got
    T, k, E = case["T"], case["k"], case["E"]
    slots, weights = d["slots"].long(), d["weights"].double()
    o = d["offsets"].tolist()
    token = d["rows"].long() // k  # -1 for a row of zeros
    if op == "experts":
        y = torch.zeros(T, case["N"], dtype=torch.float64, device=DEV)
        a = _held(d["x"].double(), 1)[0]
        for e in range(E):
            at = torch.arange(o[e], o[e + 1], device=DEV)
            at = at[token[at] >= 0]
            if len(at):
                c = a[token[at]] @ _tiled(d["w"][e], d["ws"][e])
                y.index_add_(0, token[at], c * weights.flatten()[d["rows"][at].long()][:, None])
        return {"y": y}
    block = torch.arange(_gathered(case), device=DEV) // BLOCK
    dx = torch.zeros(T, case["K"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(E, case["K"], case["N"], dtype=torch.float64, device=DEV)
    for e in range(E):
        at = torch.arange(o[e], o[e + 1], device=DEV)
        if len(at):
            used = token[at] >= 0
            f = torch.where(used, weights.flatten()[d["rows"][at].long().clamp(min=0)], 0.0)
            dc = d["dy"].double()[token[at].clamp(min=0)] * f[:, None]
            dc = dc.float().double()  # the gathered row is the product in 32 bits
            part = _held(dc, 1)[0] @ _tiled(d["w"][e], d["ws"][e]).t()
            dx.index_add_(0, token[at][used], part[used])
            x = d["x"][at].double() * d["xs"].double()[block[at]]
            dw[e] = x.t() @ _held(dc, 0)[0]
    c = d["c"].double()
    dweights = torch.stack([(d["dy"].double() * c[slots[:, j]]).sum(1) for j in range(k)], 1)
    return {"dx": dx, "dw": dw, "dweights": dweights}
