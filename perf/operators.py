"""The low-bit products of the library as a user's program calls them, each
beside a plain form in elementary torch operations (32-bit arithmetic, one
rounding at the end) and its definition in 64 bits.

  w4_product   C = A . W with W in 4 bits: W[k][n] = (q[k][n] - z[g][n]) * s[g][n],
               g = k / group. One row of A is a decoded token, many a prompt.
  w4_quantize  W (K x N, 2-byte) to 4-bit codes, scales and zero points, and back
               to 2-byte values: what loading a model does to its weights.
  q8_roundtrip X (M x K, 2-byte) to 8-bit codes with a scale for each column of
               128 rows, and back: what saving an activation for the backward
               pass and restoring it does.
  q8_wgrad     dW = X^T . dY with X as saved in 8 bits: the weight gradient of a
               linear layer whose input was checkpointed.

4-bit codes are packed four bits a weight, N rows of ceil(K / 128) 64-byte
blocks; a block holds 128 consecutive k of one column n: word w of the 16-byte
quarter c holds k = 32 w + 8 c + i, i = 0..7, at nibbles 0, 4, 1, 5, 2, 6, 3, 7.
8-bit codes are rows of K values padded to a multiple of 16.
"""

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 128   # k of one packed 4-bit block
ROWS = 128    # rows that share an 8-bit scale
TINY = 2.0 ** -100  # columns whose largest magnitude is below this are saved as zeros
DEV = "cuda"


def listed():
    return [
        # One decoded token through a small projection: latency counts.
        {"name": "w4_token_1024", "op": "w4_product", "M": 1, "N": 1024, "K": 1024, "group": 128,
         "zeros": True, "type": "bf16"},
        # One decoded token through a wide feed-forward matrix: the weights' bytes count.
        {"name": "w4_token_8192x32768", "op": "w4_product", "M": 1, "N": 32768, "K": 8192,
         "group": 128, "zeros": True, "type": "bf16"},
        # A few requests at once, sizes off every boundary, fine groups, no zero points.
        {"name": "w4_batch_7_odd", "op": "w4_product", "M": 7, "N": 4097, "K": 8190, "group": 32,
         "zeros": False, "type": "f16"},
        # A serving batch of decoded tokens.
        {"name": "w4_batch_48", "op": "w4_product", "M": 48, "N": 8192, "K": 8192, "group": 64,
         "zeros": True, "type": "bf16"},
        # A long prompt: as many operations as a dense product.
        {"name": "w4_prompt_4096", "op": "w4_product", "M": 4096, "N": 8192, "K": 8192,
         "group": 128, "zeros": True, "type": "bf16"},
        # A large weight matrix as a model is loaded.
        {"name": "w4_quantize_8192", "op": "w4_quantize", "N": 8192, "K": 8192, "group": 128,
         "zeros": True, "type": "bf16"},
        # A small one off every boundary, fine groups, no zero points.
        {"name": "w4_quantize_odd", "op": "w4_quantize", "N": 3001, "K": 1023, "group": 32,
         "zeros": False, "type": "f16"},
        # The activations of a training step's tokens.
        {"name": "q8_roundtrip_8192", "op": "q8_roundtrip", "M": 8192, "K": 8192, "type": "bf16"},
        # A short ragged batch of them.
        {"name": "q8_roundtrip_odd", "op": "q8_roundtrip", "M": 1001, "K": 1023, "type": "f16"},
        # The weight gradient of a large layer: the largest case.
        {"name": "q8_wgrad_8192", "op": "q8_wgrad", "M": 8192, "N": 8192, "K": 8192,
         "type": "bf16"},
        # Many tokens into a narrow layer: a long sum over few outputs.
        {"name": "q8_wgrad_narrow", "op": "q8_wgrad", "M": 32768, "N": 640, "K": 512,
         "type": "bf16"},
        # A small layer and batch, sizes off every boundary.
        {"name": "q8_wgrad_odd", "op": "q8_wgrad", "M": 1001, "N": 1023, "K": 515, "type": "f16"},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of low .. high: half of them odd, half multiples of 40
    (rows on 16-byte boundaries that are no whole tiles)."""
    v = int(low * (high / low) ** rng.random())
    return v | 1 if rng.random() < 0.5 else max(40, v // 40 * 40)


def draw(rng):
    case = {"op": rng.choice(["w4_product", "w4_product", "w4_quantize", "q8_roundtrip",
                              "q8_wgrad", "q8_wgrad"]),
            "type": rng.choice(["bf16", "f16"])}
    while True:
        if case["op"] == "w4_product":
            tokens = rng.choice([1, int(8192 ** rng.random()), int(128 ** rng.random())])
            case.update(M=tokens, N=_size(rng, 256, 32768), K=_size(rng, 256, 16384))
        elif case["op"] == "w4_quantize":
            case.update(N=_size(rng, 256, 16384), K=_size(rng, 256, 16384))
        elif case["op"] == "q8_roundtrip":
            case.update(M=_size(rng, 64, 32768), K=_size(rng, 256, 16384))
        else:
            case.update(M=_size(rng, 64, 32768), N=_size(rng, 256, 16384),
                        K=_size(rng, 256, 16384))
        if case["op"].startswith("w4"):
            case.update(group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
        if case.get("M", 1) * case.get("N", 1) * case["K"] <= 1 << 38:
            return case


def work(case):
    K, flops = case["K"], 0
    if case["op"].startswith("w4"):
        N = case["N"]
        groups = -(-K // case["group"])
        held = K * N // 2 + groups * N * (3 if case["zeros"] else 2)
        if case["op"] == "w4_quantize":
            return {"bytes": 4 * K * N + held, "flops": 0}
        return {"bytes": 2 * case["M"] * K + held + 4 * case["M"] * N,
                "flops": 2 * case["M"] * N * K}
    M = case["M"]
    held = M * K + 4 * -(-M // ROWS) * K
    if case["op"] == "q8_roundtrip":
        return {"bytes": 4 * M * K + held, "flops": 0}
    return {"bytes": held + 2 * M * case["N"] + 4 * K * case["N"], "flops": 2 * M * case["N"] * K}


# ------------------------------------------------------------ inputs

def _normal(gen, rows, cols):
    return torch.randn(rows, cols, generator=gen, device=DEV)


def _activations(gen, rows, cols, dtype):
    """Tokens x channels with the few loud channels that activations have."""
    x = _normal(gen, rows, cols)
    loud = torch.rand(cols, generator=gen, device=DEV) < 1 / 64
    return (x * torch.where(loud, 8.0, 1.0)).to(dtype)


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    dtype, op, K = TYPES[case["type"]], case["op"], case["K"]
    if op == "w4_quantize":
        return {"w": (_normal(gen, K, case["N"]) * 0.02).to(dtype)}
    if op == "q8_roundtrip":
        return {"x": _activations(gen, case["M"], K, dtype)}
    if op == "q8_wgrad":
        q, s = _q8_plain(_activations(gen, case["M"], K, dtype))
        return {"q": q, "s": s, "dy": (_normal(gen, case["M"], case["N"]) * 0.02).to(dtype)}
    w = (_normal(gen, K, case["N"]) * 0.02).to(dtype)
    q, s, z = _w4_plain(w, case["group"], case["zeros"])
    return {"q": q, "s": s, "z": z, "x": _activations(gen, case["M"], K, dtype)}


def prepare(case, seed):
    """Weights and saved activations are held in the library's layouts, as a program that loaded
    a model or ran the forward pass holds them."""
    d = _inputs(case, seed)
    if case["op"] == "w4_product":
        d["codes"] = _w4_pack(d.pop("q"))
    elif case["op"] == "q8_wgrad":
        d["codes"] = torch.nn.functional.pad(d.pop("q"), (0, -case["K"] % 16)).contiguous()
    return {"case": dict(case), "dtype": TYPES[case["type"]], **d}


# ------------------------------------------------------------ plain forms

def _grouped(w, group):
    """K x N values as groups x group x N, the last group filled up with zeros."""
    K, N = w.shape
    return torch.nn.functional.pad(w, (0, 0, 0, -K % group)).view(-1, group, N)


def _w4_plain(w, group, zeros):
    """(codes K x N, scales, zero points or None) of 2-byte weights. Zeros filled up at the end
    change nothing: each group's range includes zero."""
    K, N = w.shape
    g = _grouped(w.float(), group)
    if zeros:
        low, high = g.amin(1).clamp(max=0), g.amax(1).clamp(min=0)
        s = ((high - low) * torch.tensor(1 / 15, device=w.device)).to(w.dtype)
    else:
        low = None
        s = (g.abs().amax(1) * torch.tensor(1 / 7, device=w.device)).to(w.dtype)
    inv = torch.reciprocal(s.float())
    z = torch.full_like(inv, 8) if low is None else torch.round(-low * inv).clamp(0, 15)
    z = torch.where(s == 0, torch.full_like(z, 0 if zeros else 8), z)
    q = (torch.round(g * inv[:, None]) + z[:, None]).clamp(0, 15)
    q = torch.where(s[:, None] == 0, z[:, None], q)
    q = q.reshape(-1, N)[:K].to(torch.uint8)
    return q, s, z.to(torch.uint8) if zeros else None


def _w4_values(q, s, z, group):
    """(q - z) * s in 32 bits, K x N."""
    K = q.shape[0]
    zero = 8.0 if z is None else z.float()[:, None]
    return ((_grouped(q.float(), group) - zero) * s.float()[:, None]).view(-1, q.shape[1])[:K]


def _w4_pack(q):
    """Codes K x N as N rows of packed blocks."""
    K, N = q.shape
    t = torch.nn.functional.pad(q.t(), (0, -K % BLOCK)).reshape(N, -1, 4, 4, 8)  # n block w c i
    t = t.permute(0, 1, 3, 2, 4)[..., [0, 2, 4, 6, 1, 3, 5, 7]].reshape(N, -1, 2)
    return (t[..., 0] | t[..., 1] << 4).contiguous()


def _w4_unpack(codes, K):
    """The K x N codes of N packed rows."""
    N = codes.shape[0]
    t = torch.stack((codes & 15, codes >> 4), -1).view(N, -1, 4, 4, 8)  # n block c w nibble
    t = t[..., [0, 4, 1, 5, 2, 6, 3, 7]].permute(0, 1, 3, 2, 4).reshape(N, -1)
    return t[:, :K].t()


def _q8_plain(x):
    """(codes M x K int8, scales for each 128 rows x column) of 2-byte activations."""
    M, K = x.shape
    g = _grouped(x.float(), ROWS)
    top = g.abs().amax(1)
    s = top * torch.tensor(1 / 127, device=x.device)
    s = torch.where(top < TINY, torch.zeros_like(s), s)
    inv = torch.where(s == 0, torch.zeros_like(s), torch.reciprocal(s))
    q = torch.round(g * inv[:, None]).clamp(-127, 127)
    return q.reshape(-1, K)[:M].to(torch.int8), s


def _q8_values(q, s):
    """q * s in 32 bits, M x K."""
    M, K = q.shape
    return (_grouped(q.float(), ROWS) * s[:, None]).view(-1, K)[:M]


def _run_plain(state):
    case, dtype = state["case"], state["dtype"]
    if case["op"] == "w4_product":
        q = _w4_unpack(state["codes"], case["K"])
        return {"y": state["x"].float() @ _w4_values(q, state["s"], state["z"], case["group"])}
    if case["op"] == "w4_quantize":
        q, s, z = _w4_plain(state["w"], case["group"], case["zeros"])
        got = {"w": _w4_values(q, s, z, case["group"]).to(dtype), "scales": s}
        return {**got, "zeros": z} if case["zeros"] else got
    if case["op"] == "q8_roundtrip":
        q, s = _q8_plain(state["x"])
        return {"x": _q8_values(q, s).to(dtype), "scales": s}
    x = _q8_values(state["codes"][:, :case["K"]], state["s"])
    return {"dw": x.t() @ state["dy"].float()}


# ------------------------------------------------------------ the library's calls

def _run_own(state):
    import register_tiled_matrix_gb300 as rtm

    case, bf16 = state["case"], state["dtype"] == torch.bfloat16
    if case["op"] == "w4_product":
        product = rtm.gemm_bf16w4f32 if bf16 else rtm.gemm_f16w4f32
        return {"y": product(state["x"], state["codes"], state["s"], state["z"], case["group"])}
    if case["op"] == "w4_quantize":
        codes, s, z = rtm.gemm_w4_quantize(state["w"], case["group"], zeros=case["zeros"])
        got = {"w": rtm.gemm_w4_dequantize(codes, s, z, case["K"], case["group"]), "scales": s}
        return {**got, "zeros": z} if case["zeros"] else got
    if case["op"] == "q8_roundtrip":
        codes, s = rtm.gemm_q8_quantize(state["x"])
        return {"x": rtm.gemm_q8_dequantize(codes, s, case["M"], case["K"], state["dtype"]),
                "scales": s}
    gradient = rtm.gemm_q8tbf16f32 if bf16 else rtm.gemm_q8tf16f32
    return {"dw": gradient(state["codes"], state["s"], state["dy"])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    d = _inputs(case, seed)
    K, op, dtype = case["K"], case["op"], TYPES[case["type"]]
    if op.startswith("w4"):
        g = torch.arange(K, device=DEV) // case["group"]
        if op == "w4_product":
            z = 8 if d["z"] is None else d["z"].double()[g]
            return {"y": d["x"].double() @ ((d["q"].double() - z) * d["s"].double()[g])}
        w = d["w"].double()
        groups, N = int(g[-1]) + 1, case["N"]
        index = g[:, None].expand(K, N)
        nil = torch.zeros(groups, N, dtype=torch.float64, device=DEV)
        high = nil.scatter_reduce(0, index, w, "amax")
        low = nil.scatter_reduce(0, index, w, "amin")
        top = high - low if case["zeros"] else torch.maximum(high, -low)
        s = (top / (15 if case["zeros"] else 7)).to(dtype).double()
        z = torch.round(-low / s) if case["zeros"] else nil + 8
        q = (torch.round(w / s[g]) + z[g]).clamp(0, 15)
        got = {"w": torch.nan_to_num((q - z[g]) * s[g]), "scales": s}
        return {**got, "zeros": None} if case["zeros"] else got
    block = torch.arange(case["M"], device=DEV) // ROWS
    if op == "q8_wgrad":
        return {"dw": (d["q"].double() * d["s"].double()[block]).t() @ d["dy"].double()}
    x = d["x"].double()
    top = torch.zeros(int(block[-1]) + 1, K, dtype=torch.float64, device=DEV)
    s = top.scatter_reduce(0, block[:, None].expand(case["M"], K), x.abs(), "amax") / 127
    return {"x": torch.nan_to_num(torch.round(x / s[block]) * s[block]), "scales": s}
