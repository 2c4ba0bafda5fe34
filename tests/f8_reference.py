"""Definitions in 64 bits of the 8-bit floating-point operands, of routing and of the experts'
layer, in torch on whatever device the inputs are on. No code of the library is used."""

import torch

F8 = torch.float8_e4m3fn
BLOCK = 128
NIL = 1e-20


def e4m3(v):
    """The nearest e4m3 value (halves to even) of 64-bit values with |v| <= 448."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1].double()
    step = torch.exp2(e - 4)
    return torch.round(v / step) * step


def spread(s, bm, bk, M, K):
    return s.repeat_interleave(bm, -2)[..., :M, :].repeat_interleave(bk, -1)[..., :K]


def blocks_of(kind):
    return {"rows": (1, BLOCK), "columns": (BLOCK, 1), "tiles": (BLOCK, BLOCK)}[kind]


def quantize(x, kind):
    """(values of the codes, scales) in 64 bits of one matrix."""
    bm, bk = blocks_of(kind)
    M, K = x.shape
    x = x.double()
    p = torch.nn.functional.pad(x, (0, -K % bk, 0, -M % bm))
    top = p.abs().view(p.shape[0] // bm, bm, p.shape[1] // bk, bk).nan_to_num(
        nan=torch.inf, posinf=torch.inf).amax((1, 3))
    m, e = torch.frexp(top / 448)
    s = torch.exp2(e.double() - (m == 0.5).double())
    s = torch.where(top < 2.0 ** -100, torch.zeros_like(s), s)
    s = torch.where(top == torch.inf, torch.full_like(s, torch.nan), s)
    t = spread(s, bm, bk, M, K)
    return torch.where(t > 0, e4m3(x / t), torch.zeros_like(x)), s


def values(codes, s, kind):
    bm, bk = blocks_of(kind)
    return codes.double() * spread(s.double(), bm, bk, *codes.shape[-2:])


def gathered(x, rows, fan, factors):
    """Row i: x[rows[i] // fan] * factors[rows[i]] in 32 bits, zeros where rows[i] names none."""
    rows = rows.long()
    fine = (rows >= 0) & (rows < x.shape[0] * fan)
    at = torch.where(fine, rows, torch.zeros_like(rows))
    got = x.float()[at // fan]
    if factors is not None:
        got = got * factors.flatten()[at][:, None]
    return torch.where(fine[:, None], got, torch.zeros_like(got))


def scores(z, score):
    z = z.double()
    if score == "sigmoid":
        return torch.sigmoid(z)
    s = torch.softmax(z, 1)
    return torch.where((z == -torch.inf).all(1, keepdim=True), torch.zeros_like(s), s)


def route(z, k, bias=None, score="softmax", groups=1, top_groups=1, renormalise=True, scale=1.0,
          align=128):
    """(experts, weights, slots, rows, offsets); a tie goes to the lowest index, NaN counts as -inf."""
    T, E = z.shape
    s = scores(z, score)
    by = s + bias.double() if bias is not None else s
    if bias is None and groups == 1:
        by = z.double()  # what the scores rise with
    by = by.nan_to_num(nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf)
    if groups > 1:
        g = by.view(T, groups, -1)
        best = g.sort(dim=-1, descending=True)[0][..., :2].sum(-1)
        keep = best.sort(dim=-1, descending=True, stable=True)[1][:, :top_groups]
        inside = torch.zeros_like(best).scatter_(1, keep, 1.0).repeat_interleave(E // groups, 1)
        order = torch.where(inside > 0, by, torch.full_like(by, -torch.inf))
        # experts outside come after those inside, whatever their scores
        first = order.sort(dim=-1, descending=True, stable=True)[1]
        at = inside.gather(1, first).sort(dim=-1, descending=True, stable=True)[1]
        experts = first.gather(1, at)[:, :k]
    else:
        experts = by.sort(dim=-1, descending=True, stable=True)[1][:, :k]
    p = s.gather(1, experts)
    w = scale * (p / (p.sum(1, keepdim=True) + NIL) if renormalise else p)
    lists = [[] for _ in range(E)]
    for slot, e in enumerate(experts.flatten().tolist()):
        lists[e].append(slot)
    R = T * k + min(E, T * k) * (align - 1)
    rows, offsets, slots = torch.full((R,), -1), [0], torch.zeros(T * k, dtype=torch.long)
    for part in lists:
        at = offsets[-1]
        for i, slot in enumerate(part):
            rows[at + i] = slot
            slots[slot] = at + i
        offsets.append(at + -(-len(part) // align) * align)
    dev = z.device
    return (experts.int(), w, slots.view(T, k).int().to(dev), rows.int().to(dev),
            torch.tensor(offsets, dtype=torch.int32, device=dev))


def route_backward(z, experts, dw, score="softmax", renormalise=True, scale=1.0):
    """dlogits by the chain rule, from autograd in 64 bits."""
    z = z.detach().double().requires_grad_(True)
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    p = s.gather(1, experts.long())
    w = scale * (p / (p.sum(1, keepdim=True) + NIL) if renormalise else p)
    w.backward(dw.double())
    return z.grad


def close(got, want, size, blocks, extra=0.0):
    """Whether a product of codes is within what its arithmetic can be off: a block's 128 exact
    products are summed in at least 24 bits, each addition off by at most a truncated step,
    2^-23 of the block's sum of magnitudes (128 * 2^-23); its scales take two roundings and the
    total one for each block (2^-24 each). `size`: the sum of magnitudes."""
    tol = 2.0 ** -16 + (blocks + 4) * 2.0 ** -24 + extra
    err = (got.double() - want).abs()
    assert torch.isfinite(err).all()
    worst = float((err / size.clamp(min=1e-300)).max()) if err.numel() else 0.0
    assert worst <= tol, f"{worst:.3e} of the sum of magnitudes, {tol:.3e} allowed"
