"""The low-bit formats and products on the host, from their definitions: the
conversions step by step in fp32 as include/gemm.h states them (every step is
an IEEE operation, so codes and scales are compared bit for bit), the products
in 64 bits."""

import numpy as np
import torch

TINY = 2.0 ** -100


def f32(x):
    return torch.tensor(x, dtype=torch.float32)


def w4_quantize(W, group, zeros):
    """(q K x N uint8, scales, zero points or None) of a 2-byte CPU tensor."""
    K, N = W.shape
    w = W.float()
    qs, ss, zs = [], [], []
    for k0 in range(0, K, group):
        g = w[k0:k0 + group]
        finite = torch.isfinite(g).all(0)
        hi, lo = g.amax(0).clamp(min=0), g.amin(0).clamp(max=0)
        s = (hi - lo) * f32(1 / 15) if zeros else torch.maximum(hi, -lo) * f32(1 / 7)
        s = torch.where(finite, s, f32(float("nan"))).to(W.dtype)
        s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
        sf = s.float()
        inv = torch.where(sf == 0, torch.zeros_like(sf), torch.ones_like(sf) / sf)
        z = torch.full_like(sf, 8.0)
        if zeros:
            z = torch.nan_to_num(torch.round(-lo * inv), nan=0.0).clamp(0, 15)
        q = torch.nan_to_num(torch.round(g * inv) + z, nan=0.0).clamp(0, 15)
        qs.append(q)
        ss.append(s)
        zs.append(z)
    return (torch.cat(qs).to(torch.uint8), torch.stack(ss),
            torch.stack(zs).to(torch.uint8) if zeros else None)


def w4_pack(q):
    """N x ceil(K / 128) * 64 bytes, code by code from the layout's description."""
    q = q.numpy()
    K, N = q.shape
    out = np.zeros((N, (K + 127) // 128 * 64), dtype=np.uint8)
    for k in range(K):
        block, r = divmod(k, 128)
        w, r = divmod(r, 32)
        c, i = divmod(r, 8)
        bit = 4 * (i // 2) + 16 * (i % 2)
        byte = block * 64 + c * 16 + w * 4 + bit // 8
        out[:, byte] |= (q[k] & 15) << (bit % 8)
    return torch.from_numpy(out)


def w4_unpack(codes, K):
    codes = codes.numpy()
    q = np.empty((K, codes.shape[0]), dtype=np.uint8)
    for k in range(K):
        block, r = divmod(k, 128)
        w, r = divmod(r, 32)
        c, i = divmod(r, 8)
        bit = 4 * (i // 2) + 16 * (i % 2)
        byte = block * 64 + c * 16 + w * 4 + bit // 8
        q[k] = (codes[:, byte] >> (bit % 8)) & 15
    return torch.from_numpy(q)


def w4_values(q, s, z, group):
    """(q - z) * s, K x N in 64 bits."""
    g = torch.arange(q.shape[0]) // group
    zz = 8.0 if z is None else z.double()[g]
    return (q.double() - zz) * s.double()[g]


def q8_quantize(X):
    """(codes M x K int8, scales) of a 2-byte CPU tensor."""
    x = X.float()
    qs, ss = [], []
    for m0 in range(0, x.shape[0], 128):
        g = x[m0:m0 + 128]
        finite = torch.isfinite(g).all(0)
        amax = torch.nan_to_num(g.abs(), nan=0.0).amax(0)
        s = torch.where(amax < TINY, torch.zeros_like(amax), amax * f32(1 / 127))
        s = torch.where(finite, s, f32(float("nan")))
        inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
        q = torch.nan_to_num(torch.round(g * inv), nan=0.0, posinf=0.0, neginf=0.0)
        qs.append(q.clamp(-127, 127))
        ss.append(s)
    return torch.cat(qs).to(torch.int8), torch.stack(ss)


def q8_pad(q):
    return torch.nn.functional.pad(q, (0, -q.shape[1] % 16)).contiguous()


def q8_values(q, s):
    return q.double() * s.double()[torch.arange(q.shape[0]) // 128]


def product_bound(depth, left, right):
    """Largest error of an fp32 sum of `depth` products in any order, to first
    order: each of fewer than depth + 16 additions (the 16: the scales of the
    groups and partial sums that are joined) rounds a partial sum, which is at
    most the sum of magnitudes, by half a unit in the last place, 2^-24."""
    return (depth + 16) * 2.0 ** -24 * (left.abs() @ right.abs())


def assert_within(got, want, bound):
    got = got.double().cpu()
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~finite & ~torch.isnan(want)], want[~finite & ~torch.isnan(want)])
    over = (got - want).abs()[finite] - bound[finite]
    assert not (over > 0).any(), f"{int((over > 0).sum())} outputs off by up to {float(over.max())} over the bound"
