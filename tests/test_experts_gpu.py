"""The experts' products over rows in their order, the weighted sum of them, and a run of all the
operators as a layer of experts: against 64-bit products of the values that are held."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref
from tests.test_f8_products_gpu import blocks, codes, scales

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KEPT = -77.0  # what rows hold that no product may write


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()
    yield
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0


def stack(E, K, N, seed):
    pitch = (N + 15) // 16 * 16
    w = codes(E * K, N, seed).as_strided((E, K, N), (K * pitch, pitch, 1))
    return w, scales(E, blocks(K), blocks(N), seed=seed)


def parts(lengths, first=0):
    o = [first]
    for n in lengths:
        o.append(o[-1] + n)
    return o


def device(o):
    return torch.tensor(o, dtype=torch.int32, device=DEV)


def check_rows(direction, o, R, K, N, E, given=None, seed=0):
    """o: the offsets as they count; `given`: as they are handed over."""
    w, t = stack(E, K, N, seed + 1)
    inner = K if direction == "forward" else N
    a, s = codes(R, inner, seed), scales(R, blocks(inner), seed=seed)
    out = torch.full((R, N if direction == "forward" else K), KEPT, device=DEV)
    call = rtm.gemm_f8w8f32_experts if direction == "forward" else rtm.gemm_f8w8tf32_experts
    offsets = device(given if given is not None else o)
    call(a, s, w, t, offsets, out=out)
    left = ref.values(a, s, "rows")
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        right = ref.values(w[e], t[e], "tiles")
        right = right if direction == "forward" else right.t()
        ref.close(out[rows], left[rows] @ right, left[rows].abs() @ right.abs(), blocks(inner))
    assert (out[:o[0]] == KEPT).all() and (out[o[-1]:] == KEPT).all(), "rows of no expert are kept"
    again = torch.full_like(out, KEPT)
    call(a, s, w, t, offsets, out=again)
    assert torch.equal(out, again)


LENGTHS = {"one each": [1] * 8, "single token": [0, 0, 1, 0, 0, 0, 0, 0], "none": [0] * 8,
           "all to one": [0, 0, 0, 900, 0, 0, 0, 0], "ragged": [3, 130, 0, 17, 256, 1, 64, 5],
           "long": [700, 1, 300, 0, 511, 257, 128, 90], "longer": [2100, 900, 0, 1300, 40, 777, 1, 2048]}


@pytest.mark.parametrize("direction", ["forward", "input"])
@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("K,N", [(128, 128), (300, 259), (600, 1100)])
def test_rows_by_expert(direction, name, K, N):
    o = parts(LENGTHS[name])
    check_rows(direction, o, o[-1] + 37, K, N, 8, seed=K)


@pytest.mark.parametrize("direction", ["forward", "input"])
@pytest.mark.parametrize("K,N", [(1100, 1028), (1102, 1030)])
def test_rows_by_expert_of_large_tiles(direction, K, N):
    """Experts that end at, before and behind the 32 rows that are stored at a time."""
    lengths = [n for m in range(14) for n in (256 + m, 32 * m, 33 * m, 255 - m, 31)]
    o = parts(lengths, first=3)
    check_rows(direction, o, o[-1] + 29, K, N, len(lengths), seed=N)


@pytest.mark.parametrize("E,most", [(1, 300), (200, 7), (1024, 3), (64, 200)])
def test_numbers_of_experts(E, most):
    g = torch.Generator().manual_seed(E)
    o = parts(torch.randint(0, most + 1, (E,), generator=g).tolist(), first=5)
    check_rows("forward", o, o[-1] + 3, 130, 70, E)
    check_rows("input", o, o[-1] + 3, 130, 70, E)


def test_offsets_out_of_order_stay_inside():
    """Each entry counts as at least the one before it, from 0 to the number of rows."""
    check_rows("forward", [0, 50, 50, 90, 100], 100, 64, 64, 4, given=[-5, 50, 20, 90, 2 ** 31 - 1])
    check_rows("input", [100] * 5, 100, 64, 64, 4, given=[400, -3, 200, 100, 7])
    check_rows("forward", [0] * 5, 300, 64, 64, 4, given=[-1, -2 ** 31, 0, -9, 0])


def check_weight(lengths, K, N, extra=0, seed=0):
    E, o = len(lengths), parts([-(-n // 128) * 128 for n in lengths])
    R = o[-1] + extra
    x, y = codes(max(R, 1), K, seed)[:R], codes(max(R, 1), N, seed + 1)[:R]
    for e in range(E):  # zeros after each expert's last row
        x.view(torch.uint8)[o[e] + lengths[e]:o[e + 1]] = 0
        y.view(torch.uint8)[o[e] + lengths[e]:o[e + 1]] = 0
    s, t = scales(blocks(R), K, seed=seed), scales(blocks(R), N, seed=seed + 1)
    got = rtm.gemm_f8tf8f32_experts(x, s, y, t, device(o))
    assert got.shape == (E, K, N)
    left, right = ref.values(x, s, "columns").t(), ref.values(y, t, "columns")
    for e in range(E):
        rows = slice(o[e], o[e + 1])
        if lengths[e] == 0:
            assert not got[e].any()
            continue
        a, b = left[:, rows], right[rows]
        ref.close(got[e], a @ b, a.abs() @ b.abs(), blocks(lengths[e]))
    assert torch.equal(got, rtm.gemm_f8tf8f32_experts(x, s, y, t, device(o)))


@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("K,N", [(128, 128), (300, 259), (600, 1100)])
def test_weight_gradients(name, K, N):
    check_weight(LENGTHS[name], K, N, extra=0 if name == "long" else 128, seed=N)


def test_weight_gradients_of_many_experts():
    check_weight([(i * 37) % 300 for i in range(100)], 140, 70)
    check_weight([5000], 200, 300)


def test_weight_gradient_offsets_stay_inside():
    x, y = codes(384, 130, 1), codes(384, 70, 2)
    s, t = scales(3, 130), scales(3, 70)
    got = rtm.gemm_f8tf8f32_experts(x, s, y, t, device([0, 5000, 128, -7, 384]))
    whole = rtm.gemm_f8tf8f32(x, s, y, t)
    left, right = ref.values(x, s, "columns").t(), ref.values(y, t, "columns")
    ref.close(got[0], left @ right, left.abs() @ right.abs(), 3)
    ref.close(whole, left @ right, left.abs() @ right.abs(), 3)
    assert not got[1:].any()


def test_no_rows_and_empty_sums():
    F8 = torch.float8_e4m3fn
    w, t = stack(3, 64, 32, 1)
    none = torch.empty(0, 64, dtype=torch.uint8, device=DEV).view(F8)
    o = device([0, 0, 0, 0])
    assert rtm.gemm_f8w8f32_experts(none, torch.empty(0, 1, device=DEV), w, t, o).shape == (0, 32)
    y = torch.empty(0, 32, dtype=torch.uint8, device=DEV).view(F8)
    dw = rtm.gemm_f8tf8f32_experts(none, torch.empty(0, 64, device=DEV), y,
                                   torch.empty(0, 32, device=DEV), o)
    assert dw.shape == (3, 64, 32) and not dw.any()


# ------------------------------------------------------------ joining


@pytest.mark.parametrize("T,k,N,R", [(1, 1, 1, 1), (5, 2, 7, 12), (300, 8, 1000, 2500),
                                     (64, 32, 1024, 70), (33, 3, 4100, 99)])
def test_join(T, k, N, R):
    g = torch.Generator(device=DEV).manual_seed(T)
    c = torch.randn(R, N, generator=g, device=DEV)
    slots = torch.randint(-1, R + 1, (T, k), generator=g, device=DEV, dtype=torch.int32)
    slots[0, 0] = 2 ** 31 - 1
    fine = (slots >= 0) & (slots < R)
    picked = torch.where(fine[..., None], c.double()[slots.long().clamp(0, R - 1)], 0.0)
    w = torch.randn(T, k, generator=g, device=DEV)
    for weights in (None, w):
        p = picked if weights is None else picked * w.double()[..., None]
        got = rtm.gemm_experts_join(c, slots, weights)
        assert ((got.double() - p.sum(1)).abs() <= k * 2.0 ** -24 * p.abs().sum(1) + 1e-37).all()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        dy = torch.randn(T, N, generator=g, device=DEV).to(dtype)
        got = rtm.gemm_experts_join_backward(dy, c, slots)
        p = dy.double()[:, None] * picked
        assert ((got.double() - p.sum(-1)).abs() <=
                (N / 32 + 8) * 2.0 ** -24 * p.abs().sum(-1) + 1e-37).all()
    odd = torch.randn(R * N + 1, generator=g, device=DEV)[1:].view(R, N)  # off 16 bytes
    assert torch.equal(rtm.gemm_experts_join(odd, slots, w),
                       rtm.gemm_experts_join(odd.clone(), slots, w))


def test_join_of_nothing():
    none = torch.empty(0, 2, dtype=torch.int32, device=DEV)
    c = torch.ones(4, 8, device=DEV)
    assert rtm.gemm_experts_join(c, none).shape == (0, 8)
    assert rtm.gemm_experts_join_backward(torch.ones(0, 8, device=DEV), c, none).shape == (0, 2)
    some = torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    assert not rtm.gemm_experts_join(torch.empty(0, 8, device=DEV), some).any()
    assert not rtm.gemm_experts_join_backward(torch.ones(3, 8, device=DEV),
                                              torch.empty(0, 8, device=DEV), some).any()


# ------------------------------------------------------------ as a layer


@pytest.mark.parametrize("T,E,k,K,N,align", [(1, 16, 4, 200, 130, 1), (40, 16, 4, 200, 130, 128),
                                             (40, 256, 8, 256, 128, 1), (900, 8, 2, 520, 300, 128),
                                             (900, 8, 2, 520, 300, 1)])
def test_a_layer_of_experts(T, E, k, K, N, align):
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    z = torch.randn(T, E, generator=g, device=DEV)
    w = torch.randn(E, K, N, generator=g, device=DEV).bfloat16() * 0.05
    wq, ws = rtm.gemm_f8_quantize_tiles(w)
    experts, weights, slots, rows, offsets = rtm.gemm_route(z, k, align=align)
    a, s = rtm.gemm_f8_quantize(x, "rows", gather=rows, fan=k)
    y = rtm.gemm_experts_join(rtm.gemm_f8w8f32_experts(a, s, wq, ws, offsets), slots, weights)
    held, hs = ref.quantize(x, "rows")
    left = held * ref.spread(hs, 1, 128, T, K)
    want, size = (torch.zeros(T, N, dtype=torch.float64, device=DEV) for _ in range(2))
    for j in range(k):
        for e in range(E):
            at = (experts[:, j] == e).nonzero()[:, 0]
            v = ref.values(wq[e], ws[e], "tiles")
            f = weights[at, j].double()[:, None]
            want[at] += f * (left[at] @ v)
            size[at] += f * (left[at].abs() @ v.abs())
    ref.close(y, want, size, blocks(K), extra=(k + 1) * 2.0 ** -24)


def test_gradients_of_a_layer_of_experts():
    """dX, dW and dlogits of sum(y * dy) for the values that are held, by autograd in 64 bits."""
    T, E, k, K, N = 300, 8, 2, 260, 140
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    z = torch.randn(T, E, generator=g, device=DEV)
    wq, ws = rtm.gemm_f8_quantize_tiles(torch.randn(E, K, N, generator=g, device=DEV).bfloat16())
    dy = torch.randn(T, N, generator=g, device=DEV).bfloat16()
    experts, weights, slots, rows, offsets = rtm.gemm_route(z, k)
    a, s, ac, sc = rtm.gemm_f8_quantize(x, "both", gather=rows, fan=k)
    c = rtm.gemm_f8w8f32_experts(a, s, wq, ws, offsets)
    d, ds, dc, dcs = rtm.gemm_f8_quantize(dy, "both", gather=rows, fan=k, factors=weights)
    dx = rtm.gemm_experts_join(rtm.gemm_f8w8tf32_experts(d, ds, wq, ws, offsets), slots)
    dw = rtm.gemm_f8tf8f32_experts(ac, sc, dc, dcs, offsets)
    dweights = rtm.gemm_experts_join_backward(dy, c, slots)
    dz = rtm.gemm_route_backward(z, experts, dweights)

    used = rows >= 0
    token, slot = rows[used].long() // k, rows[used].long()
    expert = experts.flatten()[slot].long()
    by_rows, by_columns = ref.values(d, ds, "rows")[used], ref.values(dc, dcs, "columns")[used]
    xv = ref.values(ac, sc, "columns")[used]
    v = ref.values(wq, ws, "tiles")
    want, size = (torch.zeros(T, K, dtype=torch.float64, device=DEV) for _ in range(2))
    for e in range(E):
        at = expert == e
        want.index_add_(0, token[at], by_rows[at] @ v[e].t())
        size.index_add_(0, token[at], by_rows[at].abs() @ v[e].abs().t())
        ref.close(dw[e], xv[at].t() @ by_columns[at], xv[at].abs().t() @ by_columns[at].abs(), 5)
    ref.close(dx, want, size, blocks(N), extra=k * 2.0 ** -24)
    # dweights and dlogits through the products as they were rounded
    p = dy.double()[:, None] * c.double()[slots.long()]
    assert ((dweights.double() - p.sum(-1)).abs() <= 16 * 2.0 ** -24 * p.abs().sum(-1)).all()
    wz = ref.route_backward(z, experts, dweights)
    total = ref.scores(z, "softmax").gather(1, experts.long()).sum(1, keepdim=True)
    size = dweights.abs().double().amax(1, keepdim=True) / total
    assert ((dz.double() - wz).abs() <= 2.0 ** -14 * size).all()
    # The held gradients are the exact ones but for the codes' half step, 2^-4 of a value: dW's
    # terms are off by two of them (X's and dC's) and what they make together.
    f = weights.double().flatten()[slot][:, None]
    full, xf = dy.double()[token] * f, x.double()[token]
    for e in range(E):
        at = expert == e
        off = (dw[e].double() - xf[at].t() @ full[at]).abs()
        # values far below their block's largest lose up to 2^-10 of 448ths of it instead
        assert (off <= 0.14 * (xf[at].abs().t() @ full[at].abs()) + 1e-2 * off.new_tensor(float(at.sum()))).all()


def test_refusals():
    w, t = stack(3, 64, 32, 1)
    a, s, o = codes(10, 64, 2), scales(10, 1), device([0, 4, 6, 10])
    y, u, x, v = codes(10, 32, 3), scales(1, 32), codes(10, 64, 4), scales(1, 64)
    slots = torch.zeros(5, 2, dtype=torch.int32, device=DEV)
    c = torch.ones(10, 32, device=DEV)
    calls = [lambda: rtm.gemm_f8w8f32_experts(a, s, w, t, o[:3]),
             lambda: rtm.gemm_f8w8f32_experts(a, s, w, t, o.long()),
             lambda: rtm.gemm_f8w8f32_experts(a, s, w, t, o.cpu()),
             lambda: rtm.gemm_f8w8f32_experts(a, s, w[0], t, o),
             lambda: rtm.gemm_f8w8f32_experts(a, s, w, t[0], o),
             lambda: rtm.gemm_f8w8f32_experts(a, s, w[:, :32], t, o),
             lambda: rtm.gemm_f8w8tf32_experts(a, s, w, t, o),
             lambda: rtm.gemm_f8tf8f32_experts(x, v, y, u, o[:1]),
             lambda: rtm.gemm_f8tf8f32_experts(x, v, y[:9], u, o),
             lambda: rtm.gemm_f8tf8f32_experts(x, v, y, u, o, out=torch.empty(64, 32, device=DEV)),
             lambda: rtm.gemm_experts_join(c, slots.long()), lambda: rtm.gemm_experts_join(c.half(), slots),
             lambda: rtm.gemm_experts_join(c, slots, torch.ones(5, 3, device=DEV)),
             lambda: rtm.gemm_experts_join(c.t(), slots),
             lambda: rtm.gemm_experts_join(c, slots, out=torch.empty(5, 31, device=DEV)),
             lambda: rtm.gemm_experts_join_backward(c[:5].double(), c, slots),
             lambda: rtm.gemm_experts_join_backward(c[:4], c, slots),
             lambda: rtm.gemm_experts_join_backward(c[:5, :31].contiguous(), c, slots)]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
