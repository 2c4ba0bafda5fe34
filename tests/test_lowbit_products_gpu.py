"""GPU tests of the products with low-bit operands: 4-bit weights and the weight
gradient from activations saved in 8 bits, against the stored values' product in
64 bits within the rounding bound of an fp32 sum."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import lowbit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


def randn(rows, cols, dtype, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=gen) * scale).to(dtype)


class Weight:
    """A 4-bit weight with random codes, on the host (q, s, z) and the GPU."""

    def __init__(self, K, N, group, zeros, dtype, seed):
        gen = torch.Generator().manual_seed(seed)
        G = (K + group - 1) // group
        self.group, self.K = group, K
        self.q = torch.randint(0, 16, (K, N), generator=gen, dtype=torch.uint8)
        self.s = (torch.rand(G, N, generator=gen) * 0.02 + 0.001).to(dtype)
        self.z = torch.randint(0, 16, (G, N), generator=gen, dtype=torch.uint8) if zeros else None
        self.codes_d = rtm.gemm_w4_pack(self.q.to(DEV))
        self.s_d = self.s.to(DEV)
        self.z_d = None if self.z is None else self.z.to(DEV)

    def values(self):
        return ref.w4_values(self.q, self.s, self.z, self.group)

    def product(self, A, **kw):
        fn = rtm.gemm_bf16w4f32 if A.dtype == torch.bfloat16 else rtm.gemm_f16w4f32
        return fn(A, self.codes_d, self.s_d, self.z_d, self.group, **kw)


def done():
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0


def check_w4(M, N, K, group, zeros, dtype, seed=0):
    W = Weight(K, N, group, zeros, dtype, seed + M + 3 * N + 5 * K)
    A = randn(M, K, dtype, seed + K)
    guard = torch.full((M * N + 64,), 7.0, device=DEV)
    C = W.product(A.to(DEV), out=guard[:M * N].view(M, N))
    done()
    assert (guard[M * N:] == 7.0).all()
    a, w = A.double(), W.values()
    ref.assert_within(C, a @ w, ref.product_bound(K, a, w))
    assert torch.equal(W.product(A.to(DEV)), C), "a second call gives other bits"


# Rows: one token, the edges of 8-row and larger tiles, more than one tile.
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64, 65, 128, 129, 255, 257, 300, 600])
@pytest.mark.parametrize("N,K,group,zeros,dtype", [
    (264, 512, 128, True, torch.bfloat16),
    (131, 456, 64, False, torch.float16),
    (72, 1000, 32, True, torch.bfloat16),
    (129, 333, 32, True, torch.float16),
])
def test_w4_rows(M, N, K, group, zeros, dtype):
    check_w4(M, N, K, group, zeros, dtype)


@pytest.mark.parametrize("K", [1, 8, 31, 32, 33, 64, 96, 127, 128, 129, 160, 256, 264, 1023, 1160, 4104, 8190])
@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_w4_depths(M, K):
    check_w4(M, 136, K, (32, 64, 128)[K % 3], K % 2 == 0, TYPES[K % 2])


@pytest.mark.parametrize("N", [1, 7, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 1030])
@pytest.mark.parametrize("M", [1, 12, 100, 260])
def test_w4_widths(M, N):
    check_w4(M, N, 264, (32, 64, 128)[N % 3], N % 2 == 0, TYPES[N % 2])


@pytest.mark.parametrize("M", [1, 3, 48, 1500])
@pytest.mark.parametrize("dtype", TYPES)
def test_w4_offset_pointers(M, dtype):
    """A, scales, zero points and C on the least alignment they may have."""
    K, N, group = 384, 200, 128
    W = Weight(K, N, group, True, dtype, 3)
    A = randn(M, K, dtype, 4)
    want = W.product(A.to(DEV))

    def off(t):
        room = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        room[1:].copy_(t.flatten())
        return room[1:].view(t.shape)

    W.s_d, W.z_d = off(W.s), off(W.z)
    out = torch.zeros(M * N + 2, device=DEV)
    got = W.product(off(A), out=out[1:-1].view(M, N))
    done()
    assert out[0] == 0 and out[-1] == 0
    w, a = W.values(), A.double()
    ref.assert_within(got, a @ w, ref.product_bound(K, a, w))
    ref.assert_within(want, a @ w, ref.product_bound(K, a, w))


@pytest.mark.parametrize("M", [6, 150])
def test_w4_nonfinite_stay_in_their_row_and_column(M):
    K, N = 300, 140
    W = Weight(K, N, 64, True, torch.bfloat16, 11)
    A = randn(M, K, torch.bfloat16, 12)
    A[1, 5] = float("inf")
    A[2, 299] = float("nan")
    A[3, 0], A[3, 1] = float("inf"), -float("inf")
    W.s[1, 7] = float("nan")
    W.s[4, 139] = float("inf")
    W.q[256:, 139] = 9
    W.z[4, 139] = 3
    W.codes_d, W.s_d, W.z_d = rtm.gemm_w4_pack(W.q.to(DEV)), W.s.to(DEV), W.z.to(DEV)
    C = W.product(A.to(DEV)).cpu()
    done()
    want = A.double() @ W.values()
    clean_rows = torch.tensor([i for i in range(M) if i not in (1, 2, 3)])
    clean_cols = torch.tensor([j for j in range(N) if j not in (7, 139)])
    a, w = A.double()[clean_rows], W.values()[:, clean_cols]
    ref.assert_within(C[clean_rows][:, clean_cols], a @ w, ref.product_bound(K, a, w))
    assert torch.isnan(C[2]).all() and torch.isnan(C[:, 7]).all()
    assert not torch.isfinite(C[1]).any() and not torch.isfinite(C[:, 139]).any()
    # one infinite product and no other: the infinity's sign is the product's
    row = want[1][clean_cols]
    inf = torch.isinf(row)
    assert inf.any() and torch.equal(C[1].double()[clean_cols][inf], row[inf])


@pytest.mark.parametrize("M", [1, 40, 300])
def test_w4_padding_codes_are_ignored(M):
    """Codes of k >= K may hold anything."""
    K, N = 200, 70
    W = Weight(K, N, 128, True, torch.float16, 1)
    A = randn(M, K, torch.float16, 2).to(DEV)
    want = W.product(A)
    for k in range(K, 256):
        r = k % 128
        byte = 64 + r % 32 // 8 * 16 + r // 32 * 4 + (4 * (r % 8 // 2) + 16 * (r % 2)) // 8
        shift = (4 * (r % 8 // 2)) % 8
        W.codes_d[:, byte] |= 15 << shift
    assert torch.equal(W.product(A), want)


def test_w4_degenerate():
    W = Weight(128, 40, 128, True, torch.bfloat16, 1)
    assert W.product(torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)).shape == (0, 40)
    E = Weight(128, 40, 128, True, torch.bfloat16, 1)
    C = rtm.gemm_bf16w4f32(torch.empty(3, 0, dtype=torch.bfloat16, device=DEV),
                           torch.empty(40, 0, dtype=torch.uint8, device=DEV),
                           torch.empty(0, 40, dtype=torch.bfloat16, device=DEV),
                           out=torch.ones(3, 40, device=DEV))
    done()
    assert (C == 0).all() and E.codes_d.shape == (40, 64)


def test_w4_quantised_weight_end_to_end():
    """The product with a quantised weight is near the dense one: within the codes' error."""
    K, N, M = 1024, 256, 32
    W, A = randn(K, N, torch.bfloat16, 1, 0.02), randn(M, K, torch.bfloat16, 2)
    codes, s, z = rtm.gemm_w4_quantize(W.to(DEV), 64)
    C = rtm.gemm_bf16w4f32(A.to(DEV), codes, s, z, 64).double().cpu()
    step = s.cpu().double()[torch.arange(K) // 64]
    err = (C - A.double() @ W.double()).abs()
    assert (err <= 1.01 * A.double().abs() @ step).all()
    # independent errors of at most a step add up like their root mean square
    rms = (A.double() ** 2 @ step ** 2).sqrt()
    assert (err.square().mean().sqrt() <= rms.square().mean().sqrt()).all()


class Saved:
    def __init__(self, M, K, seed):
        gen = torch.Generator().manual_seed(seed)
        self.q = torch.randint(-127, 128, (M, K), generator=gen).to(torch.int8)
        self.s = torch.rand((M + 127) // 128, K, generator=gen) * 0.1 + 0.001
        self.codes_d, self.s_d = ref.q8_pad(self.q).to(DEV), self.s.to(DEV)

    def values(self):
        return ref.q8_values(self.q, self.s)

    def gradient(self, dY, **kw):
        fn = rtm.gemm_q8tbf16f32 if dY.dtype == torch.bfloat16 else rtm.gemm_q8tf16f32
        return fn(self.codes_d, self.s_d, dY, **kw)


def check_q8t(M, N, K, dtype):
    X, dY = Saved(M, K, M + K), randn(M, N, dtype, N)
    guard = torch.full((K * N + 64,), 7.0, device=DEV)
    dW = X.gradient(dY.to(DEV), out=guard[:K * N].view(K, N))
    done()
    assert (guard[K * N:] == 7.0).all()
    x, d = X.values().t(), dY.double()
    # a scale times a code is not exact in fp32: one more rounding of each product
    ref.assert_within(dW, x @ d, ref.product_bound(M, x, d))
    assert torch.equal(X.gradient(dY.to(DEV)), dW), "a second call gives other bits"


@pytest.mark.parametrize("M", [1, 2, 63, 64, 65, 127, 128, 129, 191, 193, 256, 300, 1001, 4100])
@pytest.mark.parametrize("N,K,dtype", [(136, 144, torch.bfloat16), (129, 33, torch.float16)])
def test_q8t_tokens(M, N, K, dtype):
    check_q8t(M, N, K, dtype)


@pytest.mark.parametrize("K", [1, 15, 16, 17, 64, 127, 128, 129, 257, 520])
@pytest.mark.parametrize("N", [1, 8, 65, 256, 264])
def test_q8t_sizes(N, K):
    check_q8t(200, N, K, TYPES[(N + K) % 2])


@pytest.mark.parametrize("M,N,K", [(3000, 640, 512), (2500, 1030, 1000), (9000, 40, 64)])
@pytest.mark.parametrize("dtype", TYPES)
def test_q8t_larger(M, N, K, dtype):
    check_q8t(M, N, K, dtype)


def test_q8t_offset_pointers():
    M, N, K = 300, 64, 80
    X, dY = Saved(M, K, 1), randn(M, N, torch.bfloat16, 2)
    room = torch.empty(M * N + 1, dtype=torch.bfloat16, device=DEV)
    view = room[1:].view(M, N)
    view.copy_(dY)
    out = torch.zeros(K * N + 2, device=DEV)
    got = X.gradient(view, out=out[1:-1].view(K, N))
    done()
    assert out[0] == 0 and out[-1] == 0
    x, d = X.values().t(), dY.double()
    ref.assert_within(got, x @ d, ref.product_bound(M, x, d))


@pytest.mark.parametrize("M", [200, 1000])
def test_q8t_nonfinite_stay_in_their_row_and_column(M):
    N, K = 72, 90
    X, dY = Saved(M, K, 5), randn(M, N, torch.bfloat16, 6)
    X.s[1, 3] = float("nan")
    X.s[0, 4] = 0.0
    dY[150, 8] = float("nan")
    dY[5, 9] = float("inf")
    X.s_d = X.s.to(DEV)
    dW = X.gradient(dY.to(DEV)).cpu()
    done()
    want = X.values().t() @ dY.double()
    rows = torch.tensor([k for k in range(K) if k != 3])
    cols = torch.tensor([j for j in range(N) if j not in (8, 9)])
    x, d = X.values().t()[rows], dY.double()[:, cols]
    ref.assert_within(dW[rows][:, cols], x @ d, ref.product_bound(M, x, d))
    assert torch.isnan(dW[3]).all() and torch.isnan(dW[:, 8]).all()
    assert torch.equal(torch.isnan(dW[:, 9]), torch.isnan(want[:, 9]))
    inf = torch.isinf(want[:, 9])
    assert torch.equal(dW[:, 9].double()[inf], want[:, 9][inf])


def test_q8t_padding_codes_are_ignored():
    M, N, K = 260, 40, 50
    X, dY = Saved(M, K, 7), randn(M, N, torch.float16, 8).to(DEV)
    want = X.gradient(dY)
    X.codes_d[:, K:] = -128
    assert torch.equal(X.gradient(dY), want)


def test_q8t_lowest_code():
    """Codes are any int8: -128 too, which gemm_q8_quantize never writes."""
    M, N, K = 140, 24, 20
    X, dY = Saved(M, K, 9), randn(M, N, torch.bfloat16, 10)
    X.q[::3] = -128
    X.codes_d = ref.q8_pad(X.q).to(DEV)
    dW = X.gradient(dY.to(DEV))
    done()
    x, d = X.values().t(), dY.double()
    ref.assert_within(dW, x @ d, ref.product_bound(M, x, d))


def test_q8t_degenerate():
    X = Saved(128, 16, 1)
    dW = rtm.gemm_q8tbf16f32(torch.empty(0, 16, dtype=torch.int8, device=DEV),
                             torch.empty(0, 16, device=DEV),
                             torch.empty(0, 8, dtype=torch.bfloat16, device=DEV),
                             out=torch.ones(16, 8, device=DEV))
    assert (dW == 0).all()
    assert X.gradient(torch.empty(128, 0, dtype=torch.bfloat16, device=DEV)).shape == (16, 0)
    done()


def test_gradient_against_differences():
    """loss(W) = sum(Y * dY), Y = X.W with the saved X. The loss is linear in W, so a
    central difference in a direction D is its gradient there up to the rounding
    of the 64-bit losses: <dW, D>."""
    M, N, K = 333, 40, 56
    X, dY = randn(M, K, torch.bfloat16, 1), randn(M, N, torch.bfloat16, 2)
    codes, s = rtm.gemm_q8_quantize(X.to(DEV))
    dW = rtm.gemm_q8tbf16f32(codes, s, dY.to(DEV)).double().cpu()
    x = ref.q8_values(codes.cpu()[:, :K], s.cpu())
    W = randn(K, N, torch.float32, 3).double()

    def loss(w):
        return float(((x @ w) * dY.double()).sum())

    bound = ref.product_bound(M, x.t(), dY.double())
    gen = torch.Generator().manual_seed(4)
    for _ in range(8):
        D = torch.randn(K, N, generator=gen, dtype=torch.float64)
        h = 2.0 ** -10
        difference = (loss(W + h * D) - loss(W - h * D)) / (2 * h)
        size = float(((x.abs() @ (W.abs() + h * D.abs())) * dY.double().abs()).sum())
        rounding = 2 * (M * N * K) ** 0.5 * 2.0 ** -53 * size / h
        assert abs(float((dW * D).sum()) - difference) <= float((bound * D.abs()).sum()) + rounding
    # and of the activations themselves, within what 8 bits lose: half a step of each
    exact = X.double().t() @ dY.double()
    step = s.cpu().double()[torch.arange(M) // 128]
    assert ((dW - exact).abs() <= 0.51 * step.t() @ dY.double().abs() + bound).all()


def test_side_stream_and_workspace_reuse():
    """Calls on another stream, with operands that make the call use a workspace of its own."""
    side = torch.cuda.Stream()
    M, N, K = 300, 77, 131
    W, A = Weight(K, N, 64, True, torch.float16, 1), randn(M, K, torch.float16, 2).to(DEV)
    X, dY = Saved(M, K, 3), randn(M, N, torch.float16, 4).to(DEV)
    want, want_g = W.product(A), X.gradient(dY)
    torch.cuda.synchronize()
    got, got_g = [], []
    for _ in range(6):
        got.append(W.product(A, stream=side))
        got_g.append(X.gradient(dY, stream=side))
        torch.empty(1 << 20, device=DEV).fill_(3.0)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got) and all(torch.equal(g, want_g) for g in got_g)


def test_graph_capture():
    W = Weight(512, 256, 128, True, torch.bfloat16, 1)
    A = randn(4, 512, torch.bfloat16, 2).to(DEV)
    X, dY = Saved(512, 64, 3), randn(512, 256, torch.bfloat16, 4).to(DEV)
    want, want_g = W.product(A), X.gradient(dY)
    torch.cuda.synchronize()
    out, out_g = torch.zeros_like(want), torch.zeros_like(want_g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        W.product(A, out=out)
        X.gradient(dY, out=out_g)
    graph.replay()
    done()
    assert torch.equal(out, want) and torch.equal(out_g, want_g)


def test_refusals():
    W = Weight(256, 64, 128, True, torch.bfloat16, 1)
    A = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    X, dY = Saved(128, 64, 1), torch.zeros(128, 32, dtype=torch.bfloat16, device=DEV)
    f, g = rtm.gemm_bf16w4f32, rtm.gemm_q8tbf16f32
    for bad in (lambda: f(A.half(), W.codes_d, W.s_d, W.z_d),
                lambda: f(A, W.codes_d, W.s_d.half(), W.z_d),
                lambda: f(A, W.codes_d, W.s_d, W.z_d, 64),
                lambda: f(A, W.codes_d, W.s_d, W.z_d, 100),
                lambda: f(A[:, :100].contiguous(), W.codes_d, W.s_d, W.z_d),
                lambda: f(A[:, ::2], W.codes_d, W.s_d, W.z_d),
                lambda: f(A, W.codes_d.cpu(), W.s_d, W.z_d),
                lambda: f(A, W.codes_d, W.s_d, W.z_d[:1]),
                lambda: f(A, W.codes_d, W.s_d, W.z_d, out=torch.zeros(4, 63, device=DEV)),
                lambda: g(X.codes_d, X.s_d, dY.half()),
                lambda: g(X.codes_d, X.s_d, dY[:100]),
                lambda: g(X.codes_d[:, :48], X.s_d, dY),
                lambda: g(X.codes_d, X.s_d.half(), dY),
                lambda: g(X.codes_d, X.s_d, dY, out=torch.zeros(64, 33, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    out = torch.zeros(4 * 256, dtype=torch.float32, device=DEV)
    with pytest.raises(rtm.GemmError):  # C over A
        lib = rtm.load_library()
        status = lib.gemm_bf16w4f32(4, 64, 256, out.data_ptr(), W.codes_d.data_ptr(),
                                    W.s_d.data_ptr(), W.z_d.data_ptr(), 128, out.data_ptr(), 0, 0, 0)
        if status:
            raise rtm.GemmError(status, rtm.status_string(status))


@pytest.mark.parametrize("M,N,K,group", [(200, 136, 8192, 32), (48, 520, 4096, 64), (100, 136, 8192, 128),
                                         (700, 1030, 2048, 128), (3, 300, 8192, 64)])
def test_w4_repeats_exactly(M, N, K, group):
    """Many calls give the same bits, with other work between them: nothing is read
    before it has arrived or after its place has been given away."""
    W = Weight(K, N, group, True, torch.bfloat16, 1)
    A = randn(M, K, torch.bfloat16, 2).to(DEV)
    want = W.product(A)
    a, w = A.double().cpu(), W.values()
    ref.assert_within(want, a @ w, ref.product_bound(K, a, w))
    for i in range(60):
        if i % 3 == 0:
            torch.randn(2_000_000, device=DEV)
        assert torch.equal(W.product(A), want)
    done()


@pytest.mark.parametrize("M,N,K", [(9000, 264, 520), (9000, 64, 64), (5000, 1030, 700), (4096, 100, 256)])
def test_q8t_repeats_exactly(M, N, K):
    X, dY = Saved(M, K, 1), randn(M, N, torch.bfloat16, 2).to(DEV)
    want = X.gradient(dY)
    for i in range(60):
        if i % 3 == 0:
            torch.randn(2_000_000, device=DEV)
        assert torch.equal(X.gradient(dY), want)
    done()


@pytest.mark.parametrize("M", [17, 60, 128, 300])
def test_timeout_is_reported_and_the_context_stays_usable(M):
    """With the loads muted every bounded wait runs out: one status, and the next call is right."""
    W = Weight(1024, 300, 64, True, torch.bfloat16, 1)
    A = randn(M, 1024, torch.bfloat16, 2).to(DEV)
    want = W.product(A)
    rtm.gemm_bf16w4f32_selftest_timeout(A, W.codes_d, W.s_d, W.z_d, W.group,
                                        torch.empty_like(want), 20_000_000)
    assert rtm.STATUS[rtm.get_device_error()] == "GEMM_ERR_TIMEOUT"
    assert torch.equal(W.product(A), want)
    X, dY = Saved(400, 130, 3), randn(400, 8 * M, torch.bfloat16, 4).to(DEV)
    want = X.gradient(dY)
    rtm.gemm_q8tbf16f32_selftest_timeout(X.codes_d, X.s_d, dY, torch.empty_like(want), 20_000_000)
    assert rtm.STATUS[rtm.get_device_error()] == "GEMM_ERR_TIMEOUT"
    assert torch.equal(X.gradient(dY), want)
    done()


def test_workspace_given_or_refused():
    """Rows off 16-byte boundaries: with a workspace, with one too small and with none
    (the binding's own) the sums differ in order only; one over an operand is refused."""
    M, N, K = 300, 77, 131
    W, A = Weight(K, N, 64, True, torch.float16, 1), randn(M, K, torch.float16, 2).to(DEV)
    need = rtm.gemm_w4_workspace_bytes(M, N, K)
    assert need == (M * 136 * 2 + 255) // 256 * 256 and rtm.gemm_w4_workspace_bytes(16, N, K) == 0
    a, w = A.double().cpu(), W.values()
    bound = ref.product_bound(K, a, w)
    for nbytes in (need, 16):
        C = W.product(A, workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV))
        done()
        ref.assert_within(C, a @ w, bound)
    with pytest.raises(rtm.GemmError):
        out = torch.empty(M + need, N, device=DEV)
        W.product(A, out=out[:M], workspace=out)
    X, dY = Saved(M, 90, 3), randn(M, N, torch.float16, 4).to(DEV)
    x, d = X.values().t(), dY.double().cpu()
    for nbytes in (rtm.gemm_q8t_workspace_bytes(M, N, 90), 16):
        dW = X.gradient(dY, workspace=torch.empty(nbytes, dtype=torch.uint8, device=DEV))
        done()
        ref.assert_within(dW, x @ d, ref.product_bound(M, x, d))
