"""Seeded fuzz of the low-bit entry points over sizes, groups, zero points, types and
alignments, and their first calls from many threads at once."""

import os
import random
import subprocess
import sys
import textwrap

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import lowbit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


def size(rng, high):
    edge = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257]
    return min(high, rng.choice(edge) if rng.random() < 0.4 else int(high ** rng.random()))


def placed(rng, t):
    """t on the GPU, on the allocator's alignment or one element past it."""
    if rng.random() < 0.5:
        return t.to(DEV)
    room = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
    room[1:].copy_(t.flatten())
    return room[1:].view(t.shape)


def randn(rng, rows, cols, dtype, scale=1.0):
    gen = torch.Generator().manual_seed(rng.randrange(1 << 30))
    return (torch.randn(rows, cols, generator=gen) * scale).to(dtype)


@pytest.mark.parametrize("seed", range(60))
def test_w4(seed):
    rng = random.Random(seed)
    M, N, K = size(rng, 700), size(rng, 3000), size(rng, 3000)
    group, zeros, dtype = rng.choice([32, 64, 128]), rng.random() < 0.5, rng.choice(TYPES)
    W, A = randn(rng, K, N, dtype, 0.02), randn(rng, M, K, dtype)
    codes, s, z = rtm.gemm_w4_quantize(placed(rng, W), group, zeros=zeros)
    q0, s0, z0 = ref.w4_quantize(W, group, zeros)
    assert torch.equal(s.cpu(), s0) and torch.equal(ref.w4_unpack(codes.cpu(), K), q0)
    assert z is None if z0 is None else torch.equal(z.cpu(), z0)
    product = rtm.gemm_bf16w4f32 if dtype == torch.bfloat16 else rtm.gemm_f16w4f32
    s_d, z_d = placed(rng, s0), None if z0 is None else placed(rng, z0)
    C = product(placed(rng, A), codes, s_d, z_d, group, out=placed(rng, torch.zeros(M, N)))
    a, w = A.double(), ref.w4_values(q0, s0, z0, group)
    ref.assert_within(C, a @ w, ref.product_bound(K, a, w))
    back = rtm.gemm_w4_dequantize(codes, s_d, z_d, K, group)
    assert torch.equal(back.cpu(), w.float().to(dtype))  # a code times a scale is exact in fp32
    assert rtm.get_device_error() == 0


@pytest.mark.parametrize("seed", range(60))
def test_q8(seed):
    rng = random.Random(1000 + seed)
    M, N, K = size(rng, 3000), size(rng, 1500), size(rng, 1500)
    dtype = rng.choice(TYPES)
    X, dY = randn(rng, M, K, dtype), randn(rng, M, N, dtype)
    codes, s = rtm.gemm_q8_quantize(placed(rng, X))
    q0, s0 = ref.q8_quantize(X)
    assert torch.equal(s.cpu(), s0) and torch.equal(codes.cpu(), ref.q8_pad(q0))
    block = torch.arange(M) // 128
    back = rtm.gemm_q8_dequantize(codes, s, M, K, dtype)
    assert torch.equal(back.cpu(), (q0.float() * s0[block]).to(dtype))
    gradient = rtm.gemm_q8tbf16f32 if dtype == torch.bfloat16 else rtm.gemm_q8tf16f32
    dW = gradient(codes, placed(rng, s0), placed(rng, dY), out=placed(rng, torch.zeros(K, N)))
    x, d = ref.q8_values(q0, s0).t(), dY.double()
    ref.assert_within(dW, x @ d, ref.product_bound(M, x, d))
    assert rtm.get_device_error() == 0


# Integers and scales of powers of two: exact sums, equal outputs.
CHILD = textwrap.dedent(r"""
    import sys, threading
    sys.path.insert(0, sys.argv[1])
    import torch
    import register_tiled_matrix_gb300 as rtm

    gen = torch.Generator("cuda").manual_seed(5)
    ints = lambda m, n, high, t: torch.randint(-high, high + 1, (m, n), generator=gen,
                                               device="cuda").to(t)
    jobs = []
    for i, (M, N, K) in enumerate([(1, 300, 512), (4, 10001, 264), (16, 520, 1000), (20, 264, 512),
                                   (50, 131, 456), (100, 1030, 200), (300, 520, 512), (300, 77, 131),
                                   (1, 520, 333), (7, 64, 1024), (600, 264, 264), (33, 4000, 128)]):
        dtype = (torch.bfloat16, torch.float16)[i % 2]
        if i % 3 == 2:  # gradient: M tokens
            x, y = ints(M, -(-K // 16) * 16, 127, torch.int8), ints(M, N, 2, dtype)
            s = torch.full((-(-M // 128), K), 0.5, device="cuda")
            f = rtm.gemm_q8tbf16f32 if i % 2 == 0 else rtm.gemm_q8tf16f32
            jobs.append((f, (x, s, y), x[:, :K].double().t() @ y.double() * 0.5))
        else:
            q, x = ints(K, N, 7, torch.int8).add(8).to(torch.uint8), ints(M, K, 2, dtype)
            s = torch.full((-(-K // 128), N), 0.5, dtype=dtype, device="cuda")
            f = rtm.gemm_bf16w4f32 if i % 2 == 0 else rtm.gemm_f16w4f32
            codes = torch.zeros(N, -(-K // 128) * 64, dtype=torch.uint8, device="cuda")
            k = torch.arange(K, device="cuda")
            r = k % 128
            bit = 4 * (r % 8 // 2) + 16 * (r % 2)
            byte = k // 128 * 64 + r % 32 // 8 * 16 + r // 32 * 4 + bit // 8
            codes.index_add_(1, byte, (q.int() << (bit % 8)[:, None]).to(torch.uint8).t().contiguous())
            jobs.append((f, (x, codes, s), x.double() @ (q.double() - 8) * 0.5))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    results, errors, barrier = [None] * len(jobs), [], threading.Barrier(len(jobs))

    def work(i):
        try:
            f, args, _ = jobs[i]
            barrier.wait()
            for _ in range(3):
                results[i] = f(*args, stream=streams[i])
            streams[i].synchronize()
        except Exception as e:
            errors.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    wrong = [i for i in range(len(jobs)) if results[i] is None
             or not torch.equal(results[i].double(), jobs[i][2])]
    if errors or wrong or rtm.get_device_error() != 0:
        print(errors, wrong); sys.exit(2)
    print("ok")
""")


def test_first_calls_from_many_threads():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.strip().endswith("ok")
