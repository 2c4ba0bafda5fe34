"""Reuse of the raw slots of the low-bit tensor-core kernel: a slot goes back to the
copies only when the words loaded from it have arrived. Operands are small integers
with scales of powers of two, so every sum is exact and a single wrong word shows."""

import os
import re

import pytest
import torch

import register_tiled_matrix_gb300 as rtm

DEV = "cuda:0"
SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "register_tiled_matrix_gb300", "csrc", "lowbit_tc.cu")


@pytest.mark.cpu
def test_the_release_depends_on_the_loaded_words():
    """Read from the source: a slot is released in one place, whose arrival takes its address
    from the loaded words (the race cannot be shown by running it)."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    assert not re.search(r"\barrive\w*(<\w+>)?\(raw_empty", text)
    assert len(re.findall(r"\bfree_slot\(raw_empty_at \+ raw\.at \* 8, q,", text)) == 2  # w4, q8
    body = text[text.index("void free_slot("):]
    body = body[:body.index("\n}")]
    for word in ("q[0].x", "q[1].x", "q[2].x", "q[3].x", "__any_sync(0xffffffff", "& nil"):
        assert word in body
    assert re.search(r"arrive\(bar \+ none\)", body)


def integers(rows, cols, high, gen, dtype):
    return torch.randint(-high, high + 1, (rows, cols), generator=gen, device=DEV).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,group", [(20, 300, 20000, 128), (50, 520, 16384, 64),
                                         (100, 264, 16520, 32), (300, 1030, 12296, 128)])
def test_w4_slots(M, N, K, group, dtype):
    rtm.build()
    gen = torch.Generator(DEV).manual_seed(K + M)
    q = torch.randint(0, 16, (K, N), generator=gen, device=DEV, dtype=torch.uint8)
    z = torch.randint(0, 16, (-(-K // group), N), generator=gen, device=DEV, dtype=torch.uint8)
    s = torch.full(z.shape, 0.5, dtype=dtype, device=DEV)
    A = integers(M, K, 2, gen, dtype)
    codes = rtm.gemm_w4_pack(q)
    g = torch.arange(K, device=DEV) // group
    want = A.double() @ (q.double() - z.double()[g]) * 0.5  # below 2^24 halves: exact in fp32
    product = rtm.gemm_bf16w4f32 if dtype == torch.bfloat16 else rtm.gemm_f16w4f32
    for i in range(30):
        if i % 3 == 0:
            torch.randn(2_000_000, device=DEV)
        assert torch.equal(product(A, codes, s, z, group).double(), want)
    assert rtm.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(20000, 64, 130), (17001, 104, 272), (12345, 520, 400)])
def test_q8_slots(M, N, K, dtype):
    rtm.build()
    gen = torch.Generator(DEV).manual_seed(M)
    codes = integers(M, -(-K // 16) * 16, 127, gen, torch.int8)
    s = torch.full((-(-M // 128), K), 0.25, device=DEV)
    dY = integers(M, N, 2, gen, dtype)
    want = codes[:, :K].double().t() @ dY.double() * 0.25  # below 2^24 quarters
    gradient = rtm.gemm_q8tbf16f32 if dtype == torch.bfloat16 else rtm.gemm_q8tf16f32
    for i in range(30):
        if i % 3 == 0:
            torch.randn(2_000_000, device=DEV)
        assert torch.equal(gradient(codes, s, dY).double(), want)
    assert rtm.get_device_error() == 0
