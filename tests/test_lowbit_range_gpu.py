"""Values at the ends of the types' ranges in the low-bit formats and products."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import lowbit_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    rtm.build()
    rtm.load_library()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", [16, 65])
def test_w4_range_beyond_fp32(N, group):
    """Finite weights whose hi - lo overflows fp32 keep a finite scale, hi / 15 - lo / 15, and
    read back within a step."""
    gen = torch.Generator().manual_seed(N)
    W = ((torch.rand(256, N, generator=gen, dtype=torch.float64) - 0.5) * 4.8e38).to(torch.bfloat16)
    W[::16] = 2.4e38
    W[1::16] = -2.4e38
    codes, s, z = rtm.gemm_w4_quantize(W.to(DEV), group)
    fifteenth = torch.tensor(1 / 15)
    g = W.float().view(-1, group, N)
    hi, lo = g.amax(1), g.amin(1)
    assert torch.isfinite(W).all() and torch.isinf(hi - lo).all()
    want_s = (hi * fifteenth - lo * fifteenth).to(torch.bfloat16)
    inv = torch.ones_like(hi) / want_s.float()
    want_z = torch.round(-lo * inv).clamp(0, 15)
    want_q = (torch.round(g * inv[:, None]) + want_z[:, None]).clamp(0, 15).view(256, N)
    assert torch.equal(s.cpu(), want_s) and torch.equal(z.cpu(), want_z.to(torch.uint8))
    q = ref.w4_unpack(codes.cpu(), 256)
    assert torch.equal(q, want_q.to(torch.uint8))
    back = rtm.gemm_w4_dequantize(codes, s, z, 256, group).cpu().double()
    step = want_s.double()[torch.arange(256) // group]
    # a step at the clamped ends, and bf16 rounds what is read back
    assert ((back - W.double()).abs() <= step * (1 + 15 * 2.0 ** -8)).all()
