"""Large conversions along rows at every alignment of the rows: equal to the definition."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from tests import f8_reference as ref
from tests.test_f8_formats_gpu import TYPES, check, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()


@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("M,K", [(2100, 8191), (2100, 8200), (4200, 4100), (66000, 130), (131100, 9)])
def test_many_rows(M, K, type_):
    x = values(M, K, TYPES[type_], seed=K)
    x[5, 3], x[M - 1, K - 1], x[7] = torch.nan, torch.inf, 0
    check(*rtm.gemm_f8_quantize(x, "rows"), x, "rows")
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = torch.randint(-1, 2 * M, (M + 33,), generator=g, device=DEV, dtype=torch.int32)
    factors = torch.randn(M, 2, generator=g, device=DEV)
    for f in (None, factors):
        got = rtm.gemm_f8_quantize(x, "rows", gather=rows, fan=2, factors=f)
        check(*got, ref.gathered(x, rows, 2, f), "rows")
