"""CPU tests of how the 8-bit floating-point entry points take views of codes. The tensors say
that they are on a GPU; every call here ends in the binding's checks, before any CUDA call."""

import pytest
import torch

import register_tiled_matrix_gb300 as rtm
from register_tiled_matrix_gb300 import f8

pytestmark = pytest.mark.cpu


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""

    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def codes(*shape):
    return torch.zeros(shape, dtype=torch.uint8).view(torch.float8_e4m3fn).as_subclass(OnDevice)


# Views whose rows (matrices) are one and the same memory: their stride of 0 is no row pitch.
REPEATED = {
    "rows": lambda: codes(1, 64).expand(128, 64),
    "rows of a wide buffer": lambda: codes(1, 512)[:, :64].expand(128, 64),
    "one column": lambda: codes(1, 1).expand(40, 1),
    "rows of one matrix": lambda: codes(1, 1, 64).expand(1, 256, 64),
    "rows of several": lambda: codes(3, 1, 64).expand(3, 256, 64),
    "matrices": lambda: codes(1, 256, 64).expand(3, 256, 64),
    "matrices of one row": lambda: codes(1, 1, 64).expand(3, 1, 64),
}


@pytest.mark.parametrize("view", REPEATED)
def test_repeated_rows_are_refused(view):
    t = REPEATED[view]()
    with pytest.raises(ValueError, match="neighbours"):
        f8._codes("codes", t, t.dim(), 0)


def test_repeated_rows_are_refused_by_the_calls():
    a, w = codes(128, 64), codes(64, 64)
    rows, tiles = codes(1, 64).expand(128, 64), codes(1, 64).expand(64, 64)
    stack = codes(1, 1, 64).expand(1, 64, 64)
    s = torch.ones(1).as_subclass(OnDevice)
    for call in (lambda: rtm.gemm_f8w8f32(rows, s, w, s), lambda: rtm.gemm_f8w8f32(a, s, tiles, s),
                 lambda: rtm.gemm_f8w8tf32(rows, s, w, s), lambda: rtm.gemm_f8w8tf32(a, s, tiles, s),
                 lambda: rtm.gemm_f8tf8f32(rows, s, a, s), lambda: rtm.gemm_f8tf8f32(a, s, rows, s),
                 lambda: rtm.gemm_f8w8f32_experts(a, s, stack, s, s),
                 lambda: rtm.gemm_f8w8tf32_experts(a, s, stack, s, s),
                 lambda: rtm.gemm_f8tf8f32_experts(rows, s, a, s, s),
                 lambda: rtm.gemm_f8_dequantize(rows, s), lambda: rtm.gemm_f8_dequantize(stack, s, "tiles"),
                 lambda: rtm.gemm_f8w8f32_selftest_timeout(rows, s, w, s, s, 10 ** 8)):
        with pytest.raises(ValueError, match="neighbours"):
            call()


def test_views_that_hold_their_rows_are_taken():
    whole = codes(40, 256)
    for t, ld in ((whole, 256), (whole[:, 16:80], 256), (whole[::2, :100], 512), (whole[3:4], 256),
                  (codes(1, 20), 32), (codes(1, 1), 16), (codes(7, 32)[:, :20], 32),
                  (codes(7, 16)[:, :1], 16),
                  (codes(2, 9, 48), 48), (codes(2, 9, 48)[:, :, :40], 48),
                  (codes(1, 9, 48), 48), (codes(5, 1, 48), 48), (codes(5, 1, 64)[:, :, :33], 64),
                  (codes(1, 1, 33), 48), (whole.as_strided((1, 9, 48), (0, 256, 1)), 256),
                  (whole.as_strided((1, 48), (0, 1)), 48), (codes(0, 20), 32), (codes(5, 0), 0)):
        got = f8._codes("codes", t, t.dim(), 0)
        # a single row's pitch is not told by its stride
        assert got >= t.shape[-1] and got % 16 == 0 and (t.numel() == 0 or t.shape[-2] == 1 or got == ld)


@pytest.mark.parametrize("fan", [1.0, True, 0, -1, (1 << 20) + 1, "1", None])
def test_a_fan_that_is_no_whole_number_is_refused(fan):
    x, rows = (t.as_subclass(OnDevice) for t in (torch.ones(4, 16), torch.zeros(4, dtype=torch.int32)))
    with pytest.raises(ValueError, match="fan must be a whole number"):
        rtm.gemm_f8_quantize(x, gather=rows, fan=fan)


def test_rows_of_the_order_are_as_many_as_the_library_writes():
    """gemm_route makes `rows` by a formula of its own, and the C entry cannot see its length."""
    rtm.build()
    for T in (0, 1, 2, 31, 33, 1000, 70000, (2 ** 31 - 1 - 256 - 1024 * 1024) // 32):
        for E in (1, 2, 7, 64, 1000, 1024):
            for k in (1, 2, 8, 32):
                for align in (1, 2, 127, 128, 1024):
                    if k <= E:
                        assert f8._route_rows(T, E, k, align) == rtm.gemm_route_rows(T, E, k, align)
