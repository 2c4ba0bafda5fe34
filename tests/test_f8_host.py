"""CPU tests of the 8-bit floating-point, routing and joining entry points: what they refuse on
the host before any CUDA call, sizes of rows and workspaces, and arguments that are no tensors."""

import numpy as np
import pytest
import torch

import register_tiled_matrix_gb300 as rtm

pytestmark = pytest.mark.cpu
A, B, C, D, E, F = (0x10000000 * i for i in range(1, 7))
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    rtm.build()
    return rtm.load_library()


def test_pitch(lib):
    assert [lib.gemm_f8_pitch(k) for k in (0, 1, 16, 17, 8190)] == [0, 16, 16, 32, 8192]
    assert lib.gemm_f8_pitch(-1) == -1 and lib.gemm_f8_pitch(1 << 31) == -1


def test_route_rows(lib):
    f = lib.gemm_route_rows
    assert f(0, 8, 2, 128) == 0
    assert f(1, 8, 2, 1) == 2 and f(1, 8, 2, 128) == 2 + 2 * 127
    assert f(100, 8, 2, 128) == 200 + 8 * 127
    for bad in ((-1, 8, 2, 1), (1, 0, 1, 1), (1, 1025, 1, 1), (1, 8, 0, 1), (1, 8, 9, 1),
                (1, 64, 33, 1), (1, 8, 2, 0), (1, 8, 2, 1025), (1 << 30, 8, 4, 1)):
        assert f(*bad) == -1, bad
    assert lib.gemm_route_workspace_bytes(1, 64) == 0
    assert lib.gemm_route_workspace_bytes(1 << 20, 64) > 0
    assert lib.gemm_route_workspace_bytes(4, 0) == -1


@pytest.mark.parametrize("name", ["gemm_f8w8f32", "gemm_f8w8tf32", "gemm_f8tf8f32"])
def test_products(lib, name):
    f = getattr(lib, name)

    def call(M=64, N=64, K=64, a=A, lda=64, s=B, b=C, ldb=64, t=D, c=E):
        return f(M, N, K, a, lda, s, b, ldb, t, c, None)

    assert call(M=0, K=0) == 0 if name == "gemm_f8tf8f32" else call(M=0) == 0
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(lda=40), dict(lda=48),
                dict(ldb=0), dict(ldb=56), dict(a=None), dict(s=None), dict(b=None), dict(t=None),
                dict(c=None), dict(c=A), dict(c=A + 64 * 64 - 4), dict(c=C + 16), dict(c=B + 4)):
        assert call(**bad) == -1, bad
    for bad in (dict(a=A + 8), dict(b=C + 1), dict(s=B + 2), dict(t=D + 1), dict(c=E + 2)):
        assert call(**bad) == -2, bad


@pytest.mark.parametrize("name", ["gemm_f8w8f32_experts", "gemm_f8w8tf32_experts",
                                  "gemm_f8tf8f32_experts"])
def test_experts_products(lib, name):
    f = getattr(lib, name)

    def call(R=64, N=64, K=64, n=4, o=F, a=A, lda=64, s=B, b=C, ldb=64, t=D, c=E):
        return f(R, N, K, n, o, a, lda, s, b, ldb, t, c, None)

    assert call(n=0) == 0
    for bad in (dict(n=-1), dict(n=1025), dict(R=-1), dict(o=None), dict(lda=63), dict(c=F),
                dict(c=None)):
        assert call(**bad) == -1, bad
    assert call(o=F + 2) == -2


def test_quantize(lib):
    f = lib.gemm_bf16_f8_quantize

    def call(M=64, K=64, x=A, source=64, rows=None, fan=1, fac=None, rc=B, rs=C, cc=D, cs=E):
        return f(M, K, x, source, rows, fan, fac, rc, rs, cc, cs, None)

    assert call(M=0, source=0) == 0 and call(K=0) == 0
    for bad in (dict(M=-1), dict(K=-1), dict(source=63), dict(fan=2), dict(fac=F), dict(fan=0),
                dict(rows=F, fan=1 << 26), dict(x=None), dict(rc=None), dict(rs=None),
                dict(cc=None), dict(rc=None, rs=None, cc=None, cs=None), dict(rc=A), dict(cc=B),
                dict(rows=F, rc=F), dict(rows=F, fac=F + MB, cs=F + MB)):
        assert call(**bad) == -1, bad
    for bad in (dict(x=A + 1), dict(rc=B + 8), dict(rs=C + 2), dict(cc=D + 4), dict(cs=E + 1),
                dict(rows=F + 2)):
        assert call(**bad) == -2, bad
    g = lib.gemm_f32_f8_quantize_tiles
    assert g(0, 64, 64, None, None, None, None) == 0
    assert g(-1, 64, 64, A, B, C, None) == -1 and g(1, 64, 64, A, A + 4, C, None) == -1
    assert g(1, 64, 64, A + 2, B, C, None) == -2 and g(1, 64, 64, A, None, C, None) == -1


def test_dequantize(lib):
    f = lib.gemm_f16_f8_dequantize

    def call(n=2, M=64, K=60, kind=2, q=A, ld=64, s=B, x=C):
        return f(n, M, K, kind, q, ld, s, x, None)

    assert call(n=0) == 0 and call(M=0) == 0 and call(K=0) == 0
    for bad in (dict(kind=3), dict(kind=-1), dict(ld=60), dict(ld=48), dict(n=-1), dict(q=None),
                dict(s=None), dict(x=None), dict(x=A), dict(x=B)):
        assert call(**bad) == -1, bad
    assert call(q=A + 4) == -2 and call(s=B + 2) == -2 and call(x=C + 1) == -2


def test_route(lib):
    f = lib.gemm_f32_route

    def call(T=200, n=64, k=4, z=A, bias=None, groups=1, top=1, align=1, e=B, w=C, s=D, r=E, o=F,
             ws=F + MB, wb=MB):
        return f(T, n, k, z, bias, groups, top, 0, 1, 1.0, align, e, w, s, r, o, ws, wb, None)

    for bad in (dict(T=-1), dict(n=0), dict(n=1025), dict(k=0), dict(k=33), dict(n=3, k=4),
                dict(groups=0), dict(groups=33, n=66), dict(groups=3), dict(groups=2, top=3),
                dict(groups=32, top=1), dict(top=0), dict(align=0), dict(align=1025), dict(z=None),
                dict(e=None), dict(w=None), dict(s=None), dict(r=None), dict(o=None), dict(wb=0),
                dict(wb=-1), dict(ws=None), dict(e=A), dict(w=B), dict(o=E), dict(ws=D),
                dict(bias=C)):
        assert call(**bad) == -1, bad
    for bad in (dict(z=A + 2), dict(e=B + 1), dict(w=C + 2), dict(s=D + 2), dict(r=E + 2),
                dict(o=F + 1), dict(bias=F + 2 * MB + 1)):
        assert call(**bad) == -2, bad
    g = lib.gemm_f32_route_backward
    assert g(0, 8, 2, None, 0, 1, 1.0, None, None, None, None) == 0
    assert g(4, 8, 9, A, 0, 1, 1.0, B, C, D, None) == -1
    assert g(4, 8, 2, A, 0, 1, 1.0, B, C, A, None) == -1
    assert g(4, 8, 2, A, 0, 1, 1.0, B, C + 2, D, None) == -2


def test_join(lib):
    f = lib.gemm_experts_join
    assert f(0, 8, 2, 16, None, None, None, None, None) == 0
    for bad in ((4, 8, 0, 16, A, B, C, D), (4, 8, 33, 16, A, B, C, D), (-4, 8, 2, 16, A, B, C, D),
                (4, 8, 2, -16, A, B, C, D), (4, 8, 2, 16, None, B, C, D), (4, 8, 2, 16, A, None, C, D),
                (4, 8, 2, 16, A, B, C, None), (4, 8, 2, 16, A, B, C, A)):
        assert f(*bad, None) == -1, bad
    assert f(4, 8, 2, 16, A, B + 2, C, D, None) == -2
    g = lib.gemm_bf16_experts_join_backward
    assert g(0, 8, 2, 16, None, None, None, None, None) == 0
    assert g(4, 8, 2, 16, A, B, C, B, None) == -1 and g(4, 8, 2, 16, A + 1, B, C, D, None) == -2
    assert g(4, 8, 2, 16, A, None, C, D, None) == -1


def test_selftest(lib):
    f = lib.gemm_f8w8f32_selftest_timeout
    fine = (64, 64, 64, A, 64, B, C, 64, D, E)
    assert f(*fine, 10, None) == -1 and f(*fine, 10 ** 11, None) == -1
    assert f(64, 64, 0, *fine[3:], 10 ** 8, None) == -1


@pytest.mark.parametrize("bad", [None, 3, [[1.0]], np.ones((1, 64), dtype=np.float32),
                                 torch.zeros(4, 4)], ids=lambda v: type(v).__name__)
def test_no_cuda_tensors(bad):
    for call in (lambda: rtm.gemm_f8_quantize(bad), lambda: rtm.gemm_f8_quantize_tiles(bad),
                 lambda: rtm.gemm_f8_dequantize(bad, bad), lambda: rtm.gemm_f8w8f32(bad, bad, bad, bad),
                 lambda: rtm.gemm_f8w8tf32(bad, bad, bad, bad),
                 lambda: rtm.gemm_f8tf8f32(bad, bad, bad, bad),
                 lambda: rtm.gemm_f8w8f32_experts(bad, bad, bad, bad, bad),
                 lambda: rtm.gemm_f8tf8f32_experts(bad, bad, bad, bad, bad),
                 lambda: rtm.gemm_route(bad, 2), lambda: rtm.gemm_route_backward(bad, bad, bad),
                 lambda: rtm.gemm_experts_join(bad, bad),
                 lambda: rtm.gemm_experts_join_backward(bad, bad, bad)):
        with pytest.raises(ValueError):
            call()
