"""The 8-bit floating-point products, routing and the experts' layer captured into graphs,
replayed on new inputs, and run on two streams at once; and their bounded waits running out."""

import time

import pytest
import torch

import register_tiled_matrix_gb300 as rtm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    rtm.build()
    yield
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0


def make(T, E, k, K, N, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    wq, ws = rtm.gemm_f8_quantize_tiles(torch.randn(E, K, N, generator=g, device=DEV) * 0.1)
    return dict(x=torch.randn(T, K, generator=g, device=DEV).bfloat16(), k=k, wq=wq, ws=ws,
                z=torch.randn(T, E, generator=g, device=DEV),
                dy=torch.randn(T, N, generator=g, device=DEV).bfloat16())


def step(d):
    """A forward and backward pass of a layer of experts and of one shared weight."""
    k = d["k"]
    experts, weights, slots, rows, offsets = rtm.gemm_route(d["z"], k)
    a, s, ac, sc = rtm.gemm_f8_quantize(d["x"], "both", gather=rows, fan=k)
    c = rtm.gemm_f8w8f32_experts(a, s, d["wq"], d["ws"], offsets)
    y = rtm.gemm_experts_join(c, slots, weights)
    q, t, qc, tc = rtm.gemm_f8_quantize(d["dy"], "both", gather=rows, fan=k, factors=weights)
    dx = rtm.gemm_experts_join(rtm.gemm_f8w8tf32_experts(q, t, d["wq"], d["ws"], offsets), slots)
    dw = rtm.gemm_f8tf8f32_experts(ac, sc, qc, tc, offsets)
    dweights = rtm.gemm_experts_join_backward(d["dy"], c, slots)
    dz = rtm.gemm_route_backward(d["z"], experts, dweights)
    xq, xs = rtm.gemm_f8_quantize(d["x"], "rows")
    shared = rtm.gemm_f8w8f32(xq, xs, d["wq"][0], d["ws"][0])
    return [experts, weights, slots, y, dx, dw, dweights, dz, shared]


SIZES = [(3, 8, 2, 300, 200), (60, 32, 4, 256, 260), (700, 8, 2, 520, 300)]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_captured_and_replayed(sizes):
    d, other = make(*sizes, seed=1), make(*sizes, seed=2)
    wants = [[t.clone() for t in step(v)] for v in (d, other)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(d)
    for v, want in ((d, wants[0]), (other, wants[1])):
        for n in ("x", "z", "dy", "wq", "ws"):
            if v is not d:
                d[n].view(torch.uint8).copy_(v[n].view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_graphs_at_once():
    d, other = make(*SIZES[2], seed=1), make(*SIZES[2], seed=2)
    wants = [[t.clone() for t in step(v)] for v in (d, other)]
    torch.cuda.synchronize()
    graphs, gots = [], []
    for v in (d, other):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            gots.append(step(v))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(gots, wants):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    work = [make(*s, seed=i) for i, s in enumerate(SIZES)]
    wants = [[t.clone() for t in step(v)] for v in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    gots = [None] * len(work)
    for _ in range(4):
        for i, (v, s) in enumerate(zip(work, streams)):
            with torch.cuda.stream(s):
                gots[i] = step(v)
    torch.cuda.synchronize()
    for got, want in zip(gots, wants):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K", [(1, 1024, 1024), (40, 300, 500), (128, 256, 700),
                                   (300, 300, 600), (2000, 2000, 300)])
def test_waits_run_out(M, N, K):
    """With the loads muted every role gives up in time, the error is recorded, and the next
    product is right."""
    a, s = rtm.gemm_f8_quantize(torch.ones(M, K, device=DEV))
    w, t = rtm.gemm_f8_quantize_tiles(torch.ones(K, N, device=DEV))
    torch.cuda.synchronize()
    out = torch.empty(M, N, device=DEV)
    begin = time.monotonic()
    rtm.gemm_f8w8f32_selftest_timeout(a, s, w, t, out, 20_000_000)
    assert rtm.status_string(rtm.get_device_error()).startswith("GEMM_ERR_TIMEOUT")
    assert time.monotonic() - begin < 10
    assert (rtm.gemm_f8w8f32(a, s, w, t) == K).all()
    torch.cuda.synchronize()
    assert rtm.get_device_error() == 0
