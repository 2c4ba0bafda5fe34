"""Several host threads make their first calls of the 8-bit floating-point, routing and joining
entry points into a freshly loaded library at once, each on its own stream: kernel attributes and
cluster occupancies are filled on first use, and results are those of calls made one by one. Runs
in a child process so that the library's first use really happens inside the threads."""

import os
import subprocess
import sys
import textwrap

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent(r"""
    import sys, threading
    sys.path.insert(0, sys.argv[1])
    import torch
    import register_tiled_matrix_gb300 as rtm
    from tests import f8_reference as ref

    torch.cuda.init()
    gen = torch.Generator("cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def layer(x, w, dy, stream):
        # a product and its gradients, as a training step makes them
        a, s, ac, sc = rtm.gemm_f8_quantize(x, "both", stream=stream)
        q, t = rtm.gemm_f8_quantize_tiles(w, stream=stream)
        d, u, dc, uc = rtm.gemm_f8_quantize(dy, "both", stream=stream)
        return (rtm.gemm_f8w8f32(a, s, q, t, stream=stream),
                rtm.gemm_f8w8tf32(d, u, q, t, stream=stream),
                rtm.gemm_f8tf8f32(ac, sc, dc, uc, stream=stream),
                rtm.gemm_f8_dequantize(a, s, "rows", torch.float32, stream=stream))

    def experts(x, logits, w, dy, k, align, stream):
        chosen, weights, slots, rows, offsets = rtm.gemm_route(logits, k, align=align, stream=stream)
        a, s = rtm.gemm_f8_quantize(x, gather=rows, fan=k, stream=stream)
        q, t = rtm.gemm_f8_quantize_tiles(w, stream=stream)
        out = torch.zeros(len(rows), w.shape[2], device="cuda")
        c = rtm.gemm_f8w8f32_experts(a, s, q, t, offsets, out=out, stream=stream)
        dw = rtm.gemm_experts_join_backward(dy, c, slots, stream=stream)
        return (weights, slots, rows, offsets, c, dw,
                rtm.gemm_experts_join(c, slots, weights, stream=stream),
                rtm.gemm_route_backward(logits, chosen, dw, stream=stream))

    jobs = [(layer, (normal(M, K).to(dt), normal(K, N), normal(M, N).to(dt)))
            for M, N, K, dt in ((1, 300, 700, torch.bfloat16), (20, 500, 1030, torch.float16),
                                (60, 1000, 400, torch.float32), (100, 260, 2100, torch.bfloat16),
                                (300, 520, 260, torch.float16), (2100, 2000, 1040, torch.bfloat16))]
    jobs += [(experts, (normal(T, K).bfloat16(), normal(T, E), normal(E, K, N), normal(T, N), k, align))
             for T, K, N, E, k, align in ((1, 200, 300, 8, 2, 1), (30, 130, 256, 64, 6, 1),
                                          (400, 256, 200, 8, 2, 128), (3000, 256, 512, 16, 4, 128))]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    results, errors, barrier = [None] * len(jobs), [], threading.Barrier(len(jobs))

    def work(i):
        try:
            f, args = jobs[i]
            barrier.wait()
            with torch.cuda.stream(streams[i]):
                for _ in range(3):
                    results[i] = f(*args, streams[i])
            streams[i].synchronize()
        except Exception as e:  # reported by the parent
            errors.append(f"thread {i}: {e!r}")

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        print("\n".join(errors)); sys.exit(2)
    if rtm.get_device_error() != 0:
        print("device error word set"); sys.exit(3)
    for i, (f, args) in enumerate(jobs):
        for j, (a, b) in enumerate(zip(results[i], f(*args, None))):
            if not torch.equal(a, b):
                print(f"job {i}: result {j} differs from that of a call by itself"); sys.exit(4)
    x, w, dy = jobs[5][1]
    a = ref.values(*rtm.gemm_f8_quantize(x), "rows")
    b = ref.values(*rtm.gemm_f8_quantize_tiles(w), "tiles")
    ref.close(results[5][0], a @ b, a.abs() @ b.abs(), 9)
    print("ok")
""")


def test_first_calls_from_many_threads():
    import register_tiled_matrix_gb300 as rtm
    rtm.build()  # build in this process; the child only loads the library
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.strip().endswith("ok")
