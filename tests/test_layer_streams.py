"""The layer operators on two streams at once, captured, and with tensors of an
earlier stream: the library keeps nothing between calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import blockwise_fp8_gemm_bfp8_amd as bfp8  # noqa: E402

BF = torch.bfloat16


def work(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *s: torch.randn(s, device="cuda", generator=gen).to(BF)
    x, residual, dy, gate, up = (new(1024, 1024) for _ in range(5))
    w = torch.rand(1024, device="cuda", generator=gen) + 0.5
    grads = [new(n) for n in (5, 100000, 1 << 20)]
    plan = bfp8.GradClip(grads, [torch.empty_like(g) for g in grads])

    def run():
        y, r, rstd = bfp8.rmsnorm(x, w, residual)
        out = [y, r, rstd, *bfp8.rmsnorm_quantize(x, w, residual, transposed=True),
               *bfp8.rmsnorm_backward(dy, r, w, rstd, residual), bfp8.swiglu(gate, up),
               *bfp8.swiglu_quantize(gate, up), *bfp8.swiglu_backward(dy, gate, up),
               *bfp8.swiglu_backward_quantize(dy, gate, up, scales="mx32", transposed=True)]
        norm = plan.clip(1.0)
        return out + [norm, *plan.out]
    return run


def test_two_streams_at_once():
    runs = [work(1), work(2)]
    want = [[t.clone() for t in run()] for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for run, stream in zip(runs, streams):
            with torch.cuda.stream(stream):
                got.append(run())
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_of_one_plan():
    """Workspaces are a call's own: two graphs captured from the same program and
    replayed one after the other, with eager calls between, share none."""
    run = work(3)
    want = [t.clone() for t in run()]
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for _ in range(2):
        for graph, out in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, want))
            assert all(torch.equal(x, y) for x, y in zip(run(), want))


def test_refusals_of_the_binding():
    x = torch.randn((128, 256), device="cuda").to(BF)
    w = torch.ones(256, device="cuda")
    for call in (lambda: bfp8.rmsnorm(x, w[:128]), lambda: bfp8.rmsnorm(x, w.double()),
                 lambda: bfp8.rmsnorm(x, w, x.float()), lambda: bfp8.rmsnorm(x, w, x[:64]),
                 lambda: bfp8.rmsnorm(x, w, sum_out=x), lambda: bfp8.rmsnorm(x.half(), w),
                 lambda: bfp8.rmsnorm(x.t(), w[:128]), lambda: bfp8.rmsnorm(x[0], w),
                 lambda: bfp8.rmsnorm(x, w, out=x.float()),
                 lambda: bfp8.rmsnorm_quantize(x, w, scales="fp8"),
                 lambda: bfp8.rmsnorm_quantize(x, w, qt=x),
                 lambda: bfp8.rmsnorm_quantize(x, w, s=torch.empty((128, 2), device="cuda")),
                 lambda: bfp8.rmsnorm_backward(x, x, w, torch.ones(64, device="cuda")),
                 lambda: bfp8.swiglu(x, x[:, :128]), lambda: bfp8.swiglu(x, x.float()),
                 lambda: bfp8.GradClip([x.half()]), lambda: bfp8.GradClip([x.t()]),
                 lambda: bfp8.GradClip([x], [x.float()]), lambda: bfp8.GradClip([x, w, x]),
                 lambda: bfp8.GradClip([x, x.clone()], [x.clone(), x]), lambda: bfp8.GradClip([x], []),
                 lambda: bfp8.GradClip([x]).clip(1.0, norm=torch.ones(1)),
                 lambda: bfp8.GradClip([x]).norm(out=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bfp8.rmsnorm(x, w, eps=0.0), lambda: bfp8.swiglu(x[:, 1:], x[:, 1:]),
                 lambda: bfp8.rmsnorm_quantize(x[:, :200], w[:200]),
                 lambda: bfp8.rmsnorm_quantize(x[:100], w, transposed=True),
                 lambda: bfp8.rmsnorm_backward(x, x, w, torch.ones(128, device="cuda"), workspace=w),
                 lambda: bfp8.clip_grads([x], float("nan")), lambda: bfp8.clip_grads([x], -1.0)):
        with pytest.raises(bfp8.BFP8Error):
            call()
