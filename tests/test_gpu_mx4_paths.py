"""The kernels of the products on 4-bit weights, each call asked first which one it takes: the
weights' stream in 16 and in 32 columns a workgroup, and the tiles."""

import pytest
import torch

from test_gpu_mxfp4 import _product

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import fp8_dynamic_quant_amd as wq


@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("M, G, N, K", [
    (1, 1, 8208, 128), (16, 1, 8208, 512), (3, 1, 16304, 384), (7, 1, 9232, 1152), (1, 8, 1040, 256), (16, 8, 1040, 640),
    (15, 8, 1024, 4096), (2, 40, 208, 128), (16, 255, 64, 128), (9, 171, 48, 1280)])
def test_weights_that_stream_past_in_32_columns(M, G, N, K, a8):
    # odd numbers of 16-column slices (the last workgroup's second half is past the end), fewer steps
    # than waves, more, and no multiple of either
    assert wq.wq_mx4_path(M, N, K, G) == 2
    _product(M, G, N, K, a8, pad=16, ypad=8, tokens=4)


@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("M, G, N, K, path", [
    (16, 3, 1008, 896, 1), (17, 1, 16, 128, 3), (64, 8, 1024, 512, 3), (1000, 1, 2064, 384, 4), (70, 7, 2320, 256, 4),
    (2100, 1, 4112, 384, 5), (4000, 3, 800, 256, 5)])
def test_every_other_kernel(M, G, N, K, path, a8):
    assert wq.wq_mx4_path(M, N, K, G) == path
    _product(M, G, N, K, a8, pad=16, ypad=8, tokens=4)


@pytest.mark.parametrize("a8", [False, True])
@pytest.mark.parametrize("M, G, N, K, path", [(1, 1, 1024, 512, 1), (16, 8, 1040, 256, 2), (64, 2, 208, 384, 3), (1000, 1, 2064, 256, 4),
                                              (2100, 1, 4112, 256, 5)])
def test_graphs_with_eager_calls_between(M, G, N, K, path, a8):
    assert wq.wq_mx4_path(M, N, K, G) == path
    gen = torch.Generator(device="cuda").manual_seed(M)
    rows = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    cast = [wq.wq_group_quant_mxfp4(rows(N, 1, K)) for _ in range(G)]
    w, ws = torch.stack([c[0].view(N, K // 2) for c in cast]), torch.cat([c[2] for c in cast])
    x = rows(M, G, K)

    def call():
        a, _, s = wq.wq_group_quant_fp8_ue8m0(x, group=32) if a8 else wq.wq_group_quant_mxfp4(x)
        return wq.wq_quant_matmul(a, s, w, ws, fp8_groups=G, mx4=True)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
    for _ in range(4):
        x.copy_(rows(M, G, K))
        graph.replay()
        eager = call()
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), eager.view(torch.int16)) and torch.isfinite(y).all() and y.any()
