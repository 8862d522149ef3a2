"""Quantisation and product one behind the other on one stream, with nothing
between them that waits: buffers of 8-bit values and scales that the next pair of
calls writes again."""

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import clean_status, gen, torch  # noqa: F401
from tests.test_serving_gpu import status_is

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [1, 128])
@pytest.mark.parametrize("rows", [1, 5, 16, 40, 130, 300])
def test_scales_written_while_the_next_product_starts(torch, rows, group):
    """Every pair's product reads the values and scales of its own quantisation:
    bit for bit those of calls that wait for one another.  The steps' inputs differ
    in size by powers of two, so that a scale of another step shows."""
    K, N, steps = 1024, 2048, 24
    g = gen(torch, rows + group)
    f8 = dict(device="cuda", dtype=torch.float8_e4m3fn)
    w = (torch.randn(N, K, generator=g, device="cuda") / 32).bfloat16()
    W, WS = torch.empty(N, K, **f8), torch.empty(N // group, K // 128, device="cuda")
    sg.quantize_fp8(w, W, WS)
    x = [(torch.randn(rows, K, generator=g, device="cuda") * 2.0 ** (i % 7 - 3)).bfloat16() for i in range(steps)]
    X, XS = torch.empty(rows, K, **f8), torch.empty(rows, K // 128, device="cuda")
    out = {}
    for apart in (True, False, False, False):
        y = [torch.empty(rows, N, device="cuda", dtype=torch.bfloat16) for _ in x]
        torch.cuda.synchronize()
        for a, b in zip(x, y):
            sg.quantize_fp8(a, X, XS)
            if apart:
                torch.cuda.synchronize()
            sg.matmul_fp8(X, XS, W.t(), WS.t(), b)
            if apart:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        if apart:
            out = y
        else:
            for i, (a, b) in enumerate(zip(y, out)):
                assert torch.equal(a, b), f"step {i}"
    status_is(0)
    # The same from a graph, whose launches follow one another without the host.
    y = [torch.empty(rows, N, device="cuda", dtype=torch.bfloat16) for _ in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a, b in zip(x, y):
            sg.quantize_fp8(a, X, XS)
            sg.matmul_fp8(X, XS, W.t(), WS.t(), b)
    for _ in range(3):
        for b in y:
            b.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(y, out))
    status_is(0)
