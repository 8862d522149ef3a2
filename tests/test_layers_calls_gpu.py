"""Calls of the operators around a layer's products that the documentation allows
beside the plain ones: broadcast inputs, the same matrix twice, chains of calls on
one stream, captured graphs with workspaces of their own, several streams at once,
calls without the fast-call module; and refusals that need a device.  Bounds as in
test_layers_gpu."""

import math

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import HALF, TINY, U, Rope, Shared, check_fp8, clean_status, fp8_operand, gen, torch  # noqa: F401
from tests.test_serving_gpu import assert_within, status_is

pytestmark = pytest.mark.gpu


def status(f, *args, **kw):
    try:
        f(*args, **kw)
    except sg.SbgemmError as e:
        return e.status
    return sg.SBGEMM_OK


def test_broadcast_inputs(torch):
    """One latent row as every head's keys, and the gradient of a sum over heads:
    inputs whose strides are 0."""
    tokens, heads = 19, 6
    r = Rope(torch, "bf16", tokens, 64, False, [(1, 64, 64, 0)])
    wide = Rope(torch, "bf16", tokens, 64, False, [(heads, 64, 64, 0)])
    wide.positions, wide.w = r.positions, r.w
    wide.x = [r.x[0].expand(tokens, heads, 64)]
    wide.dy = [r.dy[0].expand(tokens, heads, 64)]
    wide.check()
    one = wide.dy[0][:1, :1].expand(tokens, heads, 64)          # a gradient of one row for all
    wide.dy = [one]
    wide.check()


def test_a_matrix_by_itself(torch):
    g = gen(torch, 3)
    A, S, v = fp8_operand(torch, g, 1, 200, 384, "k", "e4m3", 1)
    v = v.nan_to_num(0.0)
    A = A.float().nan_to_num(0.0).to(A.dtype)
    C = torch.full((1, 200, 200), math.nan, device="cuda")
    sg.matmul_fp8(A, S, A.transpose(1, 2), S.transpose(1, 2), C, alpha=1e-6)
    ref, size = 1e-6 * v @ v.transpose(1, 2), 1e-6 * v.abs() @ v.abs().transpose(1, 2)
    assert_within(torch, C, ref, (384 + 3 + 8) * U * size + HALF["fp32"] * ref.abs() + TINY)


def test_fp8_shared_operand_of_a_large_batch(torch):
    """More batches than a cluster or a wave has, one weight for all."""
    g = gen(torch, 4)
    A, SA, va = fp8_operand(torch, g, 700, 3, 160, "k", "e5m2", 1)
    B, SB, vb = fp8_operand(torch, g, 1, 40, 160, "k", "e4m3", 128)
    A, B = (x.float().nan_to_num(0.0).clamp(-400, 400).to(x.dtype) for x in (A, B))
    rows = lambda s, n, group: s.double().repeat_interleave(group, 1)[:, :n].repeat_interleave(128, 2)[..., :160]
    va, vb = A.double() * rows(SA, 3, 1), B.double() * rows(SB, 40, 128)
    C = torch.full((700, 3, 40), math.nan, device="cuda")
    sg.matmul_fp8(A, SA, B.transpose(1, 2), SB.transpose(1, 2), C, alpha=1e-5)
    ref, size = 1e-5 * va @ vb.transpose(1, 2), 1e-5 * va.abs() @ vb.abs().transpose(1, 2)
    assert_within(torch, C, ref, (160 + 2 + 8) * U * size + HALF["fp32"] * ref.abs() + TINY)


def chain(torch, steps, apart, x, W, WS):
    """Layers one behind the other: each norms its input, quantises it, multiplies
    it and attends over a cache with the result; every buffer is used again by
    the next one."""
    tokens, n = x.shape
    h, q = x.clone(), torch.empty(tokens, n, device="cuda", dtype=torch.float8_e4m3fn)
    s = torch.empty(tokens, n // 128, device="cuda")
    attend = Shared(torch, "bf16", [(300, *range(1, tokens))], 8, 1, 128, 0, 16, seed=2)
    wait = torch.cuda.synchronize if apart else (lambda: None)
    for _ in range(steps):
        sg.norm_rope([sg.RopePart(h, h, norm=n)], None, None)
        wait()
        sg.quantize_fp8(h, q, s)
        wait()
        sg.matmul_fp8(q, s, W.t(), WS.t(), h)
        wait()
        attend.o = h.view(tokens, 1, 8, 128)[:len(attend.lens)]
        attend.q = attend.o.clone()
        attend.run()
        wait()
    torch.cuda.synchronize()
    return h


@pytest.mark.parametrize("tokens", [5, 40, 300])
def test_chains_of_calls_equal_calls_one_at_a_time(torch, tokens):
    """The kernels start while those before them still run: results are those of
    calls that wait for one another, also when a graph replays them."""
    n, g = 1024, gen(torch, 5)
    x = torch.randn(tokens, n, generator=g, device="cuda").bfloat16()
    w = torch.randn(n, n, generator=g, device="cuda").bfloat16()
    W, WS = torch.empty(n, n, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(n // 128, n // 128, device="cuda")
    sg.quantize_fp8(w, W, WS)
    want = chain(torch, 6, True, x, W, WS)
    assert bool(want.isfinite().all())
    for _ in range(4):
        assert torch.equal(chain(torch, 6, False, x, W, WS), want)
    status_is(0)


def test_graphs_with_workspaces_of_their_own_replay_at_once(torch):
    shared = [Shared(torch, "fp16", [(500 + 40 * i, 3, 90, 1)], 16, 1, 512, 64, 16, seed=i) for i in range(2)]
    ropes = [Rope(torch, "bf16", 300, 64, False, [(16, 128, 128, 0), (2, 128, 128, 0)], seed=i) for i in range(2)]
    graphs, outs = [], []
    for c, r in zip(shared, ropes):
        dx = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in r.x]
        dw = [torch.empty(128, device="cuda") for _ in r.x]
        ws = torch.empty(sg.sbgemm_norm_rope_workspace_bytes([128, 128]), device="cuda", dtype=torch.uint8)
        parts = [sg.RopeGrad(x, dy, o, norm=128, weight=w, dweight=d) for x, dy, o, w, d in zip(r.x, r.dy, dx, r.w, dw)]
        c.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run()
            sg.norm_rope_backward(parts, r.positions, r.table, workspace=ws)
        c.o.fill_(math.nan)
        graphs.append(graph)
        outs.append((dx, dw))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for c, r, (dx, dw) in zip(shared, ropes, outs):
        c.check(torch)
        for i in range(2):
            rx, lx, rw, lw = r.gradient(i)
            assert_within(torch, dx[i], rx, lx)
            assert_within(torch, dw[i], rw, lw)


def test_products_on_two_streams_at_once(torch):
    """Kernels that hold tensor memory beside one another."""
    g = gen(torch, 6)
    W, WS, vw = fp8_operand(torch, g, 1, 2048, 1024, "k", "e4m3", 128)
    W = W.float().nan_to_num(0.0).to(W.dtype)
    cases, want = [], []
    for M in (16, 50, 200, 1000):
        A, S, _ = fp8_operand(torch, g, 1, M, 1024, "k", "e4m3", 1)
        A = A.float().nan_to_num(0.0).to(A.dtype)
        C = torch.empty(1, M, 2048, device="cuda", dtype=torch.bfloat16)
        sg.matmul_fp8(A, S, W.transpose(1, 2), WS.transpose(1, 2), C, alpha=1e-4)
        cases.append((A, S, C))
        want.append(C.clone())
    att = Shared(torch, "bf16", [(2000, *range(1, 30))], 16, 1, 512, 64, 64)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (A, S, C) in enumerate(cases):
            with torch.cuda.stream(streams[i % 2]):
                sg.matmul_fp8(A, S, W.transpose(1, 2), WS.transpose(1, 2), C, alpha=1e-4)
        with torch.cuda.stream(streams[2]):
            att.run()
    torch.cuda.synchronize()
    for (_, _, C), w in zip(cases, want):
        assert torch.equal(C, w)
    att.check(torch)
    status_is(0)


def test_calls_without_the_fast_call_module(torch, monkeypatch):
    monkeypatch.setattr(sg, "_fast", None)
    r = Rope(torch, "fp32", 9, 64, True, [(4, 128, 128, 0), (1, 96, 64, 32)])
    r.check()
    c = Shared(torch, "bf16", [(64, 30, 0, 100, 7)], 16, 1, 512, 64, 64)
    c.run()
    c.check(torch)
    x = torch.randn(30, 300, generator=gen(torch, 7), device="cuda").bfloat16()
    out = []
    for fast in (False, True):
        if fast:
            monkeypatch.undo()
        y, s = torch.empty(30, 300, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(30, 3, device="cuda")
        C = torch.empty(30, 30, device="cuda")
        sg.quantize_fp8(x, y, s)
        sg.matmul_fp8(y, s, y.t(), s.t(), C)
        out.append((y.float(), s, C))
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_refusals_on_a_device(torch):
    r = Rope(torch, "bf16", 9, 64, False, [(2, 64, 64, 0)])
    dx, dw = torch.empty_like(r.x[0], memory_format=torch.contiguous_format), torch.empty(64, device="cuda")
    part = sg.RopeGrad(r.x[0], r.dy[0], dx, norm=64, weight=r.w[0], dweight=dw)
    need = sg.sbgemm_norm_rope_workspace_bytes([64])
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    for w in (None, ws[:need - 256]):
        assert status(sg.norm_rope_backward, [part], r.positions, r.table, workspace=w) == sg.SBGEMM_ERR_INVALID_VALUE
    sg.norm_rope_backward([part], r.positions, r.table, workspace=ws)
    with pytest.raises(TypeError):
        sg.norm_rope([sg.RopePart(r.x[0], dx)], None, r.table)
    with pytest.raises(ValueError):
        sg.norm_rope([sg.RopePart(r.x[0], dx)], r.positions[:8], r.table)
    with pytest.raises(TypeError):
        sg.norm_rope([sg.RopePart(r.x[0], dx.float())], r.positions, r.table)
    with pytest.raises(TypeError):
        sg.norm_rope_backward([sg.RopeGrad(None, r.dy[0], dx, norm=64)], r.positions, r.table)
    c = Shared(torch, "bf16", [(64, 30, 7)], 16, 1, 512, 64, 64)
    whole = c.workspace
    for w in (None, whole[:whole.numel() - 256]):
        c.workspace = w
        assert status(c.run) == sg.SBGEMM_ERR_INVALID_VALUE
    c.workspace = whole
    c.run()
    c.check(torch)
    x, y = torch.zeros(8, 256, device="cuda").bfloat16(), torch.empty(8, 256, device="cuda", dtype=torch.float8_e4m3fn)
    for scale in (torch.empty(8, 1, device="cuda"), torch.empty(3, 2, device="cuda")):
        with pytest.raises(ValueError):
            sg.quantize_fp8(x, y, scale)
    with pytest.raises(TypeError):
        sg.quantize_fp8(x, x, torch.empty(8, 2, device="cuda"))
    host = torch.zeros(8, 256).bfloat16()
    with pytest.raises(TypeError):
        sg.quantize_fp8(host, y, torch.empty(8, 2, device="cuda"))


@pytest.mark.parametrize("tc", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("lc", ["c", "t", "o"])
@pytest.mark.parametrize("size", [(1, 700, 1000, 640), (3, 260, 264, 256), (1, 16, 2048, 2000), (1, 2600, 1032, 384), (2, 4, 6, 300)])
def test_fp8_added_to_c(torch, tc, lc, size):
    """Tiles of every shape added to C, whose rows are vectors, in either order, or not."""
    check_fp8(torch, *size, lc=lc, tc=tc, alpha=1.5, accumulate=True)


@pytest.mark.parametrize("tc", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("size", [(1, 700, 1000, 640), (2, 2600, 1033, 384), (1, 130, 4099, 128)])
def test_fp8_rows_of_c_that_are_not_vectors(torch, tc, size):
    check_fp8(torch, *size, lc="o", tc=tc, alpha=1.5)
    check_fp8(torch, *size, lc="c", tc=tc, accumulate=True)
    check_fp8(torch, *size, lc="t", tc=tc)
