"""The operators around a layer's products on the GPU against plain computations
in 64 bits: products of 8-bit floats with block scales, their quantisation,
norms with rotations and their gradient, and latent attention over shared
prefixes.

Bounds, with u = 2^-23 for an fp32 operation and h = half a step of the output's
type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32, relative; 2^-25 absolute below fp16's
normals):

product   K products are summed with the blocks' two scales:
          |C - ref| <= (K + ceil(K / 128) + 8) u S + h |ref| + 2^-25,
          S = |alpha| sum |a b| (+ |C_old|)
quantise  bit for bit: both quotients are rounded to fp32 by definition
norm      a normed element is off by (n / 2 + 8) 2^-24 of itself (the sum of n
          squares, the root, two products), cosine and sine by 3 u of the
          magnitude (the angle's float by 2^-26 of a radian, the functions by an
          ulp, the product) and a rotated element has two more products and a
          sum:  |y - ref| <= (n / 2 + 8 + 16) 2^-24 m (|z_a| + |z_b|) + h |ref| + 2^-25
gradient  with G = m (|dy_a| + |dy_b|) for g and n normed elements:
          |dx - ref| <= (n + 32) u r (|w| G + |x r| mean(G |w x r|)) + h |ref| + 2^-25
          |dw - ref| <= (rows + n + 32) 2^-24 sum G |x r|
attention as in test_serving_gpu: the prefix is another split of the keys."""

import math

import pytest

import strided_gemm_gb300 as sg
from tests.test_serving_gpu import assert_within, attention_bound, attention_reference, status_is

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = 2.0 ** -25


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a CUDA device"
    sg.load()
    return t


@pytest.fixture(autouse=True)
def clean_status(torch):
    sg.sbgemm_device_status()
    yield


def dtype_of(torch, t):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn,
            "e5m2": torch.float8_e5m2}[t]


def gen(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---- quantisation --------------------------------------------------------------------

def quantise_reference(torch, x, group, t8):
    """(8-bit values, scales) of x [batch, M, K] by the definition, in 64 bits with its roundings."""
    batch, M, K = x.shape
    largest = 448.0 if t8 == "e4m3" else 57344.0
    x = x.double()
    finite = torch.isfinite(x)
    size = torch.where(finite, x.abs(), 0.0)
    size = torch.nn.functional.pad(size, (0, -K % 128, 0, -M % group))
    top = size.unflatten(2, (-1, 128)).unflatten(1, (-1, group)).amax((2, 4))
    scale = torch.clamp((top / largest).float(), min=2.0 ** -126)
    wide = scale.repeat_interleave(group, 1)[:, :M].repeat_interleave(128, 2)[..., :K]
    q = (x / wide.double()).float().double()
    bits, least = (3, -6) if t8 == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** least)))
    step = torch.exp2(e - bits)
    q = torch.clamp(torch.round(q / step) * step, -largest, largest)
    return torch.where(finite, q, math.nan), scale


def check_quantise(torch, x, group, t8, pad=0):
    batch, M, K = x.shape
    y = torch.full((batch, M, K + pad), 1.0, device="cuda").to(dtype_of(torch, t8))
    s = torch.full((batch, -(-M // group), -(-K // 128)), -1.0, device="cuda")
    sg.quantize_fp8(x, y[..., :K], s)
    q, scale = quantise_reference(torch, x, group, t8)
    assert torch.equal(s, scale)
    got = y[..., :K].double()
    assert torch.equal(got.nan_to_num(-1e9), q.nan_to_num(-1e9))
    assert bool((y[..., K:].float() == 1).all())
    status_is(0)


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("group", [1, 128])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 128), (2, 3, 127), (1, 129, 200), (1, 300, 1030), (3, 64, 256),
                                   (1, 5, 4096)])
def test_quantise_against_the_definition(torch, t, group, shape):
    g = gen(torch, sum(shape))
    x = (torch.randn(*shape, generator=g, device="cuda") * torch.exp(3 * torch.randn(shape[2], generator=g, device="cuda"))
         ).to(dtype_of(torch, t))
    for t8 in ("e4m3", "e5m2"):
        check_quantise(torch, x, group, t8)
    # Along the other axis, and rows at odd places.
    check_quantise(torch, x.transpose(1, 2), group, "e4m3", pad=3)
    wide = torch.randn(shape[0], shape[1], shape[2] + 3, generator=g, device="cuda").to(dtype_of(torch, t))
    check_quantise(torch, wide[..., 1:shape[2] + 1], group, "e4m3", pad=16)
    check_quantise(torch, wide[..., ::2], group, "e4m3")


@pytest.mark.parametrize("transposed", [False, True])
def test_quantise_odd_values(torch, transposed):
    # Ties (7 divides the largest magnitude's mantissa), zeros, NaN, infinities,
    # the smallest and largest numbers.
    x = torch.zeros(1, 256, 384, device="cuda", dtype=torch.float32)
    x[0, 0] = torch.arange(384, device="cuda") - 190.0
    x[0, 1, :128] = torch.arange(128, device="cuda") * 3.5
    x[0, 2, 5] = math.nan
    x[0, 2, 6:9] = torch.tensor([3.0, -4.0, 1e-30])
    x[0, 3, 130] = math.inf
    x[0, 3, 131] = -7.0
    x[0, 4, 0], x[0, 4, 1] = 3.4e38, -1e38
    x[0, 5, 0], x[0, 5, 1] = 1e-44, 3e-39
    x[0, 6, 0], x[0, 6, 1] = 1e-36, -0.0
    x[0, 130] = torch.randn(384, generator=gen(torch, 1), device="cuda").bfloat16().float()
    for group in (1, 128):
        for t8 in ("e4m3", "e5m2"):
            check_quantise(torch, x.transpose(1, 2).contiguous().transpose(1, 2) if transposed else x, group, t8)


def test_quantise_other_stream_and_capture(torch):
    x = torch.randn(1, 70, 300, generator=gen(torch, 3), device="cuda").bfloat16()
    want = quantise_reference(torch, x, 1, "e4m3")
    y = torch.zeros(1, 70, 300, device="cuda").to(torch.float8_e4m3fn)
    s = torch.zeros(1, 70, 3, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.quantize_fp8(x, y, s)
    side.synchronize()
    assert torch.equal(y.double(), want[0]) and torch.equal(s, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.quantize_fp8(x, y, s)
    x.copy_(torch.randn(1, 70, 300, generator=gen(torch, 4), device="cuda"))
    graph.replay()
    want = quantise_reference(torch, x, 1, "e4m3")
    assert torch.equal(y.double(), want[0]) and torch.equal(s, want[1])


# ---- the 8-bit product ----------------------------------------------------------------

def fp8_operand(torch, g, batch, rows, K, layout, t8, group, share=False):
    """(data [n, rows, K], scales [n, groups, blocks], values in 64 bits); layout:
    "k" unit stride along K, "p" the same with padded rows, "o" at an odd
    address, "r" unit stride along the rows, "i" the batch in the middle."""
    n, dt = 1 if share else batch, dtype_of(torch, t8)
    full = torch.randn(n, rows, K, generator=g, device="cuda") * (100.0 if t8 == "e4m3" else 1000.0)
    if layout == "k":
        x = full.to(dt)
    elif layout == "p":
        x = torch.nn.functional.pad(full, (0, -K % 16 + 16)).to(dt)[..., :K]
    elif layout == "o":
        x = torch.nn.functional.pad(full, (1, 0)).to(dt)[..., 1:]
    elif layout == "r":
        x = full.transpose(1, 2).contiguous().to(dt).transpose(1, 2)
    else:
        wide = torch.nn.functional.pad(full, (0, -K % 16))
        x = wide.transpose(0, 1).contiguous().to(dt).transpose(0, 1)[..., :K]
    s = torch.exp2(2 * torch.randn(n, -(-rows // group), -(-K // 128), generator=g, device="cuda"))
    wide = s.double().repeat_interleave(group, 1)[:, :rows].repeat_interleave(128, 2)[..., :K]
    return x, s, x.double() * wide


def check_fp8(torch, batch, M, N, K, la="k", lb="k", lc="c", ta="e4m3", tb="e4m3", ga=1, gb=128, tc="bf16",
              alpha=1.0, accumulate=False, share_a=False, share_b=False):
    g = gen(torch, 1000 * M + 10 * N + K)
    A, SA, va = fp8_operand(torch, g, batch, M, K, la, ta, ga, share_a)
    B, SB, vb = fp8_operand(torch, g, batch, N, K, lb, tb, gb, share_b)
    dt = dtype_of(torch, tc)
    size = 1e-4 / K
    if lc == "c":
        C = torch.randn(batch, M, N, generator=g, device="cuda").to(dt)
    elif lc == "t":
        C = torch.randn(batch, N, M, generator=g, device="cuda").to(dt).transpose(1, 2)
    else:
        C = torch.randn(batch, M, N + 3, generator=g, device="cuda").to(dt)[..., 1:N + 1]
    base = C if C._base is None else C._base
    if not accumulate:
        C.fill_(math.nan)
    before, old = base.clone(), C.double()
    alpha = alpha * size
    ref = alpha * torch.matmul(va, vb.transpose(1, 2))
    S = abs(alpha) * torch.matmul(va.abs(), vb.abs().transpose(1, 2))
    if accumulate:
        ref, S = ref + old, S + old.abs()
    sg.matmul_fp8(A, SA, B.transpose(1, 2), SB.transpose(1, 2), C, alpha=alpha, accumulate=accumulate)
    # (Beyond 464 or 61440 a conversion to 8 bits gives NaN: its row or column is NaN.)
    assert torch.equal(torch.isnan(C), torch.isnan(ref))
    lim = (K + -(-K // 128) + 8) * U * S + HALF[tc] * ref.abs() + TINY
    assert_within(torch, C.nan_to_num(0.0), ref.nan_to_num(0.0), lim.nan_to_num(0.0), f"{batch}x{M}x{N}x{K} {la}{lb}{lc} {ta} {tb} {ga} {gb} {tc}")
    mine = torch.zeros_like(base, dtype=torch.bool)
    torch.as_strided(mine, C.shape, C.stride(), C.storage_offset()).fill_(True)
    bits = torch.int32 if tc == "fp32" else torch.int16
    assert torch.equal(base[~mine].view(bits), before[~mine].view(bits))
    status_is(0)


FP8_SIZES = [
    (1, 1, 1, 1), (1, 1, 8, 16), (1, 1, 256, 128), (3, 5, 9, 31), (2, 17, 130, 144), (1, 16, 512, 4096),
    (1, 40, 300, 1040), (1, 64, 64, 1), (2, 127, 129, 272), (1, 128, 256, 128), (1, 129, 257, 384),
    (1, 300, 520, 640), (1, 257, 1000, 4112), (5, 33, 48, 2000), (1, 1000, 700, 256), (1, 2, 5000, 512),
]


@pytest.mark.parametrize("ga,gb", [(1, 128), (1, 1), (128, 128), (128, 1)])
@pytest.mark.parametrize("size", FP8_SIZES)
def test_fp8_sizes(torch, size, ga, gb):
    # Rows padded to whole 16 bytes take the tensor cores, odd ones the other kernel.
    check_fp8(torch, *size, la="p", lb="p", ga=ga, gb=gb, tc="bf16")
    check_fp8(torch, *size, la="k", lb="k", ga=ga, gb=gb, tc="fp32", lc="t")


@pytest.mark.parametrize("tc", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ta,tb", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_fp8_types(torch, tc, ta, tb):
    check_fp8(torch, 1, 150, 300, 400, la="p", lb="p", ta=ta, tb=tb, tc=tc)
    check_fp8(torch, 2, 20, 70, 160, la="r", lb="o", ta=ta, tb=tb, tc=tc)


@pytest.mark.parametrize("la,lb,lc", [("p", "p", "c"), ("i", "p", "o"), ("i", "i", "t"), ("r", "p", "c"), ("o", "r", "o")])
def test_fp8_layouts_alpha_accumulate_and_sharing(torch, la, lb, lc):
    for tc in ("bf16", "fp32"):
        check_fp8(torch, 3, 70, 200, 272, la, lb, lc, tc=tc, alpha=-0.37, accumulate=True)
        check_fp8(torch, 3, 140, 72, 400, la, lb, lc, tc=tc, ga=128, gb=1, alpha=0.0)
        check_fp8(torch, 4, 33, 128, 512, la, lb, lc, tc=tc, share_a=True)
        check_fp8(torch, 4, 33, 600, 512, la, lb, lc, tc=tc, share_b=True, accumulate=True)


def test_fp8_small_integers_are_exact(torch):
    g = gen(torch, 9)
    for M, N, K in ((16, 512, 4096), (300, 260, 1024), (70, 40, 48)):
        A = torch.randint(-2, 3, (M, K), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
        B = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
        SA = torch.full((M, -(-K // 128)), 2.0, device="cuda")
        SB = torch.full((-(-N // 128), -(-K // 128)), 0.5, device="cuda")
        C = torch.empty(M, N, device="cuda")
        sg.matmul_fp8(A, SA, B.t(), SB.t(), C)
        assert torch.equal(C.double(), A.double() @ B.double().t())


def test_fp8_edges(torch):
    e4 = torch.float8_e4m3fn
    C = torch.ones(2, 3, 8, device="cuda")
    A, SA = torch.ones(2, 3, 0, device="cuda").to(e4), torch.ones(2, 3, 0, device="cuda")
    B, SB = torch.ones(2, 0, 8, device="cuda").to(e4), torch.ones(2, 0, 1, device="cuda")
    sg.matmul_fp8(A, SA, B, SB, C, accumulate=True)
    assert bool((C == 1).all())
    sg.matmul_fp8(A, SA, B, SB, C)
    assert bool((C == 0).all())
    # NaN in an operand or a scale goes to its own rows and columns and nowhere else.
    for M, N, K in ((130, 260, 256), (5, 260, 256)):
        A, SA = torch.ones(M, K, device="cuda").to(e4), torch.ones(M, 2, device="cuda")
        B, SB = torch.ones(N, K, device="cuda").to(e4), torch.ones(N, 2, device="cuda")
        A[2, 3] = math.nan
        SA[3, 1] = math.inf
        SB[9, 0] = math.nan
        C = torch.empty(M, N, device="cuda", dtype=torch.float16)
        sg.matmul_fp8(A, SA, B.t(), SB.t(), C)
        want = torch.full((M, N), float(K), device="cuda")
        want[3] = math.inf
        want[:, 9] = math.nan
        want[2] = math.nan
        assert torch.equal(torch.nan_to_num(C.float(), nan=-1.0, posinf=-2.0), torch.nan_to_num(want, nan=-1.0, posinf=-2.0))


def test_fp8_repeats_and_captures(torch):
    g = gen(torch, 12)
    for M, N, K in ((16, 512, 7168), (300, 520, 1024)):
        A, SA, _ = fp8_operand(torch, g, 1, M, K, "k", "e4m3", 1)
        B, SB, _ = fp8_operand(torch, g, 1, N, K, "k", "e4m3", 128)
        C = torch.empty(1, M, N, device="cuda")
        sg.matmul_fp8(A, SA, B.transpose(1, 2), SB.transpose(1, 2), C)
        first = C.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            sg.matmul_fp8(A, SA, B.transpose(1, 2), SB.transpose(1, 2), C)
        C.fill_(math.nan)
        for _ in range(3):
            graph.replay()
        assert torch.equal(C.nan_to_num(0.5), first.nan_to_num(0.5))


def test_linear_layer_forward_and_backward_in_8_bits(torch):
    """A linear layer's three products from quantised operands: each against the
    64-bit product of the very operands it read."""
    g = gen(torch, 21)
    T, N, K = 200, 272, 400
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    w = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).bfloat16()
    dy = torch.randn(T, N, generator=g, device="cuda").bfloat16()

    def quantised(a, group):
        rows, k = a.shape
        y = torch.zeros(rows, -(-k // 16) * 16, device="cuda").to(torch.float8_e4m3fn)[:, :k]
        s = torch.empty(-(-rows // group), -(-k // 128), device="cuda")
        sg.quantize_fp8(a, y, s)
        return y, s, y.double() * s.double().repeat_interleave(group, 0)[:rows].repeat_interleave(128, 1)[:, :k]

    for a, ga, b, gb in ((x, 1, w, 128), (dy, 1, w.t(), 128), (dy.t(), 1, x.t(), 1)):
        (A, SA, va), (B, SB, vb) = quantised(a, ga), quantised(b, gb)
        C = torch.empty(a.shape[0], b.shape[0], device="cuda")
        sg.matmul_fp8(A, SA, B.t(), SB.t(), C)
        ref, S = va @ vb.t(), va.abs() @ vb.abs().t()
        k = a.shape[1]
        assert_within(torch, C, ref, (k + -(-k // 128) + 8) * U * S + HALF["fp32"] * ref.abs() + TINY)
        # Two roundings of at most 2^-4 each (2^-10 / 448 of the block's largest
        # below e4m3's normals) stand between the product and the unrounded one.
        full, size = a.double() @ b.double().t(), a.double().abs() @ b.double().abs().t()
        assert float((C.double() - full).abs().max()) <= 0.14 * float(size.max())


# ---- norms and rotations ---------------------------------------------------------------

def pairs_of(x, start, dims, interleaved):
    z = x[..., start:start + dims]
    return (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., :dims // 2], z[..., dims // 2:])


class Rope:
    """Parts (heads, D, norm, start) over `tokens` tokens, packed side by side."""

    def __init__(self, torch, t, tokens, dims, interleaved, parts, factor=1.0, longest=100000, seed=0, gap=0,
                 weights=True, negative=False):
        g = gen(torch, seed)
        dt = dtype_of(torch, t)
        self.torch, self.t, self.tokens, self.dims, self.interleaved, self.parts = torch, t, tokens, dims, interleaved, parts
        self.frequencies = sg.rope_frequencies(dims, factor=factor) if dims else []
        self.table = sg.rope_table(dims, factor=factor)
        lo = -longest if negative else 0
        self.positions = torch.randint(lo, longest, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        wide = sum(h * d for h, d, _, _ in parts) + gap
        new = lambda: torch.randn(tokens, wide, generator=g, device="cuda").to(dt)
        self.packed, self.dpacked = new(), new()
        self.x, self.dy, self.w, at = [], [], [], gap
        for h, d, n, _ in parts:
            self.x.append(self.packed[:, at:at + h * d].unflatten(1, (h, d)))
            self.dy.append(self.dpacked[:, at:at + h * d].unflatten(1, (h, d)))
            at += h * d
            self.w.append((1 + 0.2 * torch.randn(n, generator=g, device="cuda")).to(dt) if n and weights else None)

    def angles(self):
        torch = self.torch
        f = torch.tensor(self.frequencies, device="cuda", dtype=torch.float64)
        a = self.positions.double()[:, None, None] * f
        return a.cos() * self.table.magnitude, a.sin() * self.table.magnitude

    def reference(self, i):
        """(y, bound) of part i."""
        torch = self.torch
        _, _, n, start = self.parts[i]
        z = self.x[i].double()
        if n:
            r = torch.rsqrt(z[..., :n].square().mean(-1, keepdim=True) + 1e-6)
            w = self.w[i].double() if self.w[i] is not None else 1.0
            z = torch.cat([z[..., :n] * r * w, z[..., n:]], -1)
        y, size = z.clone(), z.abs()
        if self.dims:
            cos, sin = self.angles()
            a, b = pairs_of(z, start, self.dims, self.interleaved)
            u, v = pairs_of(y, start, self.dims, self.interleaved)
            u.copy_(a * cos - b * sin)
            v.copy_(a * sin + b * cos)
            for s in pairs_of(size, start, self.dims, self.interleaved):
                s.copy_(self.table.magnitude * (a.abs() + b.abs()))
        return y, (n / 2 + 24) * 2.0 ** -24 * size + HALF[self.t] * y.abs() + TINY

    def gradient(self, i):
        """(dx, its bound, dw, its bound) of part i."""
        torch = self.torch
        h, _, n, start = self.parts[i]
        dy = self.dy[i].double()
        g, G = dy.clone(), dy.abs()
        if self.dims:
            cos, sin = self.angles()
            u, v = pairs_of(dy, start, self.dims, self.interleaved)
            a, b = pairs_of(g, start, self.dims, self.interleaved)
            a.copy_(u * cos + v * sin)
            b.copy_(v * cos - u * sin)
            for s in pairs_of(G, start, self.dims, self.interleaved):
                s.copy_(self.table.magnitude * (u.abs() + v.abs()))
        dx, lim = g.clone(), (n + 32) * U * G
        dw = wlim = None
        if n:
            x = self.x[i].double()[..., :n]
            w = self.w[i].double() if self.w[i] is not None else torch.ones(n, device="cuda", dtype=torch.float64)
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
            xh = x * r
            gw, Gw = g[..., :n] * w, G[..., :n] * w.abs()
            dx[..., :n] = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
            lim[..., :n] = (n + 32) * U * r * (Gw + xh.abs() * (Gw * xh.abs()).mean(-1, keepdim=True))
            dw = (g[..., :n] * xh).sum((0, 1))
            wlim = (self.tokens * h + n + 32) * 2.0 ** -24 * (G[..., :n] * xh.abs()).sum((0, 1)) + TINY
        return dx, lim + HALF[self.t] * dx.abs() + TINY, dw, wlim

    def forward(self, y):
        sg.norm_rope([sg.RopePart(x, o, norm=p[2], weight=w, start=p[3])
                      for x, o, w, p in zip(self.x, y, self.w, self.parts)], self.positions, self.table,
                     interleaved=self.interleaved)

    def backward(self, dx, dw, accumulate=False):
        torch = self.torch
        ws = torch.full((sg.sbgemm_norm_rope_workspace_bytes([p[2] for p in self.parts]),), 255, device="cuda",
                        dtype=torch.uint8)
        sg.norm_rope_backward([sg.RopeGrad(x if p[2] else None, dy, o, norm=p[2], weight=w, dweight=d, start=p[3])
                               for x, dy, o, w, d, p in zip(self.x, self.dy, dx, self.w, dw, self.parts)],
                              self.positions, self.table, interleaved=self.interleaved, accumulate=accumulate,
                              workspace=ws)

    def check(self):
        torch = self.torch
        y = [torch.full_like(x, math.nan, memory_format=torch.contiguous_format) for x in self.x]
        self.forward(y)
        for i, o in enumerate(y):
            ref, lim = self.reference(i)
            assert_within(torch, o, ref, lim, f"part {i}")
        dx = [torch.full_like(o, math.nan) for o in y]
        dw = [torch.full((p[2],), math.nan, device="cuda") if p[2] else None for p in self.parts]
        self.backward(dx, dw)
        for i in range(len(y)):
            rx, lx, rw, lw = self.gradient(i)
            assert_within(torch, dx[i], rx, lx, f"dx of part {i}")
            if rw is not None:
                assert_within(torch, dw[i], rw, lw, f"dw of part {i}")
        status_is(0)


ROPES = [
    # tokens, dims, parts (heads, D, norm, start)
    (1, 2, [(1, 2, 0, 0)]),
    (1, 64, [(16, 192, 0, 128), (1, 576, 512, 512)]),
    (33, 128, [(32, 128, 128, 0), (8, 128, 128, 0)]),
    (70, 32, [(15, 64, 0, 0), (5, 64, 0, 0)]),
    (5, 40, [(3, 80, 80, 40)]),
    (5, 80, [(3, 80, 80, 0)]),
    (9, 48, [(7, 96, 96, 24), (2, 96, 0, 48)]),
    (6, 6, [(3, 7, 5, 1)]),
    (4, 16, [(2, 33, 33, 17)]),
    (3, 64, [(2, 256, 100, 128), (1, 320, 256, 256), (4, 64, 64, 0)]),
    (700, 64, [(3, 64, 64, 0)]),
    (2, 1024, [(2, 2048, 2048, 512)]),
    (2, 4096, [(1, 4096, 4096, 0)]),
    (3, 0, [(5, 128, 128, 0), (1, 100, 60, 0)]),
    (5, 16, [(12, 16, 16, 0)]),
]


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", range(len(ROPES)))
def test_rope_against_64_bits(torch, t, interleaved, case):
    tokens, dims, parts = ROPES[case]
    Rope(torch, t, tokens, dims, interleaved, parts, seed=case).check()
    Rope(torch, t, tokens, dims, interleaved, parts, seed=case + 50, factor=8.0, gap=1, weights=False,
         negative=True).check()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_far_positions(torch, interleaved):
    r = Rope(torch, "fp32", 40, 64, interleaved, [(2, 64, 0, 0)], longest=1000000, seed=3)
    r.positions[:6] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 16777217], device="cuda", dtype=torch.int32)
    # At 2^31 positions the reference's own angles (64 bits, 10^9 radians) are off by 2^-23.
    r.frequencies = [1.0 / 2 ** i for i in range(32)]
    r.table = sg.rope_table(64, frequencies=r.frequencies)
    y = [torch.empty_like(r.x[0], memory_format=torch.contiguous_format)]
    r.forward(y)
    ref, lim = r.reference(0)
    assert_within(torch, y[0], ref, lim + 2.0 ** -22 * r.x[0].double().abs().amax(-1, keepdim=True))


def test_rope_in_place(torch):
    for parts, dims in (([(16, 192, 0, 128), (1, 576, 512, 512)], 64), ([(4, 128, 128, 0), (2, 128, 128, 0)], 128),
                        ([(3, 7, 5, 1), (2, 9, 9, 0)], 6)):
        r = Rope(torch, "bf16", 37, dims, True, parts, gap=8)
        want = [r.reference(i) for i in range(len(parts))]
        grads = [r.gradient(i) for i in range(len(parts))]
        edge = r.packed[:, :8].clone()
        dw = [torch.empty(p[2], device="cuda") if p[2] else None for p in parts]
        r.backward(r.dy, dw)
        for i in range(len(parts)):
            assert_within(torch, r.dy[i], *grads[i][:2], "dx in dy's place")
        r.forward(r.x)
        for i in range(len(parts)):
            assert_within(torch, r.x[i], *want[i], "y in x's place")
        assert torch.equal(r.packed[:, :8], edge)


def test_rope_gradient_accumulates_and_repeats(torch):
    r = Rope(torch, "bf16", 600, 64, False, [(9, 64, 64, 0), (2, 64, 64, 0)])
    dx = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in r.x]
    a = [torch.zeros(64, device="cuda") for _ in r.parts]
    r.backward(dx, a)
    b = [w.clone() for w in a]
    first = [d.clone() for d in dx]
    r.backward(dx, b, accumulate=True)
    for x, y in zip(a, b):
        assert torch.equal(2 * x, y)
    for _ in range(3):
        r.backward(dx, b)
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and all(torch.equal(x, y) for x, y in zip(first, dx))
    # One of the weights' gradients alone, and none.
    r.backward(dx, [None, b[1].fill_(math.nan)])
    assert torch.equal(b[1], a[1])
    r.backward(dx, [None, None])
    assert all(torch.equal(x, y) for x, y in zip(first, dx))


def test_workspaces_are_kept_to(torch):
    """Nothing is written behind a workspace of the size that is asked for."""
    for tokens, parts in ((2000, [(64, 128, 128, 0), (1, 16, 16, 0), (1, 16, 16, 0), (1, 16, 16, 0)]),
                          (900, [(9, 9, 9, 0), (1, 7, 7, 0)]), (5000, [(1, 64, 64, 0)])):
        r = Rope(torch, "bf16", tokens, 0, False, parts)
        need = sg.sbgemm_norm_rope_workspace_bytes([p[2] for p in parts])
        whole = torch.full((need + 65536,), 77, device="cuda", dtype=torch.uint8)
        dx = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in r.x]
        dw = [torch.empty(p[2], device="cuda") for p in parts]
        sg.norm_rope_backward([sg.RopeGrad(x, dy, o, norm=p[2], weight=w, dweight=d)
                               for x, dy, o, w, d, p in zip(r.x, r.dy, dx, r.w, dw, parts)], None, None,
                              workspace=whole[:need])
        assert bool((whole[need:] == 77).all())
        for i in range(len(parts)):
            _, _, rw, lw = r.gradient(i)
            assert_within(torch, dw[i], rw, lw)
    for groups, heads, R in (([(300, *range(1, 50))], 16, 512), ([(n, n) for n in range(1, 90)], 5, 128), ([(1, 1)], 1, 40)):
        c = Shared(torch, "bf16", groups, heads, 1, R, 8, 16)
        need = c.workspace.numel()
        whole = torch.full((need + 65536,), 77, device="cuda", dtype=torch.uint8)
        c.workspace = whole[:need]
        c.run()
        c.check(torch)
        assert bool((whole[need:] == 77).all())


def test_rope_gradient_in_place_of_its_input(torch):
    r = Rope(torch, "fp32", 37, 64, True, [(4, 128, 128, 0), (1, 96, 64, 32)], gap=8)
    want = [r.gradient(i) for i in range(2)]
    dw = [torch.empty(128, device="cuda"), torch.empty(64, device="cuda")]
    r.backward(r.x, dw)
    for i in range(2):
        assert_within(torch, r.x[i], *want[i][:2])
        assert_within(torch, dw[i], *want[i][2:])


def test_rope_gradient_against_differences(torch):
    r = Rope(torch, "fp32", 7, 32, True, [(3, 64, 48, 16)], factor=4.0)
    x0 = r.x[0].clone()
    dx = [torch.empty_like(x0)]
    r.backward(dx, [torch.empty(48, device="cuda")])
    rx, lx, _, _ = r.gradient(0)
    d = torch.randn(x0.shape, generator=gen(torch, 8), device="cuda")
    step, y = 2.0 ** -6, [torch.empty_like(x0)]
    got = ref = noise = 0.0
    for sign in (1.0, -1.0):
        r.x[0].copy_(x0 + sign * step * d)
        r.forward(y)
        got += sign * float((y[0].double() * r.dy[0].double()).sum()) / (2 * step)
        want, lim = r.reference(0)
        ref += sign * float((want * r.dy[0].double()).sum()) / (2 * step)
        # Rounding of y and of x0 + step d itself.
        noise += float(((lim + 2.0 ** -23 * want.abs()) * r.dy[0].double().abs()).sum()) / (2 * step)
    bend = abs(ref - float((rx * d.double()).sum()))      # the difference's own error, from the formula
    have = float((dx[0].double() * d.double()).sum())
    assert abs(have - got) <= bend + noise + float((lx * d.double().abs()).sum())


def test_rope_edges(torch):
    t = sg.rope_table(4)
    x = torch.randn(0, 2, 8, device="cuda")
    none = torch.zeros(0, device="cuda", dtype=torch.int32)
    sg.norm_rope([sg.RopePart(x, torch.empty_like(x), norm=8)], none, t)
    dw = torch.full((8,), math.nan, device="cuda")
    ws = torch.empty(sg.sbgemm_norm_rope_workspace_bytes([8]), device="cuda", dtype=torch.uint8)
    sg.norm_rope_backward([sg.RopeGrad(x, x, torch.empty_like(x), norm=8, dweight=dw)], none, t, workspace=ws)
    assert bool((dw == 0).all())
    dw.fill_(3.0)
    sg.norm_rope_backward([sg.RopeGrad(x, x, torch.empty_like(x), norm=8, dweight=dw)], none, t, accumulate=True,
                          workspace=ws)
    assert bool((dw == 3).all())
    # Rows of zeros, NaN and infinity keep to themselves.
    for dims, D in ((64, 128), (4, 9)):
        x = torch.randn(4, 3, D, generator=gen(torch, 2), device="cuda")
        x[0, 0], x[1, 1, 2], x[2, 2, 3] = 0.0, math.nan, math.inf
        y = torch.empty_like(x)
        pos = torch.arange(4, device="cuda", dtype=torch.int32)
        sg.norm_rope([sg.RopePart(x, y, norm=D)], pos, sg.rope_table(dims))
        assert bool((y[0, 0] == 0).all())
        bad = torch.zeros(4, 3, device="cuda", dtype=torch.bool)
        bad[1, 1] = bad[2, 2] = True
        assert torch.equal(torch.isnan(y).any(-1), bad)
        assert bool(torch.isnan(y[1, 1]).all())


def test_rope_streams_and_capture(torch):
    r = Rope(torch, "bf16", 40, 64, True, [(16, 192, 0, 128), (1, 576, 512, 512)])
    y = [torch.zeros_like(x, memory_format=torch.contiguous_format) for x in r.x]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r.forward(y)
    side.synchronize()
    for i in range(2):
        assert_within(torch, y[i], *r.reference(i))
    dx = [torch.zeros_like(o) for o in y]
    dw = [None, torch.zeros(512, device="cuda")]
    ws = torch.empty(sg.sbgemm_norm_rope_workspace_bytes([512]), device="cuda", dtype=torch.uint8)
    parts = [sg.RopeGrad(x, dy, o, norm=p[2], weight=w, dweight=d, start=p[3])
             for x, dy, o, w, d, p in zip(r.x, r.dy, dx, r.w, dw, r.parts)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward(y)
        sg.norm_rope_backward(parts, r.positions, r.table, interleaved=True, workspace=ws)
    r.packed.copy_(torch.randn(r.packed.shape, generator=gen(torch, 5), device="cuda"))
    r.positions.add_(1)
    graph.replay()
    graph.replay()
    for i in range(2):
        assert_within(torch, y[i], *r.reference(i))
        rx, lx, rw, lw = r.gradient(i)
        assert_within(torch, dx[i], rx, lx)
        if rw is not None:
            assert_within(torch, dw[i], rw, lw)


# ---- latent attention over shared prefixes -----------------------------------------------

class Shared:
    """Groups of sequences: `groups` holds (prefix, own lengths ...), a prefix of
    None for sequences outside any group (before the first one or behind the
    last one; between others they are a group without a prefix).  Only the keys that the definition
    reads exist: the prefix at the first sequence's pages, the others' entries
    for whole pages of it -1, every other row of the cache NaN."""

    def __init__(self, torch, t, groups, heads, q_len, R, P, block, seed=0, scale=1.0, shared_pages=False):
        dt, D, g = dtype_of(torch, t), R + P, gen(torch, seed)
        self.t, self.heads, self.q_len, self.R, self.P, self.block = t, heads, q_len, R, P, block
        lens, starts, prefixes, of = [], [0], [], []
        for i, (prefix, *own) in enumerate(groups):
            if prefix is None and i == 0:
                starts = [len(own)]
            elif prefix is None and i + 1 < len(groups):
                prefix = 0
            lead = len(lens)
            for n in own:
                lead = lead if prefix else len(lens)
                lens.append((prefix or 0) + n)
                of.append((lead, prefix or 0))
            if prefix is not None:
                starts.append(len(lens))
                prefixes.append(prefix)
        S = len(lens)
        self.lens, self.of = lens, of
        most = max(1, max(-(-n // block) for n in lens)) + 1
        blocks = S * most + 3
        order = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        table = order[:S * most].view(S, most).clone()
        whole = torch.full((blocks, block, D), math.nan, device="cuda").to(dt)
        self.ctx = []
        pos = torch.arange(most * block, device="cuda")
        for s, (n, (lead, prefix)) in enumerate(zip(lens, of)):
            kv = torch.randn(n, D, generator=g, device="cuda").to(dt)
            if s != lead:
                kv[:prefix] = self.raw[lead][:prefix]
                if shared_pages:
                    table[s, :prefix // block] = table[lead, :prefix // block]
                else:
                    table[s, :prefix // block] = -1
            else:
                self.raw = getattr(self, "raw", {})
                self.raw[lead] = kv
            lo = 0 if s == lead else prefix
            if n > lo:
                whole[table[s].long()[pos[lo:n] // block], pos[lo:n] % block] = kv[lo:]
            table[s, -(-n // block):] = -1
            self.ctx.append(kv.double())
        self.cache, self.table = whole, table
        i32 = dict(device="cuda", dtype=torch.int32)
        self.seq_lens = torch.tensor(lens, **i32)
        self.starts, self.prefixes = torch.tensor(starts, **i32), torch.tensor(prefixes, **i32)
        self.q = (scale * torch.randn(S, q_len, heads, D, generator=g, device="cuda")).to(dt)
        self.o = torch.full((S, q_len, heads, R), math.nan, device="cuda", dtype=dt)
        self.alpha = 1.0 / math.sqrt(D)
        self.workspace = torch.full((sg.sbgemm_latent_shared_workspace_bytes(S, len(prefixes), q_len, heads, R),), 255,
                                    device="cuda", dtype=torch.uint8)

    def run(self, causal=True, **kw):
        return sg.latent_attention_shared(self.q, self.cache, self.table, self.seq_lens, self.starts, self.prefixes,
                                          self.o, alpha=self.alpha, causal=causal, workspace=self.workspace, **kw)

    def check(self, torch, causal=True, alive=None):
        for s, n in enumerate(self.lens):
            q = self.q[s].double().transpose(0, 1)
            m = torch.arange(self.q_len, device="cuda")[:, None]
            keep = torch.ones(self.q_len, n, device="cuda", dtype=torch.bool)
            if causal:
                keep = torch.arange(n, device="cuda")[None, :] <= n - self.q_len + m
            kv = self.ctx[s]
            O, W, Z, sv = attention_reference(q, kv, kv[:, : self.R], self.alpha, keep)
            lim = attention_bound(self.t, self.R + self.P, n, O, W, Z, sv)
            assert_within(torch, self.o[s].transpose(0, 1), O, lim, f"sequence {s} of length {n}")


SHARED = [
    # groups (prefix, own lengths ...), heads, q_len, R, P, block, causal
    ([(1, 1)], 1, 1, 512, 64, 16, True),
    ([(100, 1, 1, 1)], 16, 1, 512, 64, 16, True),
    ([(64, 30, 0, 100, 7)], 16, 1, 512, 64, 64, True),
    ([(0, 30, 5), (17, 1, 80), (200, 3)], 16, 1, 512, 64, 8, True),
    ([(1000, 130, 5, 64, 65, 1, 200, 31, 90)], 16, 1, 512, 64, 32, True),
    ([(333, 1, 100), (None, 70, 0), (50, 9, 9, 9)], 8, 3, 512, 64, 24, True),
    ([(333, 40, 100), (50, 9, 12, 9)], 20, 2, 512, 64, 1, False),
    ([(130, 5, 0, 1)], 128, 1, 512, 64, 64, True),
    ([(70, 9, 40), (300, 1, 2, 3)], 64, 2, 256, 32, 16, True),
    ([(90, 31, 2)], 33, 1, 384, 16, 17, True),
    ([(90, 31, 2)], 5, 1, 128, 0, 48, False),
    ([(70, 9, 1)], 3, 2, 96, 24, 16, True),
    ([(70, 9, 1), (5, 3)], 3, 1, 40, 7, 5, True),
    ([(5000,) + tuple(range(1, 60, 3))], 16, 1, 512, 64, 16, True),
    ([(200, 1, 0, 0, 1, 1)], 4, 4, 512, 64, 64, True),     # queries that see less than the whole prefix
    ([(3, 0, 0), (1, 0)], 16, 5, 512, 64, 64, True),       # queries without a key
    ([(n, 1) for n in range(1, 41)], 16, 1, 512, 64, 16, True),
    ([(None, 40, 3), (100, 9, 2), (None, 0, 130)], 16, 1, 512, 64, 16, True),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(SHARED)))
def test_shared_against_64_bits(torch, t, case):
    groups, heads, q_len, R, P, block, causal = SHARED[case]
    c = Shared(torch, t, groups, heads, q_len, R, P, block, seed=case)
    c.run(causal)
    c.check(torch, causal)
    status_is(0)


def test_shared_equals_the_paged_operator(torch):
    c = Shared(torch, "bf16", [(640, 100, 30, 7), (64, 5, 300)], 16, 2, 512, 64, 64, shared_pages=True)
    c.run()
    split = torch.empty(sg.sbgemm_latent_workspace_bytes(torch.cuda.current_device()), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(c.o)
    sg.latent_attention_paged(c.q, c.cache, c.table, c.seq_lens, o, alpha=c.alpha, workspace=split)
    assert float((c.o.float() - o.float()).abs().max()) <= 2 ** -7 * float(o.float().abs().max())
    # Without groups every sequence reads its own keys.
    c.starts, c.prefixes = c.starts[:1], c.prefixes[:0]
    c.o.fill_(math.nan)
    c.run()
    c.check(torch)


def test_shared_large_scores_and_scales(torch):
    for alpha in (None, -0.05, 0.0):
        c = Shared(torch, "fp16", [(300, 130, 64, 1)], 16, 1, 512, 64, 16, seed=5, scale=20.0 if alpha is None else 1.0)
        if alpha is not None:
            c.alpha = alpha
        c.run()
        c.check(torch)


def test_shared_reports_what_it_clamps(torch):
    def fresh():
        return Shared(torch, "bf16", [(64, 30, 20, 10), (32, 5, 6)], 16, 1, 512, 64, 16, shared_pages=True)

    # Starts out of range or decreasing, prefixes past the first sequence or negative, bad lengths and ids.
    def spoil_starts(c):
        c.starts[1] = -5            # an empty first group; the second one holds all
        c.starts[2] = 99

    def spoil_order(c):
        c.starts[0], c.starts[1], c.starts[2] = 4, 2, 5

    def spoil_prefix(c):
        c.prefixes[0] = 1000

    def spoil_negative(c):
        c.prefixes[1] = -3

    def spoil_lens(c):
        c.seq_lens[4] = 100000

    def spoil_table(c):
        c.table[0, 1] = 10 ** 6

    for spoil in (spoil_starts, spoil_order, spoil_prefix, spoil_negative, spoil_lens, spoil_table):
        c = fresh()
        spoil(c)
        c.run()
        status_is(10)
    c = fresh()
    c.run()
    c.check(torch)
    status_is(0)


def test_shared_sequences_shorter_than_the_prefix(torch):
    # The definition: a sequence sees its own length's keys of the prefix.
    c = Shared(torch, "bf16", [(200, 50, 0, 0)], 16, 1, 512, 64, 32)
    c.seq_lens[1] = 77
    c.lens[1], c.ctx[1] = 77, c.ctx[1][:77]
    c.seq_lens[2] = 0
    c.lens[2], c.ctx[2] = 0, c.ctx[2][:0]
    c.run()
    c.check(torch)
    assert bool((c.o[2] == 0).all())
    status_is(0)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_shared_by_many(torch, t):
    # More sequences than a planning thread each, in groups of many sizes.
    sizes = [1, 2, 3, 700, 5, 6, 400, 31]
    c = Shared(torch, t, [(10 * n % 97, *((i * 7 + n) % 40 for i in range(n))) for n in sizes], 2, 1, 128, 64, 16, seed=1)
    assert len(c.lens) > 1024
    c.run()
    c.check(torch)
    status_is(0)
    # More groups than that, most of them empty.
    empty = c.starts[1:2].repeat(2000)
    c.starts = torch.cat([c.starts[:1], empty, c.starts[2:]])
    c.prefixes = torch.cat([c.prefixes[:1], torch.full((1999,), 5, device="cuda", dtype=torch.int32), c.prefixes[1:]])
    c.workspace = torch.empty(sg.sbgemm_latent_shared_workspace_bytes(len(c.lens), len(c.prefixes), 1, 2, 128),
                              device="cuda", dtype=torch.uint8)
    c.o.fill_(math.nan)
    c.run()
    c.check(torch)
    status_is(0)


def test_shared_capture_and_two_streams(torch):
    c = Shared(torch, "bf16", [(640, 100, 30, 7), (64, 5, 300)], 16, 1, 512, 64, 64)
    d = Shared(torch, "bf16", [(900, 10, 3)], 16, 1, 512, 64, 64, seed=9)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (a, b):
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(a):
            c.run()
        with torch.cuda.stream(b):
            d.run()
    torch.cuda.synchronize()
    c.check(torch)
    d.check(torch)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run()
    # Other lengths and prefixes between replays, as a decode loop has them.
    c.seq_lens[1] += -3
    c.lens[1], c.ctx[1] = c.lens[1] - 3, c.ctx[1][:-3]
    c.prefixes[0] = 600
    c.table[1:3, :10] = c.table[0, :10]
    c.o.fill_(math.nan)
    graph.replay()
    graph.replay()
    c.check(torch)


def test_shared_strided_operands(torch):
    c = Shared(torch, "bf16", [(640, 100, 30, 7), (64, 5, 300)], 16, 2, 512, 64, 64)
    S = len(c.lens)
    wide = torch.zeros(c.q_len, S, 20, 600, device="cuda", dtype=torch.bfloat16)
    q = wide.transpose(0, 1)[:, :, 2:18, 8:584]
    q.copy_(c.q)
    c.q = q
    out = torch.full((c.q_len, S, 16, 520), 7.0, device="cuda", dtype=torch.bfloat16)
    c.o = out.transpose(0, 1)[..., 4:516]
    gap = torch.full((c.cache.shape[0], 64, 584), math.nan, device="cuda", dtype=torch.bfloat16)
    gap[..., :576] = c.cache
    c.cache = gap[..., :576]
    c.run()
    c.check(torch)
    assert bool((out[..., :4] == 7).all()) and bool((out[..., 516:] == 7).all())


# ---- together ------------------------------------------------------------------------------

def test_a_decode_step_of_forked_sequences(torch):
    """One step of a latent-attention layer for samples of one prompt: quantise,
    project with 8-bit weights, norm and rotate queries and the new latent rows,
    append them to the forks of the prompt, attend with the prompt read once.
    Each operator is held against 64 bits on the very inputs it read."""
    g = gen(torch, 77)
    S, H, R, P, nope, hidden, block, prompt = 6, 16, 512, 64, 128, 400, 32, 200
    bf, i32 = dict(device="cuda", dtype=torch.bfloat16), dict(device="cuda", dtype=torch.int32)
    x = torch.randn(S, hidden, generator=g, device="cuda").bfloat16()
    N = H * (R + P) + R + P
    w8 = torch.empty(N, hidden, device="cuda", dtype=torch.float8_e4m3fn)
    ws = torch.empty(-(-N // 128), -(-hidden // 128), device="cuda")
    sg.quantize_fp8((torch.randn(N, hidden, generator=g, device="cuda") / math.sqrt(hidden)).bfloat16(), w8, ws)
    x8, xs = torch.empty(S, hidden, device="cuda", dtype=torch.float8_e4m3fn), torch.empty(S, 4, device="cuda")
    y = torch.empty(S, N, **bf)
    sg.quantize_fp8(x, x8, xs)
    sg.matmul_fp8(x8, xs, w8.t(), ws.t(), y)
    va = x8.double() * xs.double().repeat_interleave(128, 1)[:, :hidden]
    vb = w8.double() * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :hidden]
    ref = va @ vb.t()
    assert_within(torch, y, ref, (hidden + 12) * U * (va.abs() @ vb.abs().t()) + HALF["bf16"] * ref.abs() + TINY)

    table = sg.rope_table(P, factor=4.0)
    q, row = y[:, :H * (R + P)].unflatten(1, (H, R + P)), y[:, H * (R + P):]
    before = [q.clone(), row.clone()]
    weight = (1 + 0.1 * torch.randn(R, generator=g, device="cuda")).bfloat16()
    positions = torch.full((S,), prompt, **i32)
    sg.norm_rope([sg.RopePart(q, q, start=R), sg.RopePart(row, row, norm=R, weight=weight, start=R)], positions, table,
                 interleaved=True)
    r = Rope(torch, "bf16", S, P, True, [(H, R + P, 0, R), (1, R + P, R, R)], factor=4.0)
    r.x, r.w, r.positions = [before[0], before[1].unsqueeze(1)], [None, weight], positions
    assert_within(torch, q, *r.reference(0))
    assert_within(torch, row.unsqueeze(1), *r.reference(1))

    pages = 64
    cache = torch.full((pages, block, R + P), math.nan, **bf)
    refs, tab, lens = torch.zeros(pages, **i32), torch.full((S, 16), -1, **i32), torch.zeros(S, **i32)
    work = torch.empty(sg.sbgemm_pages_workspace_bytes(pages, S, S), device="cuda", dtype=torch.uint8)
    old = torch.randn(prompt, R + P, generator=g, device="cuda").bfloat16()
    sg.pages_append([cache], refs, tab, lens, torch.zeros(1, **i32), torch.tensor([0, prompt], **i32), [old],
                    workspace=work)
    sg.pages_fork([cache], refs, tab, lens, torch.zeros(S - 1, **i32), torch.arange(1, S, **i32), workspace=work)
    sg.pages_append([cache], refs, tab, lens, torch.arange(S, **i32), torch.arange(S + 1, **i32), [row], workspace=work)
    o = torch.full((S, 1, H, R), math.nan, **bf)
    split = torch.empty(sg.sbgemm_latent_shared_workspace_bytes(S, 1, 1, H, R), device="cuda", dtype=torch.uint8)
    alpha = (nope + P) ** -0.5
    sg.latent_attention_shared(q.unsqueeze(1), cache, tab, lens, torch.tensor([0, S], **i32),
                               torch.tensor([prompt], **i32), o, alpha=alpha, workspace=split)
    for s in range(S):
        kv = torch.cat([old, row[s:s + 1]]).double()
        keep = torch.ones(1, prompt + 1, device="cuda", dtype=torch.bool)
        O, W, Z, sv = attention_reference(q[s].double()[:, None], kv, kv[:, :R], alpha, keep)
        assert_within(torch, o[s].transpose(0, 1), O, attention_bound("bf16", R + P, prompt + 1, O, W, Z, sv))
    status_is(0)
