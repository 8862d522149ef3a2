"""The 16-bit serving operators on the GPU against plain computations in 64
bits: the strided product, latent attention (absorbed over a paged cache,
expanded over packed sequences), and the page operations against a model of
the pool in Python.

Bounds, with u = 2^-23 for one fp32 addition whose excess bits may be cut off
(tensor cores) and h = half a step of the 16-bit type (2^-8 bf16, 2^-11 fp16,
relative; 2^-25 absolute below fp16's normals):

product   |C - ref| <= (K + 3) u S + h |ref| + 2^-25,  S = |alpha| sum |a b| (+ |C_old|)
attention a score is off by at most (D + 4) u Z, Z the row's largest
          |alpha| sum_d |q k|, so a weight by the factor exp of that, and the
          normalised weight by twice it, and by 2^-20 for exp2 and the joins of
          split keys; weights are rounded to the type for the second product
          (h, or 2^-25 below fp16's normals, against a sum of at least 1), and
          N + 8 additions make the sums:
          |O - ref| <= (2 (exp((D + 4) u Z) - 1) + 2^-20 + h + (N + 8) u) W + 2^-25 sum |v| + h |ref| + 2^-25,
          W = sum_n p_n |v_n|.
Caches hold NaN in every row that no sequence owns and tables -1 past each
sequence's pages, so a kernel that uses one of them fails the test."""

import math

import numpy as np
import pytest

import strided_gemm_gb300 as sg

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a CUDA device"
    sg.load()
    return t


@pytest.fixture(scope="module")
def workspace(torch):
    return torch.empty(sg.sbgemm_latent_workspace_bytes(torch.cuda.current_device()), dtype=torch.uint8,
                       device="cuda")


@pytest.fixture(autouse=True)
def clean_status(torch):
    sg.sbgemm_device_status()
    yield


def dtype_of(torch, t):
    return torch.bfloat16 if t == "bf16" else torch.float16


def status_is(code):
    st, where = sg.sbgemm_device_status()
    assert where == code, (st, where)
    assert st == (sg.SBGEMM_OK if code == 0 else sg.SBGEMM_ERR_DEVICE_CHECK)


def assert_within(torch, got, ref, lim, name=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= lim)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside the bound; first {i}: got "
                             f"{float(got[i])} want {float(ref[i])} bound {float(lim[i])}")


# ---- the product -----------------------------------------------------------------

def operand(torch, g, batch, rows, cols, layout, dt, share=False):
    """[batch, rows, cols] with the unit stride along cols ("c") or rows ("r"),
    cols with a stride of 2 ("g"), a padded row ("p": 16-byte multiple, "o":
    odd) or the batch in the middle ("i")."""
    n = 1 if share else batch
    if layout == "c":
        x = torch.randn(n, rows, cols, generator=g, device="cuda").to(dt)
    elif layout == "r":
        x = torch.randn(n, cols, rows, generator=g, device="cuda").to(dt).transpose(1, 2)
    elif layout == "g":
        x = torch.randn(n, rows, 2 * cols, generator=g, device="cuda").to(dt)[..., ::2]
    elif layout == "p":
        x = torch.randn(n, rows, -(-cols // 8) * 8 + 8, generator=g, device="cuda").to(dt)[..., :cols]
    elif layout == "o":
        x = torch.randn(n, rows, cols + 1, generator=g, device="cuda").to(dt)[..., 1:]
    else:
        x = torch.randn(rows, n, cols, generator=g, device="cuda").to(dt).transpose(0, 1)
    return x


def check_product(torch, t, batch, M, N, K, la, lb, lc, alpha=1.0, accumulate=False, share_a=False,
                  share_b=False, seed=0):
    dt = dtype_of(torch, t)
    g = torch.Generator(device="cuda").manual_seed(seed + M + 7 * N + 13 * K)
    A = operand(torch, g, batch, M, K, la, dt, share_a)
    B = operand(torch, g, batch, K, N, lb, dt, share_b)
    C = operand(torch, g, batch, M, N, lc, dt)
    base = C
    while base._base is not None:
        base = base._base
    if not accumulate:
        C.fill_(float("nan"))
    before = base.clone()
    old = C.double()
    ref = alpha * torch.matmul(A.double(), B.double())
    size = abs(alpha) * torch.matmul(A.double().abs(), B.double().abs())
    if accumulate:
        ref, size = ref + old, size + old.abs()
    sg.matmul_half(A, B, C, alpha=alpha, accumulate=accumulate)
    lim = (K + 3) * U * size + HALF[t] * ref.abs() + 2.0 ** -25
    assert_within(torch, C, ref, lim, f"{t} {batch}x{M}x{N}x{K} {la}{lb}{lc}")
    # Nothing beside C's own elements is written.
    mine = torch.zeros_like(base, dtype=torch.bool)
    torch.as_strided(mine, C.shape, C.stride(), C.storage_offset()).fill_(True)
    assert torch.equal(base[~mine].view(torch.int16), before[~mine].view(torch.int16))


PRODUCTS = [
    (1, 1, 1, 1), (1, 1, 8, 16), (3, 5, 9, 31), (2, 17, 33, 64), (1, 64, 64, 72), (2, 127, 65, 40),
    (1, 128, 128, 128), (3, 129, 136, 200), (1, 300, 264, 8), (2, 16, 512, 128), (5, 1, 128, 512),
    (1, 257, 392, 520), (1, 1000, 48, 136), (1, 2600, 2056, 72), (2, 1290, 2040, 1032),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("size", PRODUCTS)
def test_product_layouts(torch, t, size):
    for la, lb, lc in (("c", "c", "c"), ("c", "r", "c"), ("r", "c", "c"), ("r", "r", "r"), ("p", "p", "p"),
                       ("i", "r", "i"), ("g", "c", "c"), ("c", "o", "o"), ("c", "c", "r"), ("c", "r", "g")):
        check_product(torch, t, *size, la, lb, lc)
    status_is(0)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("la,lb", [("c", "r"), ("c", "c"), ("r", "c"), ("g", "o")])
def test_product_accumulate_alpha_and_sharing(torch, t, la, lb):
    check_product(torch, t, 3, 130, 72, 96, la, lb, "c", alpha=-0.37, accumulate=True)
    check_product(torch, t, 3, 40, 200, 96, la, lb, "p", alpha=0.0)
    check_product(torch, t, 4, 33, 128, 64, la, lb, "i", share_a=True)
    check_product(torch, t, 4, 33, 128, 64, la, lb, "i", share_b=True, accumulate=True)


@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_product_of_small_integers_is_exact(torch, t):
    dt = dtype_of(torch, t)
    g = torch.Generator(device="cuda").manual_seed(5)
    for M, N, K in ((130, 200, 120), (40, 264, 128), (9, 7, 31)):
        A = torch.randint(-1, 2, (2, M, K), generator=g, device="cuda").to(dt)
        B = torch.randint(-1, 2, (2, K, N), generator=g, device="cuda").to(dt)
        C = torch.empty(2, M, N, device="cuda", dtype=dt)
        sg.matmul_half(A, B, C)      # sums stay below 128: exact in both types
        assert torch.equal(C.double(), torch.matmul(A.double(), B.double()))


def test_product_edges(torch):
    C = torch.ones(2, 3, 8, device="cuda", dtype=torch.bfloat16)
    A = torch.ones(2, 3, 0, device="cuda", dtype=torch.bfloat16)
    B = torch.ones(2, 0, 8, device="cuda", dtype=torch.bfloat16)
    sg.matmul_half(A, B, C, accumulate=True)
    assert bool((C == 1).all())
    sg.matmul_half(A, B, C)
    assert bool((C == 0).all())
    # Infinity and NaN go where they belong and nowhere else.
    A = torch.ones(1, 130, 64, device="cuda", dtype=torch.float16)
    B = torch.ones(1, 64, 72, device="cuda", dtype=torch.float16)
    A[0, 5, 3], B[0, 7, 9] = float("inf"), float("nan")
    C = torch.empty(1, 130, 72, device="cuda", dtype=torch.float16)
    sg.matmul_half(A, B, C)
    want = torch.full((130, 72), 64.0, device="cuda")
    want[5] = float("inf")
    want[:, 9] = float("nan")
    assert torch.equal(torch.nan_to_num(C[0].float(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))
    # fp16 overflows to infinity.
    A = torch.full((1, 130, 64), 200.0, device="cuda", dtype=torch.float16)
    B = torch.full((1, 64, 72), 200.0, device="cuda", dtype=torch.float16)
    sg.matmul_half(A, B, C)
    assert bool(torch.isinf(C).all())


# ---- latent attention, absorbed form over a paged cache ------------------------------

def attention_reference(q, k, v, alpha, keep):
    """q [H, m, D], k and v [n, .] or [H, n, .], keep [m, n] (bool) in fp64:
    O and the terms of the bound (W, Z, sum |v|)."""
    import torch
    z = alpha * q @ k.transpose(-1, -2)
    size = abs(alpha) * (q.abs() @ k.abs().transpose(-1, -2))
    z = z.masked_fill(~keep, -math.inf)
    top = z.amax(-1, keepdim=True) if z.shape[-1] else torch.zeros(*z.shape[:-1], 1, device=z.device)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(z - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    Z = size.masked_fill(~keep, 0.0).amax(-1) if z.shape[-1] else torch.zeros(z.shape[:-1], device=z.device)
    sv = keep.double() @ v.abs()
    return p @ v, p @ v.abs(), Z, sv


def attention_bound(t, D, N, O, W, Z, sv):
    import torch
    h = HALF[t]
    rel = 2 * (torch.exp((D + 4) * U * Z) - 1) + 2.0 ** -20 + h + (N + 8) * U
    return rel[..., None] * W + 2.0 ** -25 * sv + h * O.abs() + 2.0 ** -25


class Paged:
    """A paged latent cache with the given lengths: NaN wherever no sequence's token is."""

    def __init__(self, torch, t, lens, heads, q_len, R, P, block, seed=0, spare=3, gap=0, scale=1.0):
        dt = dtype_of(torch, t)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.t, self.lens, self.R, self.P, self.block, self.q_len, self.heads = t, lens, R, P, block, q_len, heads
        S, D = len(lens), R + P
        pages = [-(-n // block) for n in lens]
        most = max(max(pages), 1)
        blocks = sum(pages) + spare
        order = rng.permutation(blocks)
        table = np.full((S, most + 1), -1, np.int32)
        whole = torch.full((blocks, block, D + gap), float("nan"), device="cuda").to(dt)
        self.cache = whole[..., :D]
        self.ctx, at = [], 0
        for s, n in enumerate(lens):
            table[s, : pages[s]] = order[at: at + pages[s]]
            at += pages[s]
            kv = torch.randn(n, D, generator=g, device="cuda").to(dt)
            self.ctx.append(kv.double())
            if n:
                ids = torch.from_numpy(table[s, : pages[s]].astype(np.int64)).cuda()
                pos = torch.arange(n, device="cuda")
                self.cache[ids[pos // block], pos % block] = kv
        self.table = torch.from_numpy(table).cuda()
        self.seq_lens = torch.tensor(lens, device="cuda", dtype=torch.int32)
        self.q = (scale * torch.randn(S, q_len, heads, D, generator=g, device="cuda")).to(dt)
        self.o = torch.full((S, q_len, heads, R), float("nan"), device="cuda", dtype=dt)
        self.alpha = 1.0 / math.sqrt(D)

    def run(self, causal, workspace, **kw):
        return sg.latent_attention_paged(self.q, self.cache, self.table, self.seq_lens, self.o, alpha=self.alpha,
                                         causal=causal, workspace=workspace, **kw)

    def check(self, torch, causal, got=None):
        got = self.o if got is None else got
        for s, n in enumerate(self.lens):
            q = self.q[s].double().transpose(0, 1)                       # [H, t, D]
            m = torch.arange(self.q_len, device="cuda")[:, None]
            keep = torch.ones(self.q_len, n, device="cuda", dtype=torch.bool)
            if causal:
                keep = torch.arange(n, device="cuda")[None, :] <= n - self.q_len + m
            kv = self.ctx[s]
            O, W, Z, sv = attention_reference(q, kv, kv[:, : self.R], self.alpha, keep)
            lim = attention_bound(self.t, self.R + self.P, n, O, W, Z, sv)
            assert_within(torch, got[s].transpose(0, 1), O, lim, f"sequence {s} of length {n}")


PAGED = [
    # lens, heads, q_len, R, P, block, causal
    ([1], 1, 1, 512, 64, 16, True),
    ([0, 1, 2, 63, 64, 65, 129], 16, 1, 512, 64, 16, True),
    ([700], 16, 1, 512, 64, 64, True),
    ([33, 500], 128, 1, 512, 64, 64, False),
    ([300, 5, 77], 20, 1, 512, 64, 24, True),
    ([2000, 1], 8, 3, 512, 64, 1, True),
    ([130, 2, 0, 1, 70], 16, 4, 512, 64, 32, True),
    ([130, 64, 3], 32, 3, 512, 64, 128, False),
    ([257, 100], 64, 2, 256, 32, 8, True),
    ([90, 31], 5, 1, 128, 64, 17, True),
    ([90, 31], 33, 1, 384, 16, 16, True),
    ([90, 31], 16, 2, 128, 0, 16, True),
    ([70, 9], 3, 2, 96, 24, 16, True),
    ([70, 9], 3, 1, 40, 7, 5, True),
    ([5000, 4097, 17, 9000], 16, 1, 512, 64, 16, True),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged_against_64_bits(torch, workspace, t, case):
    lens, heads, q_len, R, P, block, causal = PAGED[case]
    c = Paged(torch, t, lens, heads, q_len, R, P, block, seed=case)
    for ws in (workspace, None):
        c.o.fill_(float("nan"))
        c.run(causal, ws)
        c.check(torch, causal)
    status_is(0)


def test_paged_large_scores(torch, workspace):
    # Scores of a few hundred: the reference maximum rises many times, and
    # weights underflow.
    for t in ("bf16", "fp16"):
        c = Paged(torch, t, [900, 64, 1], 16, 2, 512, 64, 16, seed=3, scale=40.0)
        c.run(True, workspace)
        c.check(torch, True)
    # Rising by steps: every later key scores higher than the ones before.
    c = Paged(torch, "bf16", [1000], 16, 1, 128, 64, 16, seed=4)
    ramp = torch.linspace(-300, 300, 1000, device="cuda", dtype=torch.float64)
    ids = c.table[0].long()
    pos = torch.arange(1000, device="cuda")
    c.cache[ids[pos // 16], pos % 16, 128] = ramp.to(torch.bfloat16)
    c.ctx[0][:, 128] = ramp.to(torch.bfloat16).double()
    c.q[..., 128] = 8.0
    c.run(True, workspace)
    c.check(torch, True)


def test_paged_scales_of_any_sign(torch, workspace):
    for alpha in (-0.05, 0.0, 3.0):
        c = Paged(torch, "bf16", [130, 700], 16, 2, 512, 64, 16, seed=31)
        c.alpha = alpha
        c.run(True, workspace)
        c.check(torch, True)
        d = Packed(torch, "fp16", [140, 30], [300, 30], 2, 128, 64, 128, seed=32)
        d.alpha = alpha
        d.run(True)
        d.check(torch, True)


@pytest.mark.parametrize("dims", [(128, 64, 128), (130, 66, 70)])       # tensor cores; row kernel
def test_alpha_that_is_no_number(torch, workspace, dims):
    """A NaN alpha makes NaN of every row that has a key, and nothing of the others."""
    nan = float("nan")
    c = Packed(torch, "bf16", [100, 7, 3], [60, 0, 200], 2, *dims, seed=33)    # the first 40 rows see no key
    c.alpha = nan
    c.run(True)
    assert bool((c.o[:40] == 0).all()) and bool((c.o[100:107] == 0).all())
    assert bool(torch.isnan(c.o[40:100]).all()) and bool(torch.isnan(c.o[107:110]).all())
    R, P = (512, 64) if dims[0] == 128 else (40, 7)
    d = Paged(torch, "fp16", [2, 0, 70], 16, 3, R, P, 16, seed=34)
    d.alpha = nan
    for ws in (workspace, None):
        d.o.zero_()
        d.run(True, ws)
        assert bool((d.o[0, 0] == 0).all()) and bool((d.o[1] == 0).all())
        assert bool(torch.isnan(d.o[0, 1:]).all()) and bool(torch.isnan(d.o[2]).all())
    status_is(0)


def test_alpha_of_zero_weighs_huge_scores_alike(torch, workspace):
    for alpha in (0.0, -0.0):
        c = Packed(torch, "bf16", [140], [300], 2, 128, 64, 128, seed=35, scale=1e18)
        c.kn.mul_(1e18)                        # scores of 1e37 and more
        c.alpha = alpha
        c.run(True)
        for i in (0, 77, 139):
            v = c.v[: 161 + i].double()
            # Equal weights of 1, exact in the type: additions and one rounding.
            lim = (v.shape[0] + 8) * U * v.abs().mean(0) + 2 ** -18 * v.abs().mean(0) + HALF["bf16"] * v.mean(0).abs()
            assert_within(torch, c.o[i], v.mean(0), lim + 2.0 ** -25, f"row {i}")


def test_paged_smaller_workspaces(torch, workspace):
    """Fewer slots mean fewer CTAs, down to whole sequences: the same results
    within the bound."""
    c = Paged(torch, "bf16", [3000, 40, 700], 128, 1, 512, 64, 64, seed=33)
    for n in (0, 256, 1 << 14, 1 << 20, 5 << 20, workspace.numel()):
        c.o.fill_(float("nan"))
        c.run(True, workspace[:n] if n else None)
        c.check(torch, True)


def test_paged_more_row_groups_than_sms(torch, workspace):
    c = Paged(torch, "bf16", [200, 64], 64, 160, 128, 64, 16, seed=34)      # 160 groups of 64 rows
    c.run(True, workspace)
    c.check(torch, True)


def test_paged_offsets_past_32_bits(torch, workspace):
    """A cache of more than 2^31 elements, a sequence in its last pages; the page
    operations reach them too."""
    block, row = 64, 576
    blocks = (1 << 31) // (block * row) + 40
    c = Paged(torch, "bf16", [300], 16, 1, 512, 64, block, seed=35)
    cache = torch.empty(blocks, block, row, device="cuda", dtype=torch.bfloat16)
    old = c.table[0, :5].long()
    pairs = torch.stack([torch.arange(5, device="cuda"), torch.arange(blocks - 5, blocks, device="cuda")], 1).int()
    cache[:5] = c.cache[old]
    ws = torch.empty(sg.sbgemm_pages_workspace_bytes(blocks, 1, 8), device="cuda", dtype=torch.uint8)
    sg.pages_copy([cache], pairs, workspace=ws)
    cache[:5] = float("nan")
    c.table[0, :5] = pairs[:, 1]
    c.cache = cache
    c.run(True, workspace)
    c.check(torch, True)
    status_is(0)


def test_product_offsets_past_32_bits(torch):
    M, N, K = 70000, 32768, 16
    g = torch.Generator(device="cuda").manual_seed(36)
    A = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    B = torch.randn(K, N, generator=g, device="cuda").bfloat16()
    C = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    sg.matmul_half(A, B, C)
    for m in (0, 65535, 65536, M - 1):
        ref = A[m].double() @ B.double()
        size = A[m].double().abs() @ B.double().abs()
        assert_within(torch, C[m], ref, (K + 3) * U * size + HALF["bf16"] * ref.abs() + 2.0 ** -25, f"row {m}")


def test_paged_strided_operands(torch, workspace):
    for gap in (8, 3):      # 16-byte multiples, and a stride that no vector load can take
        c = Paged(torch, "bf16", [100, 333], 16, 2, 512, 64, 16, seed=9, gap=gap)
        q = torch.full((2, 16, 2, 576 + gap), float("nan"), device="cuda", dtype=torch.bfloat16)
        q[..., :576] = c.q.transpose(1, 2)
        c.q = q[..., :576].transpose(1, 2)                # heads outside tokens
        o = torch.full((2, 16, 2, 512 + gap), 7.0, device="cuda", dtype=torch.bfloat16)
        c.o = o[..., :512].transpose(1, 2)
        c.run(True, workspace)
        c.check(torch, True)
        assert bool((o[..., 512:] == 7.0).all())


def test_paged_bad_device_data_is_reported(torch, workspace):
    c = Paged(torch, "bf16", [200, 70], 16, 1, 512, 64, 16, seed=11)
    c.table[0, 3] = c.cache.shape[0]          # out of range: rows 48..63 of sequence 0 read as zeros
    c.run(True, workspace)
    c.ctx[0][48:64] = 0.0
    c.check(torch, True)
    status_is(10)
    status_is(0)
    c = Paged(torch, "bf16", [48, 32], 16, 1, 512, 64, 16, seed=11)
    c.seq_lens[0], c.seq_lens[1] = 49, -3     # clamped to max_len and to 0
    c.run(True, workspace, max_len=48)
    c.lens = [48, 0]
    c.ctx[1] = c.ctx[1][:0]
    c.check(torch, True)
    status_is(10)


def test_paged_lengths_default_to_max_len(torch, workspace):
    c = Paged(torch, "fp16", [96, 96], 16, 1, 512, 64, 16, seed=12)
    c.seq_lens = None
    c.run(False, workspace, max_len=96)
    c.check(torch, False)


def test_paged_repeats_and_replays(torch, workspace):
    c = Paged(torch, "bf16", [3000, 5, 900], 16, 1, 512, 64, 16, seed=13)
    first = c.run(True, workspace).clone()
    for _ in range(3):
        assert torch.equal(c.run(True, workspace), first)
    # Captured, with its own workspace; replayed after the inputs changed.
    ws = torch.empty_like(workspace)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        c.run(True, ws)
    c.o.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, first)
    c.q.mul_(0.5)
    c.seq_lens[0] = 2000
    c.lens[0], c.ctx[0] = 2000, c.ctx[0][:2000]
    graph.replay()
    torch.cuda.synchronize()
    c.check(torch, True)


def test_paged_two_streams_at_once(torch, workspace):
    a = Paged(torch, "bf16", [4000, 100], 16, 1, 512, 64, 16, seed=14)
    b = Paged(torch, "fp16", [50, 6000], 32, 1, 512, 64, 64, seed=15)
    other = torch.empty_like(workspace)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run(True, workspace)
        b.run(True, other, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    a.check(torch, True)
    b.check(torch, True)


def test_paged_many_sequences(torch, workspace):
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 400)]
    c = Paged(torch, "bf16", lens, 16, 1, 512, 64, 16, seed=16)
    c.run(True, workspace)
    c.check(torch, True)


PAIRS = [
    # lens, heads, q_len, R, P, block, causal: an even number of 64-row groups,
    # whose CTAs load the cache's blocks together
    ([0, 700, 1, 64, 65, 3000], 128, 1, 512, 64, 64, True),
    ([127, 128, 129, 0], 120, 1, 512, 64, 16, True),
    ([40, 260], 64, 4, 128, 64, 8, True),
    ([200, 3, 64], 64, 2, 384, 0, 128, True),
    ([5, 90, 1000], 70, 5, 256, 32, 32, False),
    ([130, 500], 128, 1, 512, 64, 20, True),
    ([1], 128, 1, 512, 64, 64, True),
    ([0], 128, 1, 512, 64, 64, True),
    ([20000], 128, 1, 512, 64, 64, True),
    ([64] * 300, 65, 1, 128, 64, 64, True),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(PAIRS)))
def test_paged_pairs_of_row_groups(torch, workspace, t, case):
    lens, heads, q_len, R, P, block, causal = PAIRS[case]
    c = Paged(torch, t, lens, heads, q_len, R, P, block, seed=40 + case)
    for ws in (workspace, None):
        c.o.fill_(float("nan"))
        first = c.run(causal, ws).clone()
        c.check(torch, causal)
        for _ in range(3):
            assert torch.equal(c.run(causal, ws), first)
    status_is(0)


def test_paged_pairs_replayed_beside_another_stream(torch, workspace):
    a = Paged(torch, "bf16", [4000, 100, 900], 128, 1, 512, 64, 64, seed=50)
    b = Paged(torch, "fp16", [50, 3000], 64, 4, 128, 64, 16, seed=51)
    first = a.run(True, workspace).clone()
    other = torch.empty_like(workspace)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        a.run(True, workspace)
    s2 = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        graph.replay()
        b.run(True, other, stream=s2.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a.o, first)
    a.check(torch, True)
    b.check(torch, True)
    status_is(0)


def test_paged_pairs_report_bad_device_data(torch, workspace):
    c = Paged(torch, "bf16", [200, 70], 128, 1, 512, 64, 16, seed=52)
    c.table[0, 3] = -1                        # rows 48..63 of sequence 0 read as zeros
    c.run(True, workspace)
    c.ctx[0][48:64] = 0.0
    c.check(torch, True)
    status_is(10)
    status_is(0)


# ---- latent attention, expanded form over packed sequences --------------------------

class Packed:
    def __init__(self, torch, t, q_lens, k_lens, heads, Dn, P, Dv, seed=0, front=0, back=2, gap=0, scale=1.0):
        dt = dtype_of(torch, t)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.t, self.q_lens, self.k_lens, self.dims = t, q_lens, k_lens, (heads, Dn, P, Dv)
        self.front = front
        nq, nk = front + sum(q_lens) + back, front + sum(k_lens) + back

        def rnd(n, *shape):
            x = torch.randn(n, *shape, generator=g, device="cuda")
            # Rows of no sequence hold NaN.
            x[:front], x[n - back:] = float("nan"), float("nan")
            return x
        kv = rnd(nk, heads, Dn + Dv + gap).to(dt)
        self.kn, self.v = kv[..., :Dn], kv[..., Dn: Dn + Dv]
        self.kr = rnd(nk, P).to(dt)
        self.q = (scale * rnd(nq, heads, Dn + P)).to(dt)
        self.whole = torch.full((nq, heads, Dv + gap), 7.0, device="cuda", dtype=dt)
        self.o = self.whole[..., :Dv]
        starts = lambda lens: torch.tensor(np.cumsum([front] + list(lens)), device="cuda", dtype=torch.int32)
        self.qs, self.ks = starts(q_lens), starts(k_lens)
        self.alpha = 1.0 / math.sqrt(Dn + P)

    def run(self, causal, **kw):
        return sg.latent_attention(self.q, self.kn, self.kr, self.v, self.o, self.qs, self.ks,
                                   kw.pop("max_q", max(self.q_lens + [1])), alpha=self.alpha, causal=causal, **kw)

    def check(self, torch, causal):
        heads, Dn, P, Dv = self.dims
        q0 = k0 = self.front
        mine = torch.zeros(self.whole.shape, dtype=torch.bool, device="cuda")
        for s, (m, n) in enumerate(zip(self.q_lens, self.k_lens)):
            if m:
                q = self.q[q0:q0 + m].double().transpose(0, 1)
                k = torch.cat([self.kn[k0:k0 + n].double(),
                               self.kr[k0:k0 + n].double()[:, None].expand(n, heads, P)], -1).transpose(0, 1)
                v = self.v[k0:k0 + n].double().transpose(0, 1)
                keep = torch.ones(m, n, device="cuda", dtype=torch.bool)
                if causal:
                    keep = keep.tril(n - m)
                O, W, Z, sv = attention_reference(q, k, v, self.alpha, keep)
                lim = attention_bound(self.t, Dn + P, n, O, W, Z, sv)
                assert_within(torch, self.o[q0:q0 + m].transpose(0, 1), O, lim, f"sequence {s}: {m} on {n}")
                mine[q0:q0 + m, :, :Dv] = True
            q0, k0 = q0 + m, k0 + n
        assert bool((self.whole[~mine] == 7.0).all()), "a row or column that belongs to no sequence was written"


PACKED = [
    # q_lens, k_lens, heads, Dn, P, Dv, causal
    ([1], [1], 1, 128, 64, 128, True),
    ([333], [333], 4, 128, 64, 128, True),
    ([1, 2, 127, 128, 129], [1, 2, 127, 128, 129], 3, 128, 64, 128, True),
    ([5, 0, 130], [300, 40, 131], 2, 128, 64, 128, True),
    ([257, 3], [400, 1000], 2, 128, 64, 128, False),
    ([100, 7], [60, 0], 2, 128, 64, 128, True),        # queries before the first key, and none at all
    ([40, 300], [0, 299], 2, 128, 64, 128, False),
    ([140, 20], [150, 20], 3, 64, 32, 64, True),
    ([140, 20], [150, 20], 3, 96, 32, 80, True),
    ([70, 300], [200, 300], 2, 128, 0, 128, True),
    ([70, 30], [200, 30], 2, 40, 8, 24, True),
    ([33, 30], [40, 30], 2, 130, 66, 70, True),        # no 16-byte rows
    ([600], [1500], 1, 128, 64, 128, True),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(PACKED)))
def test_packed_against_64_bits(torch, t, case):
    q_lens, k_lens, heads, Dn, P, Dv, causal = PACKED[case]
    c = Packed(torch, t, q_lens, k_lens, heads, Dn, P, Dv, seed=case, front=case % 3)
    c.run(causal)
    c.check(torch, causal)
    status_is(0)


ROPE_ONLY = [
    # q_lens, k_lens, heads, P, Dv, gap: sizes and alignments of the row kernel
    ([5, 33], [9, 40], 2, 66, 128, 0),                 # P past the tensor cores' 64
    ([7], [20], 1, 64, 136, 0),                        # Dv past their 128
    ([30, 3], [30, 50], 3, 64, 64, 3),                 # rows of V without alignment
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(ROPE_ONLY)))
def test_packed_rows_of_keys_without_a_nope_part(torch, t, case):
    """Dn == 0: keys of the shared part alone.  K_nope has no element and may be
    at any address, 0 included, which hides no key."""
    q_lens, k_lens, heads, P, Dv, gap = ROPE_ONLY[case]
    c = Packed(torch, t, q_lens, k_lens, heads, 0, P, Dv, seed=60 + case, gap=gap, scale=3.0)
    assert c.kn.data_ptr() == 0
    c.run(True)
    c.check(torch, True)
    c.whole.fill_(7.0)
    nq, nk, row = c.q.shape[0], c.v.shape[0], Dv + gap
    sg.sbgemm_latent_attention(sg.TYPE_BF16 if t == "bf16" else sg.TYPE_FP16, c.q.data_ptr(), P, heads * P, nq, 0, 0, 0,
                               c.kr.data_ptr(), P, c.v.data_ptr(), row, heads * row, nk, c.qs.data_ptr(),
                               c.ks.data_ptr(), len(q_lens), max(q_lens), c.o.data_ptr(), row, heads * row, heads, 0, P,
                               Dv, c.alpha, 1, torch.cuda.current_stream().cuda_stream)
    c.check(torch, True)
    status_is(0)


SHORT_BLOCKS = [
    # q_lens, k_lens, heads, Dn, P, Dv, causal: two or three pieces a block of keys
    # in the ring of eight, so that several blocks are under way at once
    ([300, 100], [20000, 9000], 2, 64, 0, 64, False),
    ([256], [30000], 1, 64, 0, 64, True),
    ([4000], [4000], 2, 64, 0, 64, True),
    ([1, 129, 700], [6000, 300, 1500], 3, 0, 64, 64, True),
    ([140], [140], 2, 0, 64, 128, True),
    ([300, 90], [3000, 700], 2, 32, 32, 128, False),
    ([130, 5], [130, 260], 1, 0, 16, 8, False),
]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("case", range(len(SHORT_BLOCKS)))
def test_packed_blocks_of_few_pieces(torch, t, case):
    q_lens, k_lens, heads, Dn, P, Dv, causal = SHORT_BLOCKS[case]
    c = Packed(torch, t, q_lens, k_lens, heads, Dn, P, Dv, seed=70 + case)
    first = c.run(causal).clone()
    c.check(torch, causal)
    for _ in range(20):
        assert torch.equal(c.run(causal), first)
    status_is(0)


def test_packed_large_scores_and_strides(torch):
    for gap in (8, 3):
        c = Packed(torch, "bf16", [200, 90], [333, 90], 2, 128, 64, 128, seed=21, gap=gap, scale=40.0)
        c.run(True)
        c.check(torch, True)
    c = Packed(torch, "fp16", [300], [900], 2, 128, 64, 128, seed=22)
    c.kr[:, 0] = torch.linspace(-300, 300, c.kr.shape[0], device="cuda").to(torch.float16)   # rises key by key
    c.q[..., 128] = 8.0
    c.run(True)
    c.check(torch, True)


def test_packed_infinities_of_other_sequences_stay_there(torch):
    c = Packed(torch, "bf16", [130, 50], [130, 50], 2, 128, 64, 128, seed=25)
    c.v[c.front + 130:] = float("inf")
    c.kn[c.front + 130:] = float("nan")
    c.run(True)
    assert bool(torch.isfinite(c.o[:130]).all())
    c.q_lens, c.k_lens = [130], [130]
    c.whole[130:] = 7.0
    c.check(torch, True)


def test_packed_without_any_key(torch):
    c = Packed(torch, "bf16", [20, 3], [0, 0], 2, 128, 64, 128, seed=26, back=0)
    c.run(False)
    c.check(torch, False)
    status_is(0)


def test_packed_starts_out_of_range_are_reported(torch):
    c = Packed(torch, "bf16", [20, 30], [20, 30], 2, 128, 64, 128, seed=23, back=0)
    c.ks[2] = 55                               # past total_k = 50: clamped
    c.run(True)
    c.check(torch, True)
    status_is(10)
    c = Packed(torch, "bf16", [20, 30], [20, 30], 2, 128, 64, 128, seed=23, back=0)
    c.run(True, max_q=25)                      # a sequence of 30: its last 5 rows are left
    assert bool((c.o[45:] == 7.0).all())
    status_is(10)


def test_packed_repeats_and_replays(torch):
    c = Packed(torch, "fp16", [300, 17], [700, 17], 4, 128, 64, 128, seed=24)
    first = c.run(True).clone()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        c.run(True)
    c.o.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, first)


# ---- pages -----------------------------------------------------------------------

class Model:
    """The pool's bookkeeping in Python; pages' contents by numpy."""

    def __init__(self, rng, blocks, block, seqs, max_blocks, lens, shapes):
        self.block, self.blocks = block, blocks
        self.refs = np.zeros(blocks, np.int32)
        self.table = np.full((seqs, max_blocks), -1, np.int32)
        self.lens = np.array(lens, np.int32)
        self.caches = [rng.standard_normal((blocks, block) + s).astype(np.float16) for s in shapes]
        order = list(rng.permutation(blocks))
        for s, n in enumerate(lens):
            for i in range(-(-n // block)):
                self.table[s, i] = order.pop()
                self.refs[self.table[s, i]] = 1

    def fresh(self):
        return int(np.flatnonzero(self.refs == 0)[0])

    def copy(self, pairs):
        ok = []
        inside = lambda x: 0 <= x < self.blocks
        dsts = [d for s, d in pairs if inside(s) and inside(d) and s != d]
        seen = set()
        for s, d in pairs:
            if not (inside(s) and inside(d)) or s == d:
                continue
            if d not in seen and s not in dsts:
                ok.append((s, d))
            seen.add(d)
        for c in self.caches:
            for s, d in ok:
                c[d] = c[s]

    def fork(self, parents, children):
        S, bs = len(self.lens), self.block
        lens, seen, left = self.lens.copy(), set(), int((self.refs == 0).sum())
        table = self.table.copy()
        stop = False
        for p, c in zip(parents, children):
            inside = 0 <= p < S and 0 <= c < S
            first = c not in seen
            seen.add(c)
            if not inside or not first or c in parents or lens[c] != 0:
                continue
            full, rest = divmod(int(lens[p]), bs)
            if stop or (rest > 0) > left:
                stop = True
                continue
            for i in range(full):
                self.table[c, i] = table[p, i]
                self.refs[table[p, i]] += 1
            if rest:
                page = self.fresh()
                left -= 1
                self.refs[page] = 1
                self.table[c, full] = page
                for x in self.caches:
                    x[page, :rest] = x[table[p, full], :rest]
            self.lens[c] = lens[p]

    def append(self, seqs, starts, rows):
        S, bs, total = len(self.lens), self.block, len(rows[0])
        seen, stop = set(), False
        if any(not 0 <= starts[k] <= starts[k + 1] <= total for k in range(len(seqs))):
            return
        for k, s in enumerate(seqs):
            first = s not in seen
            seen.add(s)
            n = starts[k + 1] - starts[k]
            if not 0 <= s < S or not first or self.lens[s] + n > self.table.shape[1] * bs:
                continue
            have = -(-int(self.lens[s]) // bs)
            if self.lens[s] % bs and n and self.refs[self.table[s, have - 1]] != 1:
                continue
            need = -(-int(self.lens[s] + n) // bs) - have
            if stop or need > (self.refs == 0).sum():
                stop = True
                continue
            for i in range(have, have + need):
                self.table[s, i] = self.fresh()
                self.refs[self.table[s, i]] = 1
            for j in range(n):
                at = int(self.lens[s]) + j
                for c, r in zip(self.caches, rows):
                    c[self.table[s, at // bs], at % bs] = r[starts[k] + j]
            self.lens[s] += n

    def free(self, seqs):
        for s in seqs:
            if 0 <= s < len(self.lens):
                for i in range(-(-int(self.lens[s]) // self.block)):
                    self.refs[self.table[s, i]] -= 1
                self.lens[s] = 0

    def compact(self):
        used = self.refs > 0
        U = int(used.sum())
        src = [i for i in range(U, self.blocks) if used[i]]
        dst = [i for i in range(U) if not used[i]]
        to = dict(zip(src, dst))
        for a, b in to.items():
            for c in self.caches:
                c[b] = c[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s, n in enumerate(self.lens):
            for i in range(-(-int(n) // self.block)):
                self.table[s, i] = to.get(int(self.table[s, i]), self.table[s, i])
        return len(src)


class Pool:
    """A Model and its copy on the GPU; every operation is made on both and compared."""

    def __init__(self, torch, rng, blocks, block, seqs, max_blocks, lens, shapes, n=64):
        self.torch = torch
        self.m = Model(rng, blocks, block, seqs, max_blocks, lens, shapes)
        dev = lambda x: torch.from_numpy(x.copy()).cuda()
        self.caches = [dev(c) for c in self.m.caches]
        self.refs, self.table, self.lens = dev(self.m.refs), dev(self.m.table), dev(self.m.lens)
        self.ws = torch.full((sg.sbgemm_pages_workspace_bytes(blocks, seqs, n),), 0xA5, dtype=torch.uint8,
                             device="cuda")

    def dev(self, x):
        return self.torch.tensor(np.asarray(x, np.int32), device="cuda", dtype=self.torch.int32)

    def all(self):
        return self.caches, self.refs, self.table, self.lens

    def same(self, code=0):
        for got, want in zip([self.refs, self.table, self.lens] + self.caches,
                             [self.m.refs, self.m.table, self.m.lens] + self.m.caches):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        status_is(code)

    def copy(self, pairs, code=0):
        self.m.copy(pairs)
        sg.pages_copy(self.caches, self.dev(pairs).view(-1, 2), workspace=self.ws)
        self.same(code)

    def fork(self, parents, children, code=0):
        self.m.fork(parents, children)
        sg.pages_fork(*self.all(), self.dev(parents), self.dev(children), workspace=self.ws)
        self.same(code)

    def append(self, rng, seqs, counts, code=0, starts=None):
        starts = [int(x) for x in np.cumsum([0] + list(counts))] if starts is None else starts
        total = sum(counts)
        rows = [rng.standard_normal((total,) + c.shape[2:]).astype(np.float16) for c in self.m.caches]
        self.m.append(seqs, starts, rows)
        sg.pages_append(*self.all(), self.dev(seqs), self.dev(starts),
                        [self.torch.from_numpy(r).cuda() for r in rows], workspace=self.ws)
        self.same(code)

    def free(self, seqs, code=0):
        self.m.free(seqs)
        sg.pages_free(*self.all(), self.dev(seqs))
        self.same(code)

    def compact(self):
        n = self.m.compact()
        moved = self.dev([-1])
        sg.pages_compact(*self.all(), workspace=self.ws, moved=moved)
        assert int(moved) == n
        self.same()


POOLS = [
    # blocks, block, seqs, max_blocks, longest, row shapes (fp16)
    (40, 4, 6, 8, 20, [(8,)]),
    (300, 16, 20, 12, 150, [(4, 32), (2, 8)]),
    (2500, 8, 40, 70, 300, [(72,), (8,), (16,)]),
    (64, 1, 9, 6, 6, [(64,)]),
    (5000, 32, 12, 40, 900, [(576,)]),
]


@pytest.mark.parametrize("case", range(len(POOLS)))
def test_pages_life(torch, case):
    """Random requests of every kind, valid ones only, on both sides."""
    blocks, block, seqs, max_blocks, longest, shapes = POOLS[case]
    rng = np.random.default_rng(case)
    lens = [int(x) for x in rng.integers(0, longest, seqs)]
    lens[0], lens[1], lens[2] = 0, block, 0
    p = Pool(torch, rng, blocks, block, seqs, max_blocks, lens, shapes)
    for _ in range(6):
        empty = [int(s) for s in np.flatnonzero(p.m.lens == 0)]
        full = [int(s) for s in np.flatnonzero(p.m.lens > 0)]
        kids = empty[: max(1, len(empty) // 2)]
        if kids and full and len(kids) <= (p.m.refs == 0).sum():
            p.fork([int(rng.choice(full)) for _ in kids], kids)
        room = [int(s) for s in range(seqs) if p.m.lens[s] + 2 * block + 3 <= max_blocks * block]
        rng.shuffle(room)
        room = room[: max(1, len(room) // 2)]
        counts = [int(rng.integers(0, 2 * block + 2)) for _ in room]
        if room and sum(counts) and sum(c // block + 2 for c in counts) <= (p.m.refs == 0).sum():
            p.append(rng, room, counts)
        gone = [int(s) for s in rng.permutation(seqs)[: max(1, seqs // 4)]]
        p.free(gone)
        p.compact()
        free = np.flatnonzero(p.m.refs == 0)
        used = np.flatnonzero(p.m.refs > 0)
        n = min(len(free), 5)
        if n and len(used):
            p.copy([(int(rng.choice(used)), int(d)) for d in rng.permutation(free)[:n]])


def test_pages_requests_that_are_not_valid(torch):
    rng = np.random.default_rng(7)
    p = Pool(torch, rng, 50, 4, 8, 6, [10, 0, 7, 0, 0, 4, 24, 0], [(8,)])
    # copy: out of range, the same destination twice, a source that is a destination, onto itself.
    free = [int(x) for x in np.flatnonzero(p.m.refs == 0)[:3]]
    a, b = int(p.m.table[0, 0]), int(p.m.table[2, 1])
    p.copy([(a, free[0]), (b, free[0]), (free[0], free[1]), (-1, free[2]), (a, 50), (b, b)], code=11)
    p.copy([(b, b)])
    # fork: out of range, onto a sequence in use, twice, onto a parent, from itself.
    p.fork([0, 2, 9, 0, 0, 6, 3], [1, 1, 3, -1, 2, 6, 4], code=11)
    p.fork([4, 1], [7, 7], code=11)
    # append: twice, out of range, too long; a shared unfinished page.
    p.append(rng, [0, 0, 8, 6, 5], [2, 3, 1, 1, 2], code=11)
    p.append(rng, [0, 2], [2, 1], code=11, starts=[2, 1, 3])
    p.append(rng, [0, 2], [2, 1], code=11, starts=[0, 2, 4])
    p.append(rng, [0, 2], [2, 1], code=11, starts=[-1, 2, 3])
    last = int(p.m.table[2, 1])
    p.m.refs[last], p.refs[last] = 2, 2
    p.append(rng, [2, 5], [1, 1], code=11)
    p.m.refs[last], p.refs[last] = 1, 1
    # free: out of range; twice is once.
    p.free([0, 0, -1, 8, 2], code=11)
    p.free([0, 5, 5])
    p.compact()


def test_pages_run_out_in_request_order(torch):
    rng = np.random.default_rng(8)
    p = Pool(torch, rng, 12, 4, 8, 6, [9, 6, 4, 0, 0, 0, 0, 0], [(8,)])   # 3 + 2 + 1 pages used, 6 free
    p.append(rng, [0, 1, 2], [3, 12, 16], code=12)     # 0, 3 and 4 pages: the last finds 3
    p.append(rng, [2, 0], [20, 1], code=12)            # the first one refused stops those behind it
    p.fork([1, 1, 2, 0], [3, 4, 5, 6])                 # 1, 1, 0 and 0 pages of 3
    p.free([5])
    p.fork([1, 1], [5, 7], code=12)                    # one page for two
    assert p.m.lens[5] == 18 and p.m.lens[7] == 0
    p.free([0, 1, 2, 3, 4, 5, 6])
    assert (p.m.refs == 0).all()
    p.compact()


def test_pages_of_a_large_pool_are_found(torch):
    # Free pages far behind: more than one round of the search, in the last segment.
    rng = np.random.default_rng(9)
    blocks = 40007
    p = Pool(torch, rng, blocks, 1, 4, 30000, [29000, 10990, 0, 0], [(8,)])
    p.append(rng, [2, 3], [11, 5])
    p.fork([2], [3], code=11)
    p.append(rng, [2], [1])
    p.free([0])
    p.compact()


def test_pages_with_thousands_of_requests(torch):
    """More requests than the planning CTA has threads, more sequences than its
    shared memory has claims for, more pairs and pages than the copy's; a prompt
    over a thousand pages in one request; invalid ones and the pool's end behind
    the first thousand."""
    rng = np.random.default_rng(15)
    blocks, block, seqs = 40007, 4, 5000
    lens = [int(x) for x in rng.integers(1, 9, seqs)]
    kids = [int(x) for x in rng.permutation(seqs)[:2600]]
    for s in kids:
        lens[s] = 0
    p = Pool(torch, rng, blocks, block, seqs, 1400, lens, [(8,)], n=10000)
    full = [s for s in range(seqs) if lens[s]]
    parents = [int(rng.choice(full)) for _ in kids]
    parents[2000], kids[2100] = seqs, kids[7]                  # out of range; an earlier request's child
    p.fork(parents, kids, code=11)
    who = [int(x) for x in rng.permutation(full)]
    p.append(rng, who, [5600 - 8 if i == 1500 else int(n) for i, n in enumerate(rng.integers(0, 6, len(who)))])
    free = [int(x) for x in np.flatnonzero(p.m.refs == 0)]
    used = np.flatnonzero(p.m.refs > 0)
    pairs = [(int(rng.choice(used)), int(d)) for d in rng.permutation(free)[:9000]]
    p.copy(pairs)
    pairs[8500] = (pairs[8500][0], pairs[3][1])                # a destination for the second time
    p.copy(pairs, code=11)
    left = int((p.m.refs == 0).sum())
    many = [s for s in range(seqs) if p.m.lens[s] < 40]
    p.append(rng, many, [4 * (left // 1700)] * len(many), code=12)
    p.free([int(x) for x in rng.permutation(seqs)[:3000]])
    p.compact()


def test_pages_replay(torch):
    rng = np.random.default_rng(10)
    p = Pool(torch, rng, 100, 4, 6, 10, [9, 6, 0, 0, 13, 0], [(8,), (16,)])
    seqs, starts = p.dev([0, 4]), p.dev([0, 1, 2])
    rows = [rng.standard_normal((2,) + c.shape[2:]).astype(np.float16) for c in p.m.caches]
    dev_rows = [torch.from_numpy(r).cuda() for r in rows]
    parents, children, gone = p.dev([0]), p.dev([2]), p.dev([2])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        sg.pages_append(*p.all(), seqs, starts, dev_rows, workspace=p.ws)
        sg.pages_fork(*p.all(), parents, children, workspace=p.ws)
        sg.pages_compact(*p.all(), workspace=p.ws)
        sg.pages_free(*p.all(), gone)
    for _ in range(3):
        graph.replay()
        p.m.append([0, 4], [0, 1, 2], rows)
        p.m.fork([0], [2])
        p.m.compact()
        p.m.free([2])
        torch.cuda.synchronize()
        p.same()


def test_pages_on_two_streams(torch):
    rng = np.random.default_rng(12)
    pools = [Pool(torch, rng, 200, 4, 8, 20, [9, 6, 0, 0, 13, 70, 1, 0], [(8,)]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in pools]
    rows = [rng.standard_normal((3, 8)).astype(np.float16) for _ in pools]
    dev = [torch.from_numpy(r).cuda() for r in rows]
    seqs, starts, parents, children = (pools[0].dev(x) for x in ([0, 4, 5], [0, 1, 2, 3], [5, 0], [2, 3]))
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s, d, r in zip(pools, streams, dev, rows):
            with torch.cuda.stream(s):
                sg.pages_append(*p.all(), seqs, starts, [d], workspace=p.ws)
                sg.pages_fork(*p.all(), parents, children, workspace=p.ws)
                sg.pages_free(*p.all(), children)
                sg.pages_compact(*p.all(), workspace=p.ws)
            p.m.append([0, 4, 5], [0, 1, 2, 3], [r])
            p.m.fork([5, 0], [2, 3])
            p.m.free([2, 3])
            p.m.compact()
    torch.cuda.synchronize()
    for p in pools:
        p.same()


def test_calls_through_ctypes_alone(torch, workspace, monkeypatch):
    """Without the fast-call module the same calls go through ctypes."""
    monkeypatch.setattr(sg, "_fast", None)
    check_product(torch, "bf16", 2, 33, 40, 64, "c", "r", "c")
    c = Paged(torch, "bf16", [70, 5], 16, 1, 512, 64, 16, seed=41)
    c.run(True, workspace)
    c.check(torch, True)
    d = Packed(torch, "fp16", [40], [70], 2, 128, 64, 128, seed=42)
    d.run(True)
    d.check(torch, True)
    test_pages_requests_that_are_not_valid(torch)
    test_pages_run_out_in_request_order(torch)


def test_pages_of_paged_attention_caches(torch):
    """The same operations keep an fp32 K / V cache of sbgemm_attention_paged: a
    fork attends like its parent, before and after a compaction."""
    g = torch.Generator(device="cuda").manual_seed(4)
    blocks, block, heads, D = 64, 16, 2, 64
    K, V = (torch.randn(blocks, block, heads, D, generator=g, device="cuda") for _ in range(2))
    refs = torch.zeros(blocks, device="cuda", dtype=torch.int32)
    table = torch.full((3, 8), -1, device="cuda", dtype=torch.int32)
    table[0, :5] = torch.tensor([9, 40, 3, 63, 17], dtype=torch.int32)
    refs[table[0, :5].long()] = 1
    lens = torch.tensor([70, 0, 0], device="cuda", dtype=torch.int32)
    ws = torch.empty(sg.sbgemm_pages_workspace_bytes(blocks, 3, 4), dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)
    q = torch.randn(heads, 1, D, generator=g, device="cuda")

    def attend(s):
        o = torch.empty(heads, 1, D, device="cuda")
        sg.sbgemm_attention_paged(q.data_ptr(), D, 1, D, K.data_ptr(), V.data_ptr(), blocks, block, heads,
                                  table[s].data_ptr(), 8, lens[s:].data_ptr(), o.data_ptr(), D, 1, D,
                                  1, 128, D, D, 1, 0.125, stream=torch.cuda.current_stream().cuda_stream)
        return o
    want = attend(0)
    sg.pages_fork([K, V], refs, table, lens, i32(0), i32(2), workspace=ws)
    assert torch.equal(attend(2), want)
    sg.pages_free([K, V], refs, table, lens, i32(0))
    sg.pages_compact([K, V], refs, table, lens, workspace=ws)
    assert torch.equal(attend(2), want)
    assert int(table[2, :5].max()) == 4 and int((refs > 0).sum()) == 5
    status_is(0)


# ---- a decode step of a latent-attention layer, as a server runs it ---------------------

@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_latent_layer_prompt_fork_decode(torch, workspace, t):
    """A prompt through the expanded form, its latents appended to the cache,
    forked, and decode steps through the absorbed form (products, cache, split
    attention), all in one captured graph; each output against the layer's
    definition in 64 bits on the same 16-bit inputs."""
    dt = dtype_of(torch, t)
    g = torch.Generator(device="cuda").manual_seed(17)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    H, Dn, P, R, Dv, block, blocks, T = 4, 128, 64, 512, 128, 16, 64, 150
    W = (rnd(H, Dn + Dv, R) / math.sqrt(R)).to(dt)             # W_uk rows, then W_uv rows, a head
    w_uk, w_uv = W[:, :Dn], W[:, Dn:]
    alpha = 1.0 / math.sqrt(Dn + P)
    latent = rnd(T + 8, R + P).to(dt)                          # [c | k_rope] of the prompt and later tokens
    queries = rnd(T + 8, H, Dn + P).to(dt)
    # The prompt: expand, attend.
    kv = torch.empty(T, H, Dn + Dv, device="cuda", dtype=dt)
    sg.matmul_half(latent[:T, :R], W.view(H * (Dn + Dv), R).t(), kv.view(T, -1))
    out = torch.empty(T, H, Dv, device="cuda", dtype=dt)
    i32 = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)
    sg.latent_attention(queries[:T], kv[..., :Dn], latent[:T, R:], kv[..., Dn:], out, i32(0, T), i32(0, T), T,
                        alpha=alpha)
    # The cache: append the prompt, fork it, then a token each.
    cache = torch.full((blocks, block, R + P), float("nan"), device="cuda").to(dt)
    refs = torch.zeros(blocks, device="cuda", dtype=torch.int32)
    table = torch.full((2, 20), -1, device="cuda", dtype=torch.int32)
    lens = torch.zeros(2, device="cuda", dtype=torch.int32)
    ws = torch.empty(sg.sbgemm_pages_workspace_bytes(blocks, 2, 2), dtype=torch.uint8, device="cuda")
    pool = ([cache], refs, table, lens)
    sg.pages_append(*pool, i32(0), i32(0, T), [latent[:T]], workspace=ws)
    sg.pages_fork(*pool, i32(0), i32(1), workspace=ws)
    step = {"row": torch.empty(2, R + P, device="cuda", dtype=dt), "seqs": i32(0, 1), "starts": i32(0, 1, 2),
            "q": torch.empty(2, 1, H, Dn + P, device="cuda", dtype=dt),
            "ql": torch.empty(2, 1, H, R + P, device="cuda", dtype=dt),
            "ol": torch.empty(2, 1, H, R, device="cuda", dtype=dt),
            "o": torch.empty(2, 1, H, Dv, device="cuda", dtype=dt)}

    def decode():
        sg.pages_append(*pool, step["seqs"], step["starts"], [step["row"]], workspace=ws)
        head = lambda x: x.view(2, H, -1).transpose(0, 1)
        sg.matmul_half(head(step["q"])[..., :Dn], w_uk, head(step["ql"])[..., :R])
        step["ql"][..., R:] = step["q"][..., Dn:]
        sg.latent_attention_paged(step["ql"], cache, table, lens, step["ol"], alpha=alpha, workspace=workspace)
        sg.matmul_half(head(step["ol"]), w_uv.transpose(1, 2), head(step["o"]))

    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        decode()
    seen = [[latent[:T]], [latent[:T]]]
    uk, uv = w_uk.double(), w_uv.double()

    def layer(q, rows):
        """One query token [H, Dn + P] over rows [n, R + P] in 64 bits, and six
        standard deviations of the 16-bit roundings on the way, each at most h
        of its term and independent of the others: of keys or absorbed query
        (which move a weight by as much as its score), of weights and values
        (n terms p v), of the averaged c (R terms w_uv c) and of the output."""
        c, kr = rows[:, :R].double(), rows[:, R:].double()
        k = torch.cat([torch.einsum("hdr,nr->hnd", uk, c), kr.expand(H, -1, -1)], -1)
        v = torch.einsum("her,nr->hne", uv, c)
        q = q.double()
        ql = torch.cat([torch.einsum("hd,hdr->hr", q[:, :Dn], uk), q[:, Dn:]], -1)
        p = torch.softmax(alpha * torch.einsum("hd,hnd->hn", q, k), -1)
        o = torch.einsum("hn,hne->he", p, v)
        moves = alpha * max(float((q[:, None] * k).norm(dim=-1).max()),
                            float((ql[:, None] * rows.double()).norm(dim=-1).max()))
        averaged = (uv * torch.einsum("hn,nr->hr", p, c)[:, None]).norm(dim=-1)
        spread = (p[..., None] * v).norm(dim=1)
        return o, 6 * HALF[t] * ((2 + moves) * float(spread.max()) + float(averaged.max()) + float(o.abs().max()))

    for i in (0, 1, 77, T - 1):
        want, lim = layer(queries[i], latent[: i + 1])
        assert float((out[i].double() - want).abs().max()) <= lim
    for n in range(4):
        rows = latent[T + 2 * n: T + 2 * n + 2]
        step["row"].copy_(rows)
        step["q"].copy_(queries[T + 2 * n: T + 2 * n + 2].unsqueeze(1))
        graph.replay()
        for s in range(2):
            seen[s].append(rows[s:s + 1])
            want, lim = layer(step["q"][s, 0], torch.cat(seen[s]))
            assert float((step["o"][s, 0].double() - want).abs().max()) <= lim
    assert [int(x) for x in lens] == [T + 4, T + 4]
    sg.pages_free(*pool, i32(0))
    sg.pages_compact(*pool, workspace=ws)
    before = step["ol"][1].clone()
    sg.latent_attention_paged(step["ql"][1:], cache, table[1:], lens[1:], step["ol"][1:], alpha=alpha, workspace=None)
    c64 = torch.cat(seen[1]).double()
    q = step["ql"][1].double().transpose(0, 1)
    O, Wt, Z, sv = attention_reference(q, c64, c64[:, :R], alpha, torch.ones(1, len(c64), device="cuda", dtype=torch.bool))
    lim = attention_bound(t, R + P, len(c64), O, Wt, Z, sv)
    assert_within(torch, step["ol"][1].transpose(0, 1), O, lim)
    assert_within(torch, before.transpose(0, 1), O, lim)
    status_is(0)


# ---- the status words -------------------------------------------------------------------

def test_status_of_several_kernels_is_read_at_once(torch, workspace):
    """A code of each kernel file, pending together: one is reported, all are
    cleared, and the next call reports what came since."""
    rng = np.random.default_rng(14)
    p = Pool(torch, rng, 20, 4, 4, 6, [9, 0, 0, 0], [(8,)])
    c = Paged(torch, "bf16", [40, 20], 16, 1, 512, 64, 16, seed=80)
    c.seq_lens[1] = -1
    d = Packed(torch, "bf16", [20], [20], 2, 128, 64, 128, seed=81, back=0)
    d.ks[1] = 25
    e = Packed(torch, "bf16", [20], [20], 2, 130, 66, 70, seed=82, back=0)
    e.ks[1] = 25
    for codes, calls in ((10, (lambda: c.run(True, workspace), lambda: d.run(True), lambda: e.run(True))),
                         (11, (lambda: sg.pages_free(*p.all(), p.dev([-1])),))):
        for f in calls:
            f()
        sg.sbgemm_selftest(sg.SELFTEST_FLAG, 1000)
        st, where = sg.sbgemm_device_status()            # the self-test's word comes first
        assert (st, where) == (sg.SBGEMM_ERR_DEVICE_TIMEOUT, 8)
        status_is(0)
        for f in calls:
            f()
            status_is(codes)
            status_is(0)


def test_status_costs_a_launch_and_a_copy(torch):
    """Reading the status is one launch, one copy and a wait, not one of each for
    every kernel file: within eight times a copy of one number to the host (it
    was 22 times with a read a file)."""
    import time
    x = torch.zeros(1, device="cuda")

    def median(f):
        times = []
        for _ in range(200):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return sorted(times)[100]
    for f in (sg.sbgemm_device_status, x.item):
        median(f)
    status, copy = median(sg.sbgemm_device_status), median(x.item)
    print(f"status {status * 1e6:.1f} us, copy {copy * 1e6:.1f} us")
    assert status < 8 * copy
