"""Cases of the operators around a latent-attention layer's products: products
of 8-bit floats with a scale for each block of 128 and the quantisation that
feeds them, norms of queries, keys and latents with the rotation of their
positions in one pass (and its gradient), and latent attention for a batch
whose sequences share long prefixes.

Every case has a plain form in elementary torch operations (fp32, the angles of
positions in 64 bits, rounded once at the end) and the call of the library.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_E4M3 = torch.float8_e4m3fn
_SMALLEST = 2.0 ** -126          # the least scale: fp32's smallest normal number


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # A decode step's projection: few tokens against weights kept in 8 bits, bound by their bytes.
        dict(name="linear of 16 tokens", kind="linear", type="bf16", M=16, N=7168, K=4096),
        # The same layer over the packed prompts of a batch.
        dict(name="linear of 4099 tokens", kind="linear", type="bf16", M=4099, N=7168, K=4096),
        # Training: a weight's gradient contracts over the tokens, both operands quantised along them.
        dict(name="weight gradient over 8190 tokens", kind="weight_grad", type="bf16", T=8190, N=2560, K=960),
        # Weights quantised once an optimiser step, 128 x 128 elements a scale.
        dict(name="quantise weights", kind="quantise", type="fp16", M=7100, K=4096, rows=128),
        # A decode step of latent attention: the rope part of the queries is rotated, the new row
        # of the cache is its normed latent and the rotated part shared by the heads.
        dict(name="rotate 32 tokens' latents", kind="rope", type="bf16", tokens=32, rope=64, interleaved=True,
             longest=131072, factor=32.0, parts="16 192 0 128, 1 576 512 512"),
        # A prompt's queries and keys out of one packed projection, normed for each head.
        dict(name="norm and rotate a prompt", kind="rope", type="bf16", tokens=8192, rope=128, interleaved=False,
             longest=8192, factor=1.0, parts="32 128 128 0, 8 128 128 0"),
        # Training in fp32, part of each head rotated, no norm.
        dict(name="rotate part of fp32 heads", kind="rope", type="fp32", tokens=4099, rope=32, interleaved=True,
             longest=1000000, factor=1.0, parts="15 64 0 0, 5 64 0 0"),
        # The gradient of normed and rotated queries and keys, with that of the norms' weights.
        dict(name="gradient over 4096 tokens", kind="rope_grad", type="bf16", tokens=4096, rope=128,
             interleaved=False, longest=4096, factor=4.0, parts="32 128 128 0, 8 128 128 0"),
        # The same for a short ragged batch of latents.
        dict(name="gradient over 333 tokens' latents", kind="rope_grad", type="fp32", tokens=333, rope=64,
             interleaved=True, longest=4096, factor=1.0, parts="16 192 0 128, 1 576 512 512"),
        # A few samples of one prompt: forks of a sequence that share its pages.
        dict(name="4 samples of 1500 keys", kind="shared", type="bf16", groups=1, each=4, q_len=1, heads=16,
             prefix=1500, own=200, block=64, rank=512, rope=64),
        # A served batch behind one long system prompt.
        dict(name="64 sequences behind 16001 keys", kind="shared", type="bf16", groups=1, each=64, q_len=1,
             heads=16, prefix=16001, own=1000, block=64, rank=512, rope=64),
        # Several documents, each asked many questions, all heads on one GPU.
        dict(name="4 documents of 16 questions", kind="shared", type="fp16", groups=4, each=16, q_len=1,
             heads=128, prefix=8192, own=700, block=16, rank=512, rope=64),
    ]


def _parts(case):
    """(heads, elements a head, normed ones from the first, first rotated one) of each part."""
    return [tuple(int(n) for n in p.split()) for p in case["parts"].split(",")]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["linear", "linear", "weight_grad", "quantise", "rope", "rope", "rope_grad", "rope_grad",
                       "shared", "shared", "shared"])
    c = dict(kind=kind, type=rng.choice(["bf16", "fp16"]))
    if kind == "linear":
        c["M"] = _log(rng, 1, 4096)
        c["N"] = _log(rng, 64, 8192)
        c["K"] = 16 * _log(rng, 4, 448)
        while c["M"] * c["N"] * c["K"] > 1.2e11:
            c["N"] = c["N"] * 3 // 4
    elif kind == "weight_grad":
        c["T"] = _log(rng, 1, 8192)
        c["N"] = _log(rng, 64, 4096)
        c["K"] = _log(rng, 64, 4096)
    elif kind == "quantise":
        c["type"] = rng.choice(["bf16", "fp16", "fp32"])
        c["M"] = _log(rng, 1, 8192)
        c["K"] = _log(rng, 16, 4096)
        c["rows"] = rng.choice([1, 128])
    elif kind == "shared":
        c["groups"] = rng.choice([1, 1, 2, 3, 5])
        c["each"] = _log(rng, 1, 48)
        c["heads"] = rng.choice([1, 4, 8, 16, 16, 20, 32, 64, 128])
        c["q_len"] = rng.choice([1, 1, 1, 2, 3]) if c["heads"] <= 32 else 1
        c["prefix"] = _log(rng, 1, 16384)
        c["own"] = max(c["q_len"], _log(rng, 1, 1500))
        c["block"] = rng.choice([8, 16, 24, 32, 64, 128])
        c["rank"], c["rope"] = rng.choice([(512, 64), (512, 64), (256, 32), (128, 64)])
        # Bounded by the largest listed case's rows x keys and the plain form's gathered keys.
        while (c["groups"] * c["each"] * c["heads"] * c["q_len"] * (c["prefix"] + c["own"]) > 7.0e7 or
               c["groups"] * c["each"] * (c["prefix"] + c["own"]) > 1.1e6):
            c["prefix"] = (c["prefix"] * 3 + 3) // 4
            c["own"] = max(c["q_len"], c["own"] * 3 // 4)
            c["each"] = max(1, c["each"] * 7 // 8)
    else:
        c["type"] = rng.choice(["bf16", "fp16", "fp32"])
        c["tokens"] = _log(rng, 1, 8192)
        c["interleaved"] = rng.random() < 0.5
        c["longest"] = _log(rng, 1024, 1000000)
        c["factor"] = rng.choice([1.0, 1.0, 4.0, 32.0])
        form = rng.choice(["qk", "qk", "plain", "latent"])
        if form == "latent":
            rank, nope, c["rope"] = rng.choice([(512, 128, 64), (256, 64, 32), (128, 96, 64)])
            c["parts"] = f"{_log(rng, 1, 32)} {nope + c['rope']} 0 {nope}, 1 {rank + c['rope']} {rank} {rank}"
        else:
            dim = rng.choice([32, 64, 80, 96, 128, 128, 192, 256])
            c["rope"] = rng.choice([dim, dim, dim // 2, 16])
            start = rng.choice([0, dim - c["rope"]])
            norm = dim if form == "qk" else 0
            kv = _log(rng, 1, 8)
            c["parts"] = f"{kv * _log(rng, 1, 8)} {dim} {norm} {start}, {kv} {dim} {norm} {start}"
        most = 4.3e7 if kind == "rope" else 2.2e7
        while c["tokens"] * sum(h * d for h, d, _, _ in _parts(c)) > most:
            c["tokens"] = c["tokens"] * 3 // 4
    return c


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _padded(rows, cols, multiple, dtype):
    """An uninitialised [rows, cols] whose rows start at multiples of `multiple` elements."""
    wide = -(-cols // multiple) * multiple
    return torch.empty(rows, wide, device="cuda", dtype=dtype)[:, :cols]


def _spread(n, longest, least):
    """n lengths evenly over the upper three quarters of `longest`, `least` at least."""
    return [max(least, longest - (3 * longest * i) // (4 * n)) for i in range(n)]


def prepare(case, seed):
    g = _gen(seed)
    c, t = case, _TYPES[case["type"]]
    s = {"case": dict(case)}
    if c["kind"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        # Activations with a few large channels; weights in 8 bits already.
        s["x"] = (_randn(g, M, K, dtype=torch.float32) * torch.exp(torch.randn(K, generator=g, device="cuda"))).to(t)
        s["w"], s["w_scale"] = _plain_quantise(_randn(g, N, K, dtype=torch.float32) / math.sqrt(K), 128)
        s["x8"] = torch.empty(M, K, device="cuda", dtype=_E4M3)
        s["x_scale"] = torch.empty(M, -(-K // 128), device="cuda")
        s["y"] = torch.empty(M, N, device="cuda", dtype=t)
    elif c["kind"] == "weight_grad":
        T, N, K = c["T"], c["N"], c["K"]
        s["x"] = _randn(g, T, K, dtype=t)
        s["dy"] = (_randn(g, T, N, dtype=torch.float32) * 1e-3).to(t)
        s["x8"], s["dy8"] = _padded(K, T, 16, _E4M3), _padded(N, T, 16, _E4M3)
        s["x_scale"] = torch.empty(K, -(-T // 128), device="cuda")
        s["dy_scale"] = torch.empty(N, -(-T // 128), device="cuda")
        s["dw"] = torch.empty(N, K, device="cuda", dtype=t)
    elif c["kind"] == "quantise":
        M, K = c["M"], c["K"]
        s["x"] = (_randn(g, M, K, dtype=torch.float32) * 0.02).to(t)
        s["x8"] = _padded(M, K, 16, _E4M3)
        s["x_scale"] = torch.empty(-(-M // c["rows"]), -(-K // 128), device="cuda")
    elif c["kind"] in ("rope", "rope_grad"):
        T, P = c["tokens"], c["rope"]
        s["positions"] = torch.randint(0, c["longest"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["frequencies"], s["magnitude"] = _frequencies(P, c["factor"])
        # The parts lie side by side, as one projection leaves them.
        packed = _randn(g, T, sum(h * d for h, d, _, _ in _parts(c)), dtype=t)
        s["x"], s["y"], s["weight"], at = [], [], [], 0
        s["dy"], s["dx"], s["dweight"] = [], [], []
        for h, d, norm, _ in _parts(c):
            s["x"].append(packed[:, at:at + h * d].unflatten(1, (h, d)))
            at += h * d
            s["weight"].append((1 + 0.1 * _randn(g, norm, dtype=torch.float32)).to(t) if norm else None)
            if c["kind"] == "rope":
                s["y"].append(torch.empty(T, h, d, device="cuda", dtype=t))
            else:
                s["dy"].append(_randn(g, T, h, d, dtype=t))
                s["dx"].append(torch.empty(T, h, d, device="cuda", dtype=t))
                s["dweight"].append(torch.empty(norm, device="cuda") if norm else None)
        if own:
            import strided_gemm_gb300 as sg
            s["table"] = sg.rope_table(P, base=10000.0, factor=c["factor"], original=4096)
            if c["kind"] == "rope":
                s["parts"] = [sg.RopePart(x, y, norm=p[2], weight=w, start=p[3])
                              for x, y, w, p in zip(s["x"], s["y"], s["weight"], _parts(c))]
            else:
                s["parts"] = [sg.RopeGrad(x, dy, dx, norm=p[2], weight=w, dweight=dw, start=p[3])
                              for x, dy, dx, w, dw, p in zip(s["x"], s["dy"], s["dx"], s["weight"], s["dweight"],
                                                             _parts(c))]
                s["workspace"] = torch.empty(sg.sbgemm_norm_rope_workspace_bytes([p[2] for p in _parts(c)]),
                                             device="cuda", dtype=torch.uint8)
    else:
        S, T, H, wide = c["groups"] * c["each"], c["q_len"], c["heads"], c["rank"] + c["rope"]
        B, full = c["block"], c["prefix"] // c["block"]
        tails = torch.tensor(_spread(S, c["own"], T), device="cuda", dtype=torch.int32)
        s["lens"] = c["prefix"] + tails[torch.randperm(S, generator=g, device="cuda")]
        s["starts"] = torch.arange(0, S + 1, c["each"], device="cuda", dtype=torch.int32)
        s["prefix"] = torch.full((c["groups"],), c["prefix"], device="cuda", dtype=torch.int32)
        # As forks leave them: full pages of the prefix shared, the rest each sequence's own.
        most = -(-(c["prefix"] + c["own"]) // B)
        blocks = c["groups"] * full + S * (most - full) + 3
        pages = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        table = torch.empty(S, most, device="cuda", dtype=torch.int32)
        table[:, :full] = pages[: c["groups"] * full].view(c["groups"], 1, full).expand(-1, c["each"], -1).reshape(S, full)
        table[:, full:] = pages[c["groups"] * full: blocks - 3].view(S, most - full)
        used = (s["lens"].long() + B - 1) // B
        table[torch.arange(most, device="cuda")[None, :] >= used[:, None]] = -1
        s["table"] = table
        s["cache"] = _randn(g, blocks, B, wide, dtype=t)
        s["q"] = _randn(g, S, T, H, wide, dtype=t)
        s["o"] = torch.empty(S, T, H, c["rank"], device="cuda", dtype=t)
        s["alpha"] = 1.0 / math.sqrt(128 + c["rope"])
        if own:
            import strided_gemm_gb300 as sg
            s["workspace"] = torch.empty(sg.sbgemm_latent_shared_workspace_bytes(S, c["groups"], T, H, c["rank"]),
                                         device="cuda", dtype=torch.uint8)
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["kind"]](s)


def _own_linear(s):
    import strided_gemm_gb300 as sg
    sg.quantize_fp8(s["x"], s["x8"], s["x_scale"])
    return sg.matmul_fp8(s["x8"], s["x_scale"], s["w"].t(), s["w_scale"].t(), s["y"])


def _own_weight_grad(s):
    import strided_gemm_gb300 as sg
    sg.quantize_fp8(s["dy"].t(), s["dy8"], s["dy_scale"])
    sg.quantize_fp8(s["x"].t(), s["x8"], s["x_scale"])
    return sg.matmul_fp8(s["dy8"], s["dy_scale"], s["x8"].t(), s["x_scale"].t(), s["dw"])


def _own_quantise(s):
    import strided_gemm_gb300 as sg
    sg.quantize_fp8(s["x"], s["x8"], s["x_scale"])
    return s["x8"].to(torch.bfloat16), s["x_scale"]


def _own_rope(s):
    import strided_gemm_gb300 as sg
    sg.norm_rope(s["parts"], s["positions"], s["table"], interleaved=s["case"]["interleaved"])
    return s["y"]


def _own_rope_grad(s):
    import strided_gemm_gb300 as sg
    sg.norm_rope_backward(s["parts"], s["positions"], s["table"], interleaved=s["case"]["interleaved"],
                          workspace=s["workspace"])
    return s["dx"] + [w for w in s["dweight"] if w is not None]


def _own_shared(s):
    import strided_gemm_gb300 as sg
    return sg.latent_attention_shared(s["q"], s["cache"], s["table"], s["lens"], s["starts"], s["prefix"], s["o"],
                                      alpha=s["alpha"], causal=True, workspace=s["workspace"])


_own = {"linear": _own_linear, "weight_grad": _own_weight_grad, "quantise": _own_quantise, "rope": _own_rope,
        "rope_grad": _own_rope_grad, "shared": _own_shared}


def _blocks(x, rows):
    """x [M, K] in fp32, padded with zeros to [m, rows, k, 128]."""
    M, K = x.shape
    m, k = -(-M // rows), -(-K // 128)
    if m * rows == M and k * 128 == K:
        return x.float().reshape(m, rows, k, 128)
    full = torch.zeros(m * rows, k * 128, device=x.device)
    full[:M, :K] = x
    return full.view(m, rows, k, 128)


def _plain_quantise(x, rows):
    """x in e4m3 with a scale for each `rows` x 128 elements: the largest magnitude
    becomes 448.  Both quotients are rounded to fp32 (in 64 bits first: a division
    by a number is a product with its reciprocal else): x / scale is a tie of
    e4m3 wherever 7 divides the block's largest magnitude."""
    M, K = x.shape
    b = _blocks(x, rows)
    scale = (b.abs().amax((1, 3)).double() / 448.0).float().clamp_min(_SMALLEST)
    q = (b / scale[:, None, :, None]).to(_E4M3)
    return q.reshape(-1, b.shape[2] * 128)[:M, :K].contiguous(), scale


def _plain_values(q, scale, rows):
    """The numbers that a quantised [M, K] stands for, in fp32."""
    return (_blocks(q, rows) * scale[:, None, :, None]).reshape(-1, scale.shape[1] * 128)[: q.shape[0], : q.shape[1]]


def _plain_linear(s):
    s["x8"], s["x_scale"] = _plain_quantise(s["x"], 1)
    s["y"].copy_(_plain_values(s["x8"], s["x_scale"], 1) @ _plain_values(s["w"], s["w_scale"], 128).t())
    return s["y"]


def _plain_weight_grad(s):
    s["dy8"], s["dy_scale"] = _plain_quantise(s["dy"].t(), 1)
    s["x8"], s["x_scale"] = _plain_quantise(s["x"].t(), 1)
    s["dw"].copy_(_plain_values(s["dy8"], s["dy_scale"], 1) @ _plain_values(s["x8"], s["x_scale"], 1).t())
    return s["dw"]


def _plain_quantise_case(s):
    s["x8"], s["x_scale"] = _plain_quantise(s["x"], s["case"]["rows"])
    return s["x8"].to(torch.bfloat16), s["x_scale"]


def _frequencies(dims, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Radians a position for each pair, in 64 bits, and the factor of cosine and
    sine: positions beyond `original` are reached by slowing those pairs down
    that turn less than `slow` times in it, by a ramp up to `fast` turns."""
    i = torch.arange(dims // 2, device="cuda", dtype=torch.float64)
    f = base ** (-2.0 * i / dims)
    if factor == 1.0:
        return f, 1.0

    def pair(turns):
        return dims * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), dims - 1)
    ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _pairs(x, start, dims, interleaved):
    """The two members of each rotated pair, as views."""
    z = x[..., start:start + dims]
    return (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., : dims // 2], z[..., dims // 2:])


def _cos_sin(s):
    a = s["positions"].double()[:, None, None] * s["frequencies"]
    return (a.cos() * s["magnitude"]).float(), (a.sin() * s["magnitude"]).float()


_EPS = 1e-6


def _plain_rope(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    for (h, d, norm, start), x, y, w in zip(_parts(c), s["x"], s["y"], s["weight"]):
        z = x.float()
        if norm:
            z = z.clone()
            n = z[..., :norm]
            z[..., :norm] = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + _EPS) * w.float()
        out = z.clone()
        a, b = _pairs(z, start, c["rope"], c["interleaved"])
        u, v = _pairs(out, start, c["rope"], c["interleaved"])
        u.copy_(a * cos - b * sin)
        v.copy_(a * sin + b * cos)
        y.copy_(out)
    return s["y"]


def _plain_rope_grad(s):
    c = s["case"]
    cos, sin = _cos_sin(s)
    for (h, d, norm, start), x, dy, dx, w, dw in zip(_parts(c), s["x"], s["dy"], s["dx"], s["weight"], s["dweight"]):
        g = dy.float()
        out = g.clone()
        a, b = _pairs(g, start, c["rope"], c["interleaved"])
        u, v = _pairs(out, start, c["rope"], c["interleaved"])
        u.copy_(a * cos + b * sin)
        v.copy_(b * cos - a * sin)
        if norm:
            n = x.float()[..., :norm]
            r = torch.rsqrt((n * n).mean(-1, keepdim=True) + _EPS)
            n = n * r
            dw.copy_((out[..., :norm] * n).sum((0, 1), dtype=torch.float64))
            dn = out[..., :norm] * w.float()
            out[..., :norm] = (dn - n * (dn * n).mean(-1, keepdim=True)) * r
        dx.copy_(out)
    return s["dx"] + [w for w in s["dweight"] if w is not None]


def _softmax(x):
    """Softmax over the last axis, in place; zeros where everything is masked (-inf)."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _plain_shared(s):
    c = s["case"]
    S, T, H, N = c["groups"] * c["each"], c["q_len"], c["heads"], c["prefix"] + c["own"]
    n = torch.arange(N, device="cuda")
    here = n[None, :] < s["lens"][:, None]
    page = s["table"].long()[:, n // c["block"]]
    # The prefix is read where the group's first sequence has it.
    group = torch.searchsorted(s["starts"].long(), torch.arange(S, device="cuda"), right=True) - 1
    first = s["starts"].long()[group]
    page = torch.where(n[None, :] < s["prefix"][group][:, None], page[first], page).clamp_min(0)
    kv = s["cache"][page, n % c["block"]].float() * here[..., None]
    x = torch.bmm(s["q"].float().reshape(S, T * H, -1), kv.transpose(1, 2)).mul_(s["alpha"]).view(S, T, H, N)
    last = s["lens"][:, None] - T + torch.arange(T, device="cuda")[None, :]
    x.masked_fill_((n[None, None, :] > last[..., None])[:, :, None, :], -math.inf)
    p = _softmax(x).view(S, T * H, N)
    s["o"].copy_(torch.bmm(p, kv[..., : c["rank"]]).view(S, T, H, c["rank"]))
    return s["o"]


_plain = {"linear": _plain_linear, "weight_grad": _plain_weight_grad, "quantise": _plain_quantise_case,
          "rope": _plain_rope, "rope_grad": _plain_rope_grad, "shared": _plain_shared}


# ---- the work of one pass ------------------------------------------------------

def work(case):
    c, e = case, torch.finfo(_TYPES[case["type"]]).bits // 8
    if c["kind"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": e * M * (K + N) + N * K + 4 * -(-N // 128) * -(-K // 128), "flops": 2.0 * M * N * K}
    if c["kind"] == "weight_grad":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": e * (T * (N + K) + N * K), "flops": 2.0 * T * N * K}
    if c["kind"] == "quantise":
        # The values come back as bf16.
        return {"bytes": (e + 2) * c["M"] * c["K"] + 4 * -(-c["M"] // c["rows"]) * -(-c["K"] // 128),
                "flops": 2.0 * c["M"] * c["K"]}
    if c["kind"] in ("rope", "rope_grad"):
        n = c["tokens"] * sum(h * d for h, d, _, _ in _parts(c))
        weights = sum(norm for _, _, norm, _ in _parts(c))
        if c["kind"] == "rope":
            return {"bytes": e * (2 * n + weights) + 4 * c["tokens"], "flops": 4.0 * n}
        x = c["tokens"] * sum(h * norm for h, _, norm, _ in _parts(c))
        return {"bytes": e * (2 * n + x + weights) + 4 * (weights + c["tokens"]), "flops": 8.0 * n}
    S, wide = c["groups"] * c["each"], c["rank"] + c["rope"]
    rows, tails = c["q_len"] * c["heads"], sum(_spread(S, c["own"], c["q_len"]))
    keys = c["groups"] * c["prefix"] + tails
    return {"bytes": 2 * (keys * wide + S * rows * (wide + c["rank"])) + 4 * keys / c["block"],
            "flops": 2.0 * rows * (S * c["prefix"] + tails) * (wide + c["rank"])}


# ---- the definition in 64 bits -------------------------------------------------

def _exact_quantise(x, rows):
    """(8-bit values, scales, scales of every element) of x [M, K] in 64 bits,
    both quotients rounded to fp32 as the definition says."""
    M, K = x.shape
    x = x.double()
    top = torch.nn.functional.pad(x.abs(), (0, -K % 128, 0, -M % rows))
    top = torch.amax(top.unfold(0, rows, rows).unfold(1, 128, 128), (2, 3))
    scale = torch.clamp((top / 448).float(), min=_SMALLEST).double()
    wide = scale.repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]
    q = (x / wide).float().double()
    # Steps of e4m3: 2^(e - 3) from 2^-6 on, 2^-9 below.
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return torch.round(q / step) * step, scale, wide


def _exact_rope(x, w, norm, start, dims, interleaved, positions, frequencies, magnitude):
    """One part through complex numbers in 64 bits."""
    x = x.double()
    if norm:
        n = x[..., :norm]
        x = torch.cat([n / (n.square().mean(-1, keepdim=True) + _EPS).sqrt() * w.double(), x[..., norm:]], -1)
    z = x[..., start:start + dims]
    z = z.unflatten(-1, (dims // 2, 2)) if interleaved else z.unflatten(-1, (2, dims // 2)).transpose(-1, -2)
    turn = torch.polar(torch.full_like(frequencies, magnitude)[None].expand(len(positions), -1).contiguous(),
                       positions.double()[:, None] * frequencies)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None])
    z = (z if interleaved else z.transpose(-1, -2)).flatten(-2)
    return torch.cat([x[..., :start], z, x[..., start + dims:]], -1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "linear":
        q, _, wide = _exact_quantise(s["x"], 1)
        w = s["w_scale"].double().repeat_interleave(128, 0)[: c["N"]].repeat_interleave(128, 1)[:, : c["K"]]
        return (q * wide) @ (s["w"].double() * w).t()
    if c["kind"] == "weight_grad":
        a, b = (_exact_quantise(s[x].t(), 1) for x in ("dy", "x"))
        return (a[0] * a[2]) @ (b[0] * b[2]).t()
    if c["kind"] == "quantise":
        q, scale, _ = _exact_quantise(s["x"], c["rows"])
        return q, scale
    if c["kind"] in ("rope", "rope_grad"):
        how = (c["rope"], c["interleaved"], s["positions"], s["frequencies"], s["magnitude"])
        out, weights = [], []
        for i, ((_, _, norm, start), x, w) in enumerate(zip(_parts(c), s["x"], s["weight"])):
            if c["kind"] == "rope":
                out.append(_exact_rope(x, w, norm, start, *how))
                continue
            leaves = [x.double().requires_grad_()] + ([w.double().requires_grad_()] if norm else [])
            y = _exact_rope(leaves[0], leaves[-1] if norm else None, norm, start, *how)
            grads = torch.autograd.grad(y, leaves, s["dy"][i].double())
            out.append(grads[0])
            weights += grads[1:]
        return out + weights
    out = torch.zeros(s["o"].shape, device="cuda", dtype=torch.float64)
    lens, B, wide = s["lens"].tolist(), c["block"], c["rank"] + c["rope"]
    for g in range(c["groups"]):
        head = s["cache"][s["table"][g * c["each"], : -(-c["prefix"] // B)].long()].reshape(-1, wide)[: c["prefix"]]
        for i in range(g * c["each"], (g + 1) * c["each"]):
            tail = s["cache"][s["table"][i, c["prefix"] // B: -(-lens[i] // B)].long()].reshape(-1, wide)
            kv = torch.cat([head, tail[c["prefix"] % B: c["prefix"] % B + lens[i] - c["prefix"]]]).double()
            for j in range(c["q_len"]):
                m = lens[i] - c["q_len"] + j + 1
                z = s["q"][i, j].double() @ kv[:m].t()
                out[i, j] = torch.softmax(z * s["alpha"], -1) @ kv[:m, : c["rank"]]
    return out
