"""Cases of the 16-bit serving operators: latent attention over a paged cache
(absorbed form) and over expanded keys and values, the 16-bit strided product
that goes between the two forms, and the page operations of the cache.

Every case has a plain form in elementary torch operations (fp32, rounded once
at the end) and the call of the library.  Latent attention keeps one vector a
token, [c | k_rope], for all heads: with K_h = [W_uk_h c | k_rope] and V_h =
W_uv_h c, the absorbed form scores q_lat = W_uk_h^T q against c itself and
averages the c, the expanded form makes K_h and V_h by a product first.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_WORKSPACE = 64 << 20


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # One user's chat, one new token, 16 heads left on this GPU: latency counts.
        dict(name="decode one short sequence", kind="decode", type="bf16", seqs=1, q_len=1, heads=16,
             longest=701, block=64, rank=512, rope=64),
        # A served batch of ragged contexts over small pages: bound by the cache's bytes.
        dict(name="decode ragged batch", kind="decode", type="fp16", seqs=32, q_len=1, heads=16,
             longest=8191, block=16, rank=512, rope=64),
        # All heads on one GPU and a full batch of long contexts: the most work a step has.
        dict(name="decode 128 heads", kind="decode", type="bf16", seqs=64, q_len=1, heads=128,
             longest=8192, block=64, rank=512, rope=64),
        # A short prompt whose keys and values were expanded: every launch counts.
        dict(name="prompt of 333", kind="prompt", type="fp16", seqs=1, heads=16, q_max=333, context=0,
             nope=128, rope=64, value=128, causal=True),
        # Ragged prompts of a batch, with a context that was there before the chunk.
        dict(name="prompts of 4096 after 1000", kind="prompt", type="bf16", seqs=3, heads=32, q_max=4096,
             context=1000, nope=128, rope=64, value=128, causal=True),
        # Absorbing W_uk into the queries of a decode batch: one product a head.
        dict(name="absorb 64 tokens", kind="product", type="bf16", batch=128, M=64, N=512, K=128,
             b_major="n", interleave=True),
        # Expanding the latents of a prompt into the keys and values of 32 heads.
        dict(name="expand 4099 tokens", kind="product", type="bf16", batch=1, M=4099, N=8192, K=512,
             b_major="k", interleave=False),
        # Fresh pages for pages that are to be written (copy-on-write).
        dict(name="copy pages", kind="copy", type="bf16", blocks=8192, block=64, row=576, caches=1,
             seqs=64, longest=6000, n=1500),
        # Beam search: every beam forks a parent of the step before.
        dict(name="fork 64 sequences", kind="fork", type="bf16", blocks=16384, block=16, row=576, caches=2,
             seqs=128, longest=2000, n=64),
        # One decode step's new rows.
        dict(name="append to 128 sequences", kind="append", type="bf16", blocks=16384, block=16, row=576,
             caches=2, seqs=128, longest=1900, n=128, tokens=1),
        # Finished sequences leave.
        dict(name="free 48 sequences", kind="free", type="bf16", blocks=16384, block=16, row=64, caches=1,
             seqs=128, longest=2000, n=48),
        # Packing the pages in use into the front of the pool, to give the rest back.
        dict(name="compact a pool", kind="compact", type="bf16", blocks=16384, block=64, row=576, caches=1,
             seqs=96, longest=9000, n=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prompt", "prompt", "product", "copy", "fork", "append", "free",
                       "compact"])
    c = dict(kind=kind, type=rng.choice(["bf16", "fp16"]))
    if kind == "decode":
        c["heads"] = rng.choice([1, 4, 8, 16, 16, 20, 32, 64, 128])
        c["q_len"] = rng.choice([1, 1, 1, 2, 3, 4]) if c["heads"] <= 32 else 1
        c["seqs"] = _log(rng, 1, 128)
        c["longest"] = _log(rng, 1, min(100000, 524288 // c["seqs"]))
        c["block"] = rng.choice([8, 16, 24, 32, 64, 128])
        c["rank"], c["rope"] = rng.choice([(512, 64), (512, 64), (256, 32), (128, 64)])
    elif kind == "prompt":
        c["heads"] = _log(rng, 1, 64)
        c["seqs"] = _log(rng, 1, 8)
        c["q_max"] = _log(rng, 1, 4096)
        c["context"] = rng.choice([0, 0, _log(rng, 1, 4000)])
        c["nope"], c["rope"], c["value"] = rng.choice([(128, 64, 128), (128, 64, 128), (64, 32, 64), (96, 32, 80)])
        c["causal"] = rng.random() < 0.8
        # Bounded by the largest listed case's rows x keys.
        while c["seqs"] * c["heads"] * c["q_max"] * (c["q_max"] + c["context"]) > 2.0e9:
            c["q_max"] = (c["q_max"] * 3 + 3) // 4
            c["context"] = c["context"] * 3 // 4
    elif kind == "product":
        c["interleave"] = rng.random() < 0.5
        if c["interleave"]:
            c["batch"] = _log(rng, 1, 128)
            c["M"] = _log(rng, 1, 512)
            c["N"], c["K"], c["b_major"] = rng.choice([(512, 128, "n"), (128, 512, "k"), (256, 96, "n"), (80, 264, "k")])
        else:
            c["batch"] = 1
            c["M"] = _log(rng, 1, 4096)
            c["N"] = 8 * _log(rng, 1, 1024)
            c["K"] = 8 * _log(rng, 4, 64)
            c["b_major"] = rng.choice(["n", "k"])
    else:
        c["blocks"] = _log(rng, 256, 16384)
        c["block"] = rng.choice([8, 16, 32, 64])
        c["row"] = rng.choice([64, 128, 576])
        c["caches"] = rng.choice([1, 2, 3])
        c["seqs"] = _log(rng, 2, 128)
        # At most three quarters of the pool in use.
        c["longest"] = max(1, min(9000, c["blocks"] * c["block"] * 3 // (4 * c["seqs"]) - c["block"]))
        c["n"] = rng.randint(1, max(1, c["seqs"] // 2))
        if kind == "copy":
            c["n"] = rng.randint(1, c["blocks"] // 5)
        if kind == "append":
            c["n"], c["tokens"] = rng.randint(1, c["seqs"]), rng.choice([1, 1, 2, 7, 40])
            c["n"] = min(c["n"], max(1, c["blocks"] // 4 // (c["tokens"] // c["block"] + 2)))
    return c


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _spread(n, longest):
    """n lengths evenly over the upper three quarters of `longest`."""
    return [longest - (3 * longest * i) // (4 * n) for i in range(n)]


def _lens(g, n, longest):
    """Those lengths in an order of the seed's."""
    lens = torch.tensor(_spread(n, longest), device="cuda", dtype=torch.int32)
    return lens[torch.randperm(n, generator=g, device="cuda")]


def _tables(g, lens, longest, block, blocks, max_blocks=None):
    """Block table over a random set of a pool's pages: page i of sequence s, -1 past its last."""
    n = lens.numel()
    most = max_blocks or -(-longest // block)
    used = (lens.long() + block - 1) // block
    here = torch.arange(most, device="cuda")[None, :] < used[:, None]
    order = torch.randperm(blocks, generator=g, device="cuda")
    table = torch.full((n, most), -1, device="cuda", dtype=torch.int32)
    table[here] = order[: int(used.sum())].to(torch.int32)
    return table


def prepare(case, seed):
    g = _gen(seed)
    c, t = case, _TYPES[case["type"]]
    s = {"case": dict(case)}
    if c["kind"] == "decode":
        wide = c["rank"] + c["rope"]
        lens = _lens(g, c["seqs"], c["longest"])
        blocks = c["seqs"] * -(-c["longest"] // c["block"]) + 3
        s["lens"] = lens
        s["table"] = _tables(g, lens, c["longest"], c["block"], blocks)
        s["cache"] = _randn(g, blocks, c["block"], wide, dtype=t)
        s["q"] = _randn(g, c["seqs"], c["q_len"], c["heads"], wide, dtype=t)
        s["o"] = torch.empty(c["seqs"], c["q_len"], c["heads"], c["rank"], device="cuda", dtype=t)
        s["alpha"] = 1.0 / math.sqrt(128 + c["rope"])
        s["workspace"] = torch.empty(_WORKSPACE, device="cuda", dtype=torch.uint8)
    elif c["kind"] == "prompt":
        q_lens = _lens(g, c["seqs"], c["q_max"])
        k_lens = q_lens + c["context"]
        zero = torch.zeros(1, device="cuda", dtype=torch.int32)
        s["q_starts"] = torch.cat([zero, torch.cumsum(q_lens, 0).to(torch.int32)])
        s["k_starts"] = torch.cat([zero, torch.cumsum(k_lens, 0).to(torch.int32)])
        nq, nk = int(q_lens.sum()), int(k_lens.sum())
        # Keys and values as the expanding product leaves them, side by side for each head.
        kv = _randn(g, nk, c["heads"], c["nope"] + c["value"], dtype=t)
        s["k_nope"], s["v"] = kv[..., : c["nope"]], kv[..., c["nope"]:]
        s["k_rope"] = _randn(g, nk, c["rope"], dtype=t)
        s["q"] = _randn(g, nq, c["heads"], c["nope"] + c["rope"], dtype=t)
        s["o"] = torch.empty(nq, c["heads"], c["value"], device="cuda", dtype=t)
        s["alpha"] = 1.0 / math.sqrt(c["nope"] + c["rope"])
    elif c["kind"] == "product":
        b, M, N, K = c["batch"], c["M"], c["N"], c["K"]
        if c["interleave"]:      # [tokens, heads, .], a head's rows apart
            s["a"] = _randn(g, M, b, K, dtype=t).transpose(0, 1)
            s["c"] = torch.empty(M, b, N, device="cuda", dtype=t).transpose(0, 1)
        else:
            s["a"] = _randn(g, b, M, K, dtype=t)
            s["c"] = torch.empty(b, M, N, device="cuda", dtype=t)
        w = _randn(g, b, K, N, dtype=torch.float32) / math.sqrt(K)
        s["b"] = w.to(t) if c["b_major"] == "n" else w.transpose(1, 2).contiguous().to(t).transpose(1, 2)
    else:
        most = -(-(c["longest"] + c.get("tokens", 0)) // c["block"])
        lens = _lens(g, c["seqs"], c["longest"])
        pick = torch.randperm(c["seqs"], generator=g, device="cuda")
        if c["kind"] == "fork":  # half of the rows are parents, half are free for children
            lens[pick[: c["seqs"] // 2]] = 0
        table = _tables(g, lens, c["longest"], c["block"], c["blocks"], most)
        refs = torch.zeros(c["blocks"], device="cuda", dtype=torch.int32)
        refs[table[table >= 0].long()] = 1
        # The bookkeeping before the call, and the working copy that a pass starts from.
        s["before"] = torch.cat([refs, table.reshape(-1), lens])
        s["now"] = s["before"].clone()
        s["refs"], flat, s["lens"] = s["now"].split([c["blocks"], c["seqs"] * most, c["seqs"]])
        s["table"] = flat.view(c["seqs"], most)
        s["caches"] = [_randn(g, c["blocks"], c["block"], c["row"], dtype=t) for _ in range(c["caches"])]
        s["workspace"] = torch.empty(_WORKSPACE, device="cuda", dtype=torch.uint8)
        if c["kind"] == "copy":
            used = table[table >= 0]
            free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
            n = min(c["n"], used.numel(), free.numel())
            at = torch.randint(0, used.numel(), (n,), generator=g, device="cuda")
            to = free[torch.randperm(free.numel(), generator=g, device="cuda")[:n]]
            s["pairs"] = torch.stack([used[at], to], 1).contiguous()
        elif c["kind"] == "fork":
            half = c["seqs"] // 2
            n = min(c["n"], half)
            s["children"] = pick[:half][:n].to(torch.int32)
            at = torch.randint(half, c["seqs"], (n,), generator=g, device="cuda")
            s["parents"] = pick[at].to(torch.int32)
        elif c["kind"] == "append":
            s["seqs"] = pick[: c["n"]].to(torch.int32)
            total = c["n"] * c["tokens"]
            s["starts"] = torch.arange(0, total + 1, c["tokens"], device="cuda", dtype=torch.int32)
            s["rows"] = [_randn(g, total, c["row"], dtype=t) for _ in range(c["caches"])]
        elif c["kind"] == "free":
            s["seqs"] = pick[: c["n"]].to(torch.int32)
    return s


# ---- one pass ------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["kind"]](s)


def _own_decode(s):
    import strided_gemm_gb300 as sg
    return sg.latent_attention_paged(s["q"], s["cache"], s["table"], s["lens"], s["o"], alpha=s["alpha"],
                                     causal=True, workspace=s["workspace"])


def _own_prompt(s):
    import strided_gemm_gb300 as sg
    return sg.latent_attention(s["q"], s["k_nope"], s["k_rope"], s["v"], s["o"], s["q_starts"], s["k_starts"],
                               s["case"]["q_max"], alpha=s["alpha"], causal=s["case"]["causal"])


def _own_product(s):
    import strided_gemm_gb300 as sg
    return sg.matmul_half(s["a"], s["b"], s["c"])


def _pool(s):
    return s["caches"], s["refs"], s["table"], s["lens"]


def _own_copy(s):
    import strided_gemm_gb300 as sg
    sg.pages_copy(s["caches"], s["pairs"], workspace=s["workspace"])
    return s["caches"]


def _own_fork(s):
    import strided_gemm_gb300 as sg
    s["now"].copy_(s["before"])
    sg.pages_fork(*_pool(s), s["parents"], s["children"], workspace=s["workspace"])
    return _pool(s)


def _own_append(s):
    import strided_gemm_gb300 as sg
    s["now"].copy_(s["before"])
    sg.pages_append(*_pool(s), s["seqs"], s["starts"], s["rows"], workspace=s["workspace"])
    return _pool(s)


def _own_free(s):
    import strided_gemm_gb300 as sg
    s["now"].copy_(s["before"])
    sg.pages_free(*_pool(s), s["seqs"])
    return s["refs"], s["table"], s["lens"]


def _own_compact(s):
    import strided_gemm_gb300 as sg
    s["now"].copy_(s["before"])
    sg.pages_compact(*_pool(s), workspace=s["workspace"])
    return _pool(s)


_own = {"decode": _own_decode, "prompt": _own_prompt, "product": _own_product, "copy": _own_copy,
        "fork": _own_fork, "append": _own_append, "free": _own_free, "compact": _own_compact}


def _softmax(x):
    """Softmax over the last axis, in place; zeros where everything is masked (-inf)."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _plain_decode(s):
    c = s["case"]
    S, T, H, N = c["seqs"], c["q_len"], c["heads"], c["longest"]
    n = torch.arange(N, device="cuda")
    here = n[None, :] < s["lens"][:, None]
    page = s["table"].long()[:, n // c["block"]].clamp_min(0)
    kv = s["cache"][page, n % c["block"]].float() * here[..., None]
    q = s["q"].float().reshape(S, T * H, -1)
    x = torch.bmm(q, kv.transpose(1, 2)).mul_(s["alpha"]).view(S, T, H, N)
    last = s["lens"][:, None] - T + torch.arange(T, device="cuda")[None, :]
    x.masked_fill_((n[None, None, :] > last[..., None])[:, :, None, :], -math.inf)
    p = _softmax(x).view(S, T * H, N)
    s["o"].copy_(torch.bmm(p, kv[..., : c["rank"]]).view(S, T, H, c["rank"]))
    return s["o"]


def _plain_prompt(s):
    c = s["case"]
    Q, N = c["q_max"], c["q_max"] + c["context"]
    qs, ks = s["q_starts"].long(), s["k_starts"].long()
    q_len, k_len = qs.diff(), ks.diff()
    m, n = torch.arange(Q, device="cuda"), torch.arange(N, device="cuda")
    q_at = (qs[:-1, None] + m).clamp_max(s["q"].shape[0] - 1)
    k_at = (ks[:-1, None] + n).clamp_max(s["v"].shape[0] - 1)
    k = torch.cat([s["k_nope"].float(), s["k_rope"].float()[:, None, :].expand(-1, c["heads"], -1)], -1)
    q, k = s["q"].float()[q_at].transpose(1, 2), k[k_at].transpose(1, 2)
    v = s["v"].float()[k_at].transpose(1, 2)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["alpha"])
    hide = (n[None, :] >= k_len[:, None])[:, None, :]
    if c["causal"]:
        hide = hide | (n[None, None, :] > (k_len - q_len)[:, None, None] + m[None, :, None])
    x.masked_fill_(hide[:, None], -math.inf)
    o = torch.matmul(_softmax(x), v).transpose(1, 2)
    s["o"].copy_(o[m[None, :] < q_len[:, None]])
    return s["o"]


def _plain_product(s):
    s["c"].copy_(torch.matmul(s["a"].float(), s["b"].float()))
    return s["c"]


def _plain_copy(s):
    src, dst = s["pairs"].long().unbind(1)
    s["caches"] = [x.index_copy_(0, dst, x[src]) for x in s["caches"]]
    return s["caches"]


def _plain_fork(s):
    c = s["case"]
    s["now"].copy_(s["before"])
    par, kid = s["parents"].long(), s["children"].long()
    lens = s["lens"][par]
    full, rest = (lens // c["block"]).long(), lens % c["block"]
    need = rest > 0
    i = torch.arange(s["table"].shape[1], device="cuda")
    rows = s["table"][par]
    shared = i[None, :] < full[:, None]
    s["refs"].index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    fresh = torch.nonzero(s["refs"] == 0)[:, 0][: int(need.sum())]
    s["refs"][fresh] = 1
    old = rows[need, full[need]].long()
    rows[need, full[need]] = fresh.to(torch.int32)
    s["table"][kid] = torch.where(i[None, :] < (full + need)[:, None], rows, s["table"][kid])
    s["lens"][kid] = lens
    r = torch.arange(c["block"], device="cuda")
    some = r[None, :] < rest[need][:, None]
    src, dst = (old[:, None] * c["block"] + r)[some], (fresh[:, None] * c["block"] + r)[some]
    s["caches"] = [x.view(-1, c["row"]).index_copy_(0, dst, x.view(-1, c["row"])[src]).view(x.shape) for x in s["caches"]]
    return _pool(s)


def _plain_append(s):
    c = s["case"]
    s["now"].copy_(s["before"])
    seq, count = s["seqs"].long(), s["starts"].diff()
    old = s["lens"][seq]
    have, want = (old + c["block"] - 1) // c["block"], (old + count + c["block"] - 1) // c["block"]
    i = torch.arange(s["table"].shape[1], device="cuda")
    new = (i[None, :] >= have[:, None]) & (i[None, :] < want[:, None])
    fresh = torch.nonzero(s["refs"] == 0)[:, 0][: int(new.sum())]
    s["refs"][fresh] = 1
    rows = s["table"][seq]
    rows[new] = fresh.to(torch.int32)
    s["table"][seq] = rows
    s["lens"][seq] = old + count
    j = torch.arange(s["rows"][0].shape[0], device="cuda")
    who = torch.searchsorted(s["starts"].long(), j, right=True) - 1
    at = old.long()[who] + j - s["starts"].long()[who]
    dst = rows[who, at // c["block"]].long() * c["block"] + at % c["block"]
    s["caches"] = [x.view(-1, c["row"]).index_copy_(0, dst, y).view(x.shape) for x, y in zip(s["caches"], s["rows"])]
    return _pool(s)


def _plain_free(s):
    c = s["case"]
    s["now"].copy_(s["before"])
    seq = s["seqs"].long()
    used = (s["lens"][seq] + c["block"] - 1) // c["block"]
    i = torch.arange(s["table"].shape[1], device="cuda")
    pages = s["table"][seq][i[None, :] < used[:, None]]
    s["refs"].index_add_(0, pages.long(), -torch.ones_like(pages))
    s["lens"][seq] = 0
    return s["refs"], s["table"], s["lens"]


def _plain_compact(s):
    c = s["case"]
    s["now"].copy_(s["before"])
    used = s["refs"] > 0
    total = used.sum()
    i = torch.arange(c["blocks"], device="cuda")
    src, dst = torch.nonzero(used & (i >= total))[:, 0], torch.nonzero(~used & (i < total))[:, 0]
    to = i.to(torch.int32)
    to[src] = dst.to(torch.int32)
    s["caches"] = [x.index_copy_(0, dst, x[src]) for x in s["caches"]]
    s["refs"][dst] = s["refs"][src]
    s["refs"][src] = 0
    j = torch.arange(s["table"].shape[1], device="cuda")
    live = j[None, :] < ((s["lens"] + c["block"] - 1) // c["block"])[:, None]
    s["table"].copy_(torch.where(live, to[s["table"].long().clamp_min(0)], s["table"]))
    return _pool(s)


_plain = {"decode": _plain_decode, "prompt": _plain_prompt, "product": _plain_product, "copy": _plain_copy,
          "fork": _plain_fork, "append": _plain_append, "free": _plain_free, "compact": _plain_compact}


# ---- the work of one pass ------------------------------------------------------

def work(case):
    c = case
    if c["kind"] == "decode":
        rows, wide = c["seqs"] * c["q_len"] * c["heads"], c["rank"] + c["rope"]
        keys = sum(_spread(c["seqs"], c["longest"]))
        return {"bytes": 2 * (keys * wide + rows * (wide + c["rank"])) + 4 * keys / c["block"],
                "flops": 2.0 * keys * c["q_len"] * c["heads"] * (wide + c["rank"])}
    if c["kind"] == "prompt":
        lens = _spread(c["seqs"], c["q_max"])
        q, k = sum(lens), sum(lens) + c["seqs"] * c["context"]
        pairs = sum(n * (n + c["context"]) - (n * (n - 1) // 2 if c["causal"] else 0) for n in lens)
        return {"bytes": 2 * c["heads"] * (q * (c["nope"] + c["rope"] + c["value"]) + k * (c["nope"] + c["value"]))
                + 2 * k * c["rope"],
                "flops": 2.0 * c["heads"] * pairs * (c["nope"] + c["rope"] + c["value"])}
    if c["kind"] == "product":
        b, M, N, K = c["batch"], c["M"], c["N"], c["K"]
        return {"bytes": 2.0 * b * (M * K + K * N + M * N), "flops": 2.0 * b * M * N * K}
    page = 2.0 * c["block"] * c["row"] * c["caches"]
    pages = sum(-(-n // c["block"]) for n in _spread(c["seqs"], c["longest"])) / c["seqs"]
    books = 4.0 * (c["blocks"] + c["seqs"] * -(-c["longest"] // c["block"]) + c["seqs"])
    if c["kind"] == "copy":
        n = min(c["n"], c["blocks"] - c["seqs"] * pages)
        return {"bytes": 2 * n * page + 8 * n, "flops": 0}
    if c["kind"] == "fork":
        return {"bytes": 3 * books + min(c["n"], c["seqs"] // 2) * (page + 12 * pages), "flops": 0}
    if c["kind"] == "append":
        return {"bytes": 3 * books + c["n"] * c["tokens"] * 2 * page / c["block"], "flops": 0}
    if c["kind"] == "free":
        return {"bytes": 2 * books + c["n"] * 12 * pages, "flops": 0}
    used = c["seqs"] * pages
    moved = used * max(0.0, 1 - used / c["blocks"])
    return {"bytes": 3 * books + 2 * moved * page, "flops": 0}


# ---- the definition in 64 bits -------------------------------------------------

def exact(case, seed):
    c = case
    if c["kind"] not in ("decode", "prompt", "product"):
        return None                       # pages are moved, not computed
    s = prepare(case, seed)
    if c["kind"] == "product":
        return torch.einsum("bmk,bkn->bmn", s["a"].double(), s["b"].double())
    if c["kind"] == "decode":
        out = torch.zeros(s["o"].shape, device="cuda", dtype=torch.float64)
        lens = s["lens"].tolist()
        for i, n in enumerate(lens):
            kv = s["cache"][s["table"][i, : -(-n // c["block"])].long()].reshape(-1, c["rank"] + c["rope"])[:n].double()
            for j in range(c["q_len"]):
                m = n - c["q_len"] + j + 1
                if m > 0:
                    z = s["q"][i, j].double() @ kv[:m].t()
                    out[i, j] = torch.softmax(z * s["alpha"], -1) @ kv[:m, : c["rank"]]
        return out
    out = torch.zeros(s["o"].shape, device="cuda", dtype=torch.float64)
    q0, k0 = s["q_starts"].tolist(), s["k_starts"].tolist()
    for i in range(c["seqs"]):
        q, o = s["q"][q0[i]:q0[i + 1]], out[q0[i]:q0[i + 1]]
        rope, k, v = (s[x][k0[i]:k0[i + 1]] for x in ("k_rope", "k_nope", "v"))
        keep = torch.ones(len(q), len(k), device="cuda", dtype=torch.bool)
        if c["causal"]:
            keep = keep.tril(len(k) - len(q))
        for h in range(c["heads"]):
            z = q[:, h, : c["nope"]].double() @ k[:, h].double().t() + q[:, h, c["nope"]:].double() @ rope.double().t()
            o[:, h] = torch.softmax(torch.where(keep, z * s["alpha"], -math.inf), -1) @ v[:, h].double()
    return out
