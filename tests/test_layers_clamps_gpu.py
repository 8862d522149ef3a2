"""What shared prefixes compute where starts, prefixes, lengths and block ids are out of
range: the groups and lengths as the definition clamps them, rows of zeros for bad
pages, and every row of O written."""

import math

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import Shared, clean_status, torch  # noqa: F401
from tests.test_serving_gpu import assert_within, attention_bound, attention_reference, status_is

pytestmark = pytest.mark.gpu


def clamped(c, N):
    """(lengths, the sequence with each one's prefix, prefix lengths) by the definition."""
    starts, n_seqs = c.starts.tolist(), c.table.shape[0]
    lens = [min(max(n, 0), N) for n in c.seq_lens.tolist()]
    first, prefix, top = list(range(n_seqs)), [0] * n_seqs, 0
    for i, p in enumerate(c.prefixes.tolist()):
        top = max(top, min(max(starts[i], 0), n_seqs))
        end = max(top, min(max(starts[i + 1], 0), n_seqs))
        for s in range(top, end):
            first[s], prefix[s] = top, min(max(p, 0), lens[top])
    return lens, first, prefix


def check(torch, c):
    S, most = c.table.shape
    lens, first, prefix = clamped(c, most * c.block)
    pages = c.cache.shape[0]
    pos = torch.arange(most * c.block, device="cuda")
    for s in range(S):
        page = torch.where(pos < prefix[s], c.table[first[s]].long()[pos // c.block], c.table[s].long()[pos // c.block])
        good = (page >= 0) & (page < pages)
        kv = torch.where(good[:, None], c.cache[page.clamp(0, pages - 1), pos % c.block].double(), 0.0)[:lens[s]]
        m = torch.arange(c.q_len, device="cuda")[:, None]
        keep = torch.arange(lens[s], device="cuda")[None, :] <= lens[s] - c.q_len + m
        O, W, Z, sv = attention_reference(c.q[s].double().transpose(0, 1), kv, kv[:, :c.R], c.alpha, keep)
        assert_within(torch, c.o[s].transpose(0, 1), O, attention_bound(c.t, c.R + c.P, lens[s], O, W, Z, sv), f"sequence {s}")


SPOILS = {
    "starts": lambda c: c.starts[1:3].copy_(c.starts.new_tensor([-5, 10 ** 6])),
    "order": lambda c: c.starts[:3].copy_(c.starts.new_tensor([4, 2, 5])),
    "prefix": lambda c: c.prefixes[:1].fill_(10 ** 6),
    "negative": lambda c: c.prefixes[1:2].fill_(-3),
    "lengths": lambda c: c.seq_lens[3:5].copy_(c.seq_lens.new_tensor([-7, 10 ** 6])),
    "table": lambda c: c.table[0, 1:3].copy_(c.table.new_tensor([10 ** 6, -2])),
}


@pytest.mark.parametrize("form", ["few", "many sequences", "many groups", "rows"])
@pytest.mark.parametrize("spoil", list(SPOILS))
def test_what_is_out_of_range_is_clamped(torch, form, spoil):
    """few: a thread a sequence and group plans; many: a CTA in rounds (the spoiled starts
    far from the round they end in); rows: the kernel for any sizes."""
    groups = [(64, 30, 20, 10), (32, 5, 6)]
    if form == "many sequences":
        groups += [(7, *[1] * 64)] * 17
    elif form == "many groups":
        groups += [(7, *[1] * 40)] * 3
    many = form.startswith("many")
    c = Shared(torch, "bf16", groups, 2 if many else 16, 1, 96 if form == "rows" else 128, 64, 16, shared_pages=True)
    c.cache = c.cache.nan_to_num(0.0)
    if form == "many groups":
        c.starts = torch.cat([c.starts, c.starts[-1:].repeat(1100)])
        c.prefixes = torch.cat([c.prefixes, c.prefixes.new_full((1100,), 5)])
        c.workspace = torch.empty(sg.sbgemm_latent_shared_workspace_bytes(len(c.lens), len(c.prefixes), 1, 2, 128),
                                  device="cuda", dtype=torch.uint8)
    assert max(len(c.lens), len(c.prefixes)) > 1024 or not many
    SPOILS[spoil](c)
    c.o.fill_(math.nan)
    c.run()
    status_is(10)
    check(torch, c)
