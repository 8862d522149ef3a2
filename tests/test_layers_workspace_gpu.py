"""A workspace asked for the largest batch serves every smaller one."""

import random

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_gpu import Shared, clean_status, torch  # noqa: F401
from tests.test_serving_gpu import status_is

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,q_len,R", [(16, 1, 512), (3, 2, 128), (128, 1, 512), (5, 1, 40)])
def test_fewer_groups_sequences_or_heads_fit_the_same_workspace(torch, heads, q_len, R):
    """Fewer groups have more query rows each, which other tiles take."""
    most = 24
    need = sg.sbgemm_latent_shared_workspace_bytes(most, most, q_len, heads, R)
    whole = torch.full((need + 4096,), 77, device="cuda", dtype=torch.uint8)
    few = max(1, heads // 3)
    for groups, h in (([(60, *range(q_len, q_len + most))], heads), ([(9, 5, 6, 7)] * 8, heads), ([(70, *range(5, 25))], few),
                      ([(30, 4, 9)], heads), ([(20, 3)] * most, few), ([(11, 3)], 1)):
        c = Shared(torch, "bf16", groups, h, q_len, R, 8, 16)
        c.workspace = whole[:need]
        c.run()
        c.check(torch)
        assert bool((whole[need:] == 77).all())
    status_is(0)


def test_sizes_never_shrink(torch):
    rng = random.Random(1)
    for _ in range(400):
        n_seqs, q_len, heads, R = rng.randint(1, 200), rng.randint(1, 4), rng.randint(1, 130), rng.choice([40, 128, 512])
        n_groups = rng.randint(0, n_seqs)
        need = sg.sbgemm_latent_shared_workspace_bytes(n_seqs, n_groups, q_len, heads, R)
        s = rng.randint(1, n_seqs)
        assert sg.sbgemm_latent_shared_workspace_bytes(s, rng.randint(0, min(s, n_groups)), rng.randint(1, q_len),
                                                       rng.randint(1, heads), rng.choice([r for r in (40, 128, 512) if r <= R])) <= need
