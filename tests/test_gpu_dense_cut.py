"""Items of the 128-row tensor-core attention that are cut between CTAs and joined, and the choice between
that and whole items.  A call that cuts writes its parts to the workspace; one that does not leaves it as it
was, which is how the tests here know which way a call took."""
import math

import pytest
import torch

import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, i32, starts

pytestmark = pytest.mark.gpu


def chunk_cuts(lens, news, H_q, H, page=64):
    """Whether paged_attn of `news` tokens over `lens` cells cuts its items."""
    counts = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(counts)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = torch.arange(at, at + c, device=DEV)
        at += c
    K = torch.zeros(at * page, H, 128, dtype=BF16, device=DEV)
    cache = qsa.PagedCache(K, K.clone(), page)
    n = sum(news)
    q = torch.randn(n, H_q, 128, device=DEV).to(BF16)
    out = torch.full_like(q, -7.0)
    ws = torch.full((qsa.paged_attn_workspace_size(n, len(lens), max(news), H_q, H, 128),), 255, dtype=torch.uint8, device=DEV)
    qsa.paged_attn(cache, table, i32(starts(news)), i32(lens), q, out, 1 / math.sqrt(128), max(news), workspace=ws)
    torch.cuda.synchronize()
    assert (out == 0).all()  # values of zero
    return bool((ws != 255).any())


def prompt_cuts(lens, H_q, H):
    n = sum(lens)
    q, k = torch.randn(n, H_q, 128, device=DEV).to(BF16), torch.randn(n, H, 128, device=DEV).to(BF16)
    out = torch.full_like(q, -7.0)
    ws = torch.full((qsa.prompt_attn_workspace_size(n, len(lens), H_q, H, 128),), 255, dtype=torch.uint8, device=DEV)
    qsa.prompt_attn(q, k, torch.zeros_like(k), i32(starts(lens)), out, 1 / math.sqrt(128), workspace=ws)
    torch.cuda.synchronize()
    assert (out == 0).all()
    return bool((ws != 255).any())


@pytest.mark.parametrize("lens,news,cut", [
    ([60000, 500, 500, 500], [256] * 4, True),   # one sequence has nearly all of the work
    ([60000, 1000], [512] * 2, True),
    ([60000] + [600] * 15, [512] * 16, True),    # and with more items than run at once
    ([2000] * 4, [256] * 4, False),              # short: nothing to win
    ([2000, 300, 300, 300], [256] * 4, False),
    ([2000], [400], False),
    ([20000], [400], True),
])
def test_a_long_chunk_among_short_ones_is_cut(lens, news, cut):
    assert chunk_cuts(lens, news, 32, 4) == cut


@pytest.mark.parametrize("lens,H_q,H,cut", [
    ([8000] + [1] * 15, 8, 2, True),             # as without the short ones
    ([8000], 8, 2, True),
    ([16000] + [50] * 20, 8, 2, True),
    ([900] * 3, 32, 4, False),
    ([777], 8, 2, False),
    ([2500, 700], 16, 2, False),
])
def test_a_long_prompt_among_short_ones_is_cut(lens, H_q, H, cut):
    assert prompt_cuts(lens, H_q, H) == cut
