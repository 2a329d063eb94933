"""Items of the 128-row tensor-core attention that are cut between CTAs and joined, and the choice between
that and whole items.  A call that cuts writes its parts to the workspace; one that does not leaves it as it
was, which is how the tests here know which way a call took."""
import math

import numpy as np
import pytest
import torch

import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, E4M3, Pool, check_attention, i32, run_paged, starts
from test_gpu_dense_few import widen

pytestmark = pytest.mark.gpu


def chunk_cuts(lens, news, H_q, H, page=64, cells=0, kv_dtype=BF16):
    """Whether paged_attn of `news` tokens over `lens` cells cuts its items; cells: the table's width."""
    counts = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(max(counts), cells // page)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, c in enumerate(counts):
        table[s, :c] = torch.arange(at, at + c, device=DEV)
        at += c
    K = torch.zeros(at * page, H, 128, device=DEV).to(kv_dtype)
    e = torch.full((at * page, H), 127, dtype=torch.uint8, device=DEV) if kv_dtype == E4M3 else None
    cache = qsa.PagedCache(K, K.clone(), page, K_exp=e, V_exp=e)
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


@pytest.mark.parametrize("lens,news,kv_dtype,cut", [
    # 128 items, not 152: whole, they leave SMs idle, which on e4m3 cells costs more than joining; bf16
    # products of that length run at the power cap, where fewer SMs are as fast
    ([61789], [1024], BF16, False), ([61789], [1024], E4M3, True),
    ([8000], [1024], BF16, False), ([8000], [1024], E4M3, True),
    ([2000], [1024], BF16, False), ([2000], [1024], E4M3, False),
])
def test_a_chunk_of_nearly_as_many_items_as_ctas(lens, news, kv_dtype, cut):
    assert chunk_cuts(lens, news, 32, 4, kv_dtype=kv_dtype) == cut


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


# ------------------------------------------------------------------ results

CHUNKS = [
    # lens, news, H_q, H; items (row tiles of 256 rows) below the number of CTAs, and above it
    ([1500], [300], 16, 2),                       # ten row tiles, both groups of rows, the last one short
    ([900, 1300], [100, 37], 32, 4),
    ([700, 40, 1100, 500], [400, 40, 370, 300], 32, 4),
    ([600] * 5, [250] * 5, 8, 8),                 # one head a KV head
]


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_chunks_that_are_cut(case, causal, kv_dtype):
    """A table of 65,536 cells: the host takes the sequences to be that long, and cuts."""
    lens, news, H_q, H = CHUNKS[case]
    assert chunk_cuts(lens, news, H_q, H, cells=65536)
    pool = widen(Pool(lens, H, 128, 64, kv_dtype, seed=60 + case), 65536)
    run_paged(pool, news, H_q, BF16, seed=70 + case, causal=causal)


PROMPTS = [
    # lens, H_q, H, cut; more items than run at once from the third on
    ([4000], 4, 4, True),
    ([4500], 2, 2, True),
    ([8000], 8, 2, True),
    ([6000, 1, 40, 700], 16, 2, True),
    ([900] * 3, 32, 4, False),
    ([2000, 10, 10, 1500], 32, 4, False),
]


def prompt(lens, H_q, H, seed, causal=True):
    """(call, q, k, v, out, lse) of packed prompts."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = sum(lens)
    q, k, v = (torch.randn(n, h, 128, device=DEV, generator=g).to(BF16) for h in (H_q, H, H))
    out, lse = torch.full_like(q, float("nan")), torch.full((n, H_q), float("nan"), device=DEV)
    ws = torch.full((qsa.prompt_attn_workspace_size(n, len(lens), H_q, H, 128),), 255, dtype=torch.uint8, device=DEV)
    cu = i32(starts(lens))
    call = lambda: qsa.prompt_attn(q, k, v, cu, out, 1 / math.sqrt(128), causal=causal, lse=lse, workspace=ws)
    return call, q, k, v, out, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompts_cut_and_whole_in_turns(case, causal):
    """Every row is written; of each row tile some are compared."""
    lens, H_q, H, cut = PROMPTS[case]
    assert prompt_cuts(lens, H_q, H) == cut
    call, q, k, v, out, lse = prompt(lens, H_q, H, case, causal)
    call()
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    cu = starts(lens)
    for a, b in zip(cu, cu[1:]):
        for i in np.unique(np.r_[np.arange(a, b, 53), b - 1]):
            o, l, qn = (x[i:i + 1].double().cpu().numpy() for x in (out, lse, q))
            check_attention(o, l, qn, kn[a:b], vn[a:b], i - a, 1 / math.sqrt(128), causal, BF16, BF16)


@pytest.mark.parametrize("lens,H_q,H", [([4000], 4, 4), ([8000], 8, 2)])
def test_cut_prompts_give_up_and_recover(lens, H_q, H):
    """With a limit of 0 every wait gives up without looking; the parts that are joined are NaN."""
    call, _, _, _, out, lse = prompt(lens, H_q, H, 9)
    call()
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    try:
        qsa.set_wait_options(status, 0)
        out.fill_(3.0)
        lse.fill_(3.0)
        call()
        torch.cuda.synchronize()
        assert int(status.item()) == 4  # QSA_ERR_TIMEOUT
        assert torch.isnan(out.float()).all() and torch.isnan(lse).all()
        qsa.set_wait_options(status, qsa.QSA_WAIT_DEFAULT_NS)
        status.zero_()
        for _ in range(2):
            call()
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
        assert int(status.item()) == 0
    finally:
        qsa.set_wait_options(None, qsa.QSA_WAIT_DEFAULT_NS)


def test_cut_chunks_in_a_captured_graph_with_lengths_that_change():
    """The list of work follows the lengths on the device: one capture, several lengths."""
    lens, news, H_q, H = [1500, 700], [100, 60], 16, 2
    pool = widen(Pool([2000, 2000], H, 128, 64, BF16, seed=80), 65536)
    assert chunk_cuts(lens, news, H_q, H, cells=65536)
    cu, kv_len = starts(news), i32(lens)
    q = torch.randn(cu[-1], H_q, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(cu[-1], H_q, device=DEV)
    ws = torch.full((qsa.paged_attn_workspace_size(int(cu[-1]), 2, 100, H_q, H, 128),), 255, dtype=torch.uint8, device=DEV)
    cd = i32(cu)
    call = lambda: qsa.paged_attn(pool.cache, pool.table, cd, kv_len, q, out, 0.1, 100, lse=lse, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([1500, 700], [100, 2000], [2000, 60], [130, 61]):
        kv_len.copy_(i32(now))
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        o, l, qn = (x.double().cpu().numpy() for x in (out, lse, q))
        for s in (0, 1):
            a, b = cu[s], cu[s + 1]
            check_attention(o[a:b], l[a:b], qn[a:b], pool.k[s][:now[s]], pool.v[s][:now[s]], now[s] - news[s], 0.1, True,
                            BF16, BF16)
