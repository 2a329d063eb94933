"""Queries of any magnitude over rows of codes: what a row of queries (a token and head) holds is right for that row,
whatever the rows beside it hold.  The kernels of a few rows take queries as fp16, scaled by a power of two; bounds as
test_gpu_dense's, row by row."""
import math

import numpy as np
import pytest
import torch

import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from four_bit_pool import E2M1, any_pool, kind_of
from test_gpu_dense import BF16, DEV, E4M3, F32, check_attention, i32, starts
from test_gpu_paged_sparse import lists

pytestmark = pytest.mark.gpu


def attn(pool, news, q, scale, max_q=None):
    n, H_q, d = q.shape
    out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device=DEV)
    mq = max_q or max(news)
    ws = torch.zeros(max(16, qsa.paged_attn_workspace_size(n, len(news), mq, H_q, pool.H, d)), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32(starts(news)), pool.kv_len, q, out, scale, mq, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    return out, lse


def sparse(pool, news, q, scale, blocks, counts):
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    qsa.paged_sparse_attn(pool.cache, pool.table, i32(starts(news)), pool.kv_len, i32(blocks), i32(counts), q, out, scale, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def check(pool, news, q, out, lse, scale, listed=None):
    """Each KV head by itself: the bound goes by the magnitudes of its own queries and keys."""
    cu, G = starts(news), q.shape[1] // pool.H
    o, l, qn = (t.double().cpu().numpy() for t in (out, lse, q))
    for s, m in enumerate(news):
        for g in range(pool.H):
            h = slice(g * G, (g + 1) * G)
            k, v, u = pool.k[s][:, g:g + 1], pool.v[s][:, g:g + 1], pool.units[s]
            u = None if u is None else u[:, g:g + 1]
            if listed is None:
                a, b = cu[s], cu[s + 1]
                check_attention(o[a:b, h], l[a:b, h], qn[a:b, h], k, v, pool.lens[s] - m, scale, True, q.dtype, kind_of(pool.K.dtype), u)
                continue
            for i in range(m):
                t = cu[s] + i
                c = four.listed_cells(listed[0][t], listed[1][t], pool.lens[s] - m + i)
                check_attention(o[t:t + 1, h], l[t:t + 1, h], qn[t:t + 1, h], k[c], v[c], len(c) - 1, scale, False, q.dtype,
                                kind_of(pool.K.dtype), None if u is None else u[c])


def shift_keys(pool, by):
    """KV head g's keys times 2^by[g]."""
    pool.Ke += torch.tensor(by, dtype=torch.int32, device=DEV).to(torch.uint8)  # modulo 256
    for s, n in enumerate(pool.lens):
        pool.k[s] = pool.values(s, np.arange(n))[0]


HEADS = [  # H_q, powers of two of the KV heads' queries
    (32, [40, -20, 0, -45]), (8, [-50, 50]), (28, [0, 25, -1, -25]), (32, [30, -30]), (6, [45, 3, -40])]


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("news", [1, 3, 8])
@pytest.mark.parametrize("H_q,powers", HEADS)
def test_heads_of_different_magnitude(H_q, powers, news, q_dtype):
    """Keys of a head are as much smaller as its queries are larger: logits are ordinary in all of them."""
    H = len(powers)
    pool = any_pool([300, 41], H, 128, 32, E2M1, seed=3)
    shift_keys(pool, [-p for p in powers])
    q = torch.randn(2 * news, H_q, 128, device=DEV) * torch.tensor(powers, device=DEV).exp2().repeat_interleave(H_q // H)[:, None]
    q = q.to(q_dtype)
    check(pool, [news, news], q, *attn(pool, [news, news], q, 0.09), 0.09)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [E4M3, E2M1])
@pytest.mark.parametrize("n_seq,news", [(2, 3), (2, 650)])
def test_heads_of_different_magnitude_in_lists(n_seq, news, dtype, q_dtype):
    """A few tokens, and as many as take the heads of a token in one CTA."""
    powers = [40, -20, 0, -45]
    pool = any_pool([900, 700], 4, 128, 32, dtype, seed=3)
    shift_keys(pool, [-p for p in powers])
    fresh = [news] * n_seq
    q = (torch.randn(n_seq * news, 8, 128, device=DEV) * torch.tensor(powers, device=DEV).exp2().repeat_interleave(2)[:, None]).to(q_dtype)
    b = lists(pool, fresh, 20, seed=4)
    check(pool, fresh, q, *sparse(pool, fresh, q, 0.09, *b), 0.09, b)


OUTLIERS = [(32, 4), (16, 2), (24, 1), (4, 4), (14, 2)]


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("news", [1, 2, 4])
@pytest.mark.parametrize("H_q,H", OUTLIERS)
def test_a_large_query_is_its_rows_own(H_q, H, news, q_dtype):
    """One huge finite query in the last token: every other row is what it is without it, bit for bit."""
    pool = any_pool([150, 333], H, 128, 16, E2M1, seed=17)
    n = 2 * news
    q = torch.randn(n, H_q, 128, device=DEV).to(q_dtype)
    clean, lse = attn(pool, [news, news], q, 0.09)
    check(pool, [news, news], q, clean, lse, 0.09)
    odd = torch.zeros(n, H_q, dtype=torch.bool, device=DEV)
    odd[n - 1, 1] = True
    for x in (1e30, 1e4):
        q[n - 1, 1, 7] = x
        got, l = attn(pool, [news, news], q, 0.09)
        assert torch.equal(got[~odd], clean[~odd]) and torch.equal(l[~odd], lse[~odd])
        # (more than 64 bf16 rows are a chunk, whose kernel forms logit * scale - reference in one rounding: what the
        # reference's own rounding left of it, 2^-24 of the reference, is in every exponent, 2^70 here)
        if q_dtype == F32 or news * H_q // H <= 64:
            assert torch.isfinite(got).all() and torch.isfinite(l).all()


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("H_q,H", OUTLIERS)
def test_a_large_query_is_its_rows_own_in_lists(H_q, H, dtype, q_dtype):
    pool = any_pool([150, 333], H, 128, 16, dtype, seed=17)
    q = torch.randn(4, H_q, 128, device=DEV).to(q_dtype)
    b = lists(pool, [2, 2], 30, seed=5)
    clean, lse = sparse(pool, [2, 2], q, 0.09, *b)
    check(pool, [2, 2], q, clean, lse, 0.09, b)
    odd = torch.zeros(4, H_q, dtype=torch.bool, device=DEV)
    odd[3, 1] = True
    for x in (1e30, 1e4):
        q[3, 1, 7] = x
        got, l = sparse(pool, [2, 2], q, 0.09, *b)
        assert torch.equal(got[~odd], clean[~odd]) and torch.equal(l[~odd], lse[~odd])
        assert torch.isfinite(got).all() and torch.isfinite(l).all()


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("power", [-100, -60, -20, 20, 60, 100])
@pytest.mark.parametrize("news", [1, 4])
def test_magnitudes_of_all_queries(news, power, q_dtype):
    """Queries times 2^power, the scale of the logits by as much smaller."""
    scale = 2.0 ** -power / math.sqrt(128)
    for dtype in (E2M1, E4M3):
        pool = any_pool([260, 37], 2, 128, 32, dtype, seed=6)
        q = (torch.randn(2 * news, 16, 128, device=DEV) * 2.0 ** power).to(q_dtype)
        if dtype == E2M1:
            check(pool, [news, news], q, *attn(pool, [news, news], q, scale), scale)
        b = lists(pool, [news, news], 30, seed=7)
        check(pool, [news, news], q, *sparse(pool, [news, news], q, scale, *b), scale, b)
