"""Queries of any magnitude over an 8-bit cache: a huge finite query in one token and head leaves the others of its
sequence and KV head as right as they were.  Bounds as test_gpu_dense's, of the queries without it."""
import math

import pytest
import torch

from four_bit_pool import any_pool
from test_gpu_dense import BF16, DEV, E4M3, F32
from test_gpu_query_scales import OUTLIERS, attn, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [[150, 333], [5000, 9001]])
@pytest.mark.parametrize("news", [1, 2, 4])
@pytest.mark.parametrize("H_q,H", OUTLIERS)
def test_a_large_query_is_its_rows_own(H_q, H, news, lens, q_dtype):
    pool = any_pool(lens, H, 128, 16, E4M3, seed=17)
    fresh = [news] * 2
    n = 2 * news
    q = torch.randn(n, H_q, 128, device=DEV).to(q_dtype)
    clean, lse = attn(pool, fresh, q, 0.09)
    check(pool, fresh, q, clean, lse, 0.09)
    for x in (1e30, 1e4):
        big = q.clone()
        big[n - 1, 1, 7] = x
        got, l = attn(pool, fresh, big, 0.09)
        got[n - 1, 1], l[n - 1, 1] = clean[n - 1, 1], lse[n - 1, 1]
        check(pool, fresh, q, got, l, 0.09)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("power", [-100, -60, -20, 20, 60, 100])
@pytest.mark.parametrize("news,lens", [(1, [260, 37]), (4, [260, 37]), (1, [9001, 5000])])
def test_magnitudes_of_all_queries(news, lens, power, q_dtype):
    """Queries times 2^power, the scale of the logits by as much smaller."""
    scale = 2.0 ** -power / math.sqrt(128)
    pool = any_pool(lens, 2, 128, 32, E4M3, seed=6)
    q = (torch.randn(2 * news, 16, 128, device=DEV) * 2.0 ** power).to(q_dtype)
    check(pool, [news, news], q, *attn(pool, [news, news], q, scale), scale)
