"""Pages of more cells than any tile: appends, reads, attention and sparse attention on every type of cache.  Bounds as in the
tests of the calls."""
import numpy as np
import pytest
import torch

import gather_qsa_pool_gb300 as qsa
from four_bit_pool import E2M1, any_pool
from test_gpu_append import append
from test_gpu_dense import BF16, DEV, E4M3, F32
from test_gpu_paged_sparse import lists, run
from test_gpu_query_scales import attn, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [E2M1, E4M3, BF16])
@pytest.mark.parametrize("page", [256, 1024, 4096])
def test_calls(page, dtype):
    lens = [page + 131, 700, 3 * page // 2, 1]
    pool = any_pool(lens, 2, 128, page, dtype, seed=50)
    append(pool, [90, 3, 200, 1], 8, BF16, seed=51)
    for s, n in enumerate(lens):
        pool.k[s], pool.v[s] = pool.values(s, np.arange(n))
        if dtype != BF16:
            pool.units[s] = 2.0 ** (pool.Ve[pool.rows(pool.table[s].cpu().numpy(), np.arange(n))].double().cpu().numpy() - 127)
    for news, q_dtype in (([1, 1, 1, 1], BF16), ([3, 2, 4, 1], F32), ([90, 3, 200, 1], BF16)):
        q = torch.randn(sum(news), 16, 128, device=DEV).to(q_dtype)
        check(pool, news, q, *attn(pool, news, q, 0.09), 0.09)
        run(pool, news, 16, q_dtype, *lists(pool, news, 40, seed=52))
    K, V = (torch.zeros(4, max(lens), 2, 128, device=DEV) for _ in range(2))
    qsa.paged_read(pool.cache, pool.table, pool.kv_len, pool.kv_len, max(lens), K, V)
    for s, n in enumerate(lens):
        np.testing.assert_array_equal(K[s, :n].double().cpu().numpy(), pool.k[s])
        np.testing.assert_array_equal(V[s, :n].double().cpu().numpy(), pool.v[s])
