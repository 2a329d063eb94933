"""Chunks whose running reference moves at every tile of 128 cells: the weights of a tile are then
computed twice, and the second ones must be those that are multiplied.  Tolerances are those of
test_gpu_dense.tolerance."""
import numpy as np
import pytest
import torch

from test_gpu_dense import BF16, DEV, E4M3, Pool, run_paged

pytestmark = pytest.mark.gpu


def grow(pool, steps, kv_dtype):
    """Keys whose magnitudes double `steps` times along each sequence."""
    for s, n in enumerate(pool.lens):
        rows = pool.rows(pool.table[s].cpu().numpy(), np.arange(n))
        e = torch.arange(n, device=DEV) * steps // n
        if kv_dtype == E4M3:
            pool.Ke[rows] = (118 + e).to(torch.uint8)[:, None]
        else:
            pool.K[rows] *= (2.0 ** (e - steps // 2))[:, None, None].to(BF16)
        pool.k[s] = pool.values(s, np.arange(n))[0]
    return pool


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,news,H_q", [([1900, 700], [60, 60], 16), ([900], [300], 16), ([1500], [70], 2)])
def test_logits_that_grow(lens, news, H_q, kv_dtype):
    pool = grow(Pool(lens, 2, 128, 64, kv_dtype, seed=50), 12, kv_dtype)
    run_paged(pool, news, H_q, BF16, seed=51)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_the_first_tile_far_above_and_far_below(kv_dtype):
    """Logits of thousands in the first tile, whose weights relative to nothing would be infinite, and then
    nothing that passes them; and the reverse."""
    for turn in (0, 1):
        pool = Pool([640], 2, 128, 64, kv_dtype, seed=52)
        t = pool.table[0].cpu().numpy()
        rows = pool.rows(t, np.arange(128) if turn == 0 else np.arange(512, 640))
        if kv_dtype == E4M3:
            pool.Ke[rows] = 130
        else:
            pool.K[rows] *= 64
        pool.k[0] = pool.values(0, np.arange(640))[0]
        run_paged(pool, [90], 16, BF16, seed=53)
        run_paged(pool, [90], 16, BF16, seed=54, causal=False)
