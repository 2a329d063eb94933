"""Values whose powers of two lie more than 2^50 from one, met after ordinary ones: the kernels of a few rows keep the
softmax's sum by a reference of its own from there on.  Bounds as test_gpu_dense's."""
import numpy as np
import pytest
import torch

from four_bit_pool import E2M1, any_pool
from test_gpu_dense import BF16, E4M3, F32, DEV
from test_gpu_four_bit import run_attn
from test_gpu_paged_sparse import lists, run

pytestmark = pytest.mark.gpu


def far_from(pool, first, choices, seed):
    """Exponent bytes of the values of sequence s from cell first[s] on: one of choices[s mod their number] each."""
    rng = np.random.default_rng(seed)
    for s, n in enumerate(pool.lens):
        r = pool.rows(pool.table[s].cpu().numpy(), np.arange(n))
        e = pool.Ve[r].cpu().numpy()
        e[first[s]:] = rng.choice(choices[s % len(choices)], e[first[s]:].shape)
        pool.Ve[r] = torch.from_numpy(e).to(DEV)
        pool.v[s] = pool.values(s, np.arange(n))[1]
        pool.units[s] = 2.0 ** (e.astype(float) - 127)


SMALL, LARGE, BOTH = [60, 70, 76], [178, 185, 190], [62, 120, 127, 188]


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("H_q,news,cells", [(8, 1, 2000), (32, 1, 1400), (32, 4, 900)])
def test_far_values_behind_ordinary_ones(H_q, news, cells, q_dtype):
    """So many cells that a warp takes a dozen tiles of a sequence, ordinary ones first."""
    n = 64 if news == 1 else 40
    lens = [cells + 7 * i for i in range(n)]
    pool = any_pool(lens, 4, 128, 32, E2M1, seed=30)
    far_from(pool, [m // 4 + (37 * i) % (m // 2) for i, m in enumerate(lens)], [SMALL, LARGE, BOTH], seed=31)
    run_attn(pool, [news] * n, H_q, q_dtype, seed=32)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [E4M3, E2M1])
@pytest.mark.parametrize("news", [[1], [3, 1], [30, 30, 30, 30]])
def test_far_values_in_lists(news, dtype, q_dtype):
    """512 blocks a token: shared by the CTAs of a cluster, and all of a token in one CTA."""
    lens = [2300 + 9 * i for i in range(len(news))]
    for choices in ([SMALL], [LARGE], [BOTH]) if len(news) < 4 else ([SMALL, LARGE, BOTH],):
        pool = any_pool(lens, 4, 128, 64, dtype, seed=33)
        far_from(pool, [700 + 50 * i for i in range(len(news))], choices, seed=34)
        run(pool, news, 8, q_dtype, *lists(pool, news, 512, seed=35))


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [E4M3, E2M1])
def test_far_values_everywhere_in_lists(dtype, q_dtype):
    """Exponents over their whole range but for overflow, open blocks of one to four cells, and lists of nothing else."""
    lens = [300, 301, 302, 303, 3]
    pool = any_pool(lens, 2, 128, 32, dtype, seed=36)
    far_from(pool, [0] * 5, [[27, 60, 90, 120, 127, 150], [27, 127, 200, 222]], seed=37)
    run(pool, [1] * 5, 16, q_dtype, *lists(pool, [1] * 5, 60, seed=38))
    run(pool, [1] * 5, 16, q_dtype, np.zeros((5, 0), np.int32), np.zeros(5, np.int32))
