"""Appends and sparse attention of as many tokens as a prefill chunk has, where a warp takes whole tokens and a CTA several
KV heads of one, and clusters of every size between.  Bounds as in the tests of the calls."""
import pytest

from four_bit_pool import E2M1, any_pool
from test_gpu_append import append
from test_gpu_dense import BF16, E4M3, F32
from test_gpu_paged_sparse import lists, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,H_q,H,d,rot,src,news", [
    (E2M1, 36, 1, 128, 128, BF16, [3000, 2000]),   # 19 steps, all of them a warp's
    (E4M3, 34, 3, 128, 64, BF16, [1500, 1, 499]),  # 19 steps, eight a warp: the last has queries, keys and values
    (BF16, 35, 5, 128, 128, F32, [5000]),          # 21 steps, the last of each kind with one head of two
    (F32, 3, 9, 256, 96, F32, [2600, 2600]),       # a head a step: nine of keys and values one after another
    (E2M1, 20, 6, 48, 48, F32, [900, 400]),        # heads of six lanes of eight, groups of 16 that lanes share unevenly
])
def test_appends_of_prompts(dtype, H_q, H, d, rot, src, news):
    pool = any_pool([n + 5 * i for i, n in enumerate(news)], H, d, 64, dtype, seed=40)
    append(pool, news, H_q, src, seed=41, rot=rot)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [E4M3, E2M1])
@pytest.mark.parametrize("H_q,H,news", [(8, 4, [700, 600]), (8, 4, [400, 300]), (8, 2, [700, 600]), (40, 4, [300, 100]), (40, 4, [300, 200]), (48, 2, [400, 250])])
def test_several_heads_a_cta(H_q, H, news, dtype, q_dtype):
    pool = any_pool([n + 150 for n in news], H, 128, 32, dtype, seed=42)
    run(pool, news, H_q, q_dtype, *lists(pool, news, 21, seed=43))


@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("tokens", [14, 16, 18, 20, 25, 33])
def test_clusters_of_every_size(tokens, dtype):
    pool = any_pool([1200 + 3 * i for i in range(tokens)], 4, 128, 64, dtype, seed=44)
    run(pool, [1] * tokens, 16, BF16, *lists(pool, [1] * tokens, 260, seed=45))
