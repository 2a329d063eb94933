"""Sparse attention over the blocks listed for each token, in place on a paged cache of every type, against the 64-bit
form over exactly those cells.  Bounds as test_gpu_dense's for a few tokens."""
import math

import numpy as np
import pytest
import torch

import dense_reference as ref
import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from four_bit_pool import E2M1, any_pool, kind_of
from test_gpu_dense import BF16, DEV, E4M3, F32, check_attention, i32, starts

pytestmark = pytest.mark.gpu


def lists(pool, news, k_blk, seed, full=False):
    """Blocks as a top-k writes them (ascending, complete at the token's position), some lists shorter or empty."""
    rng = np.random.default_rng(seed)
    n = sum(news)
    blocks, counts = np.full((n, k_blk), 1 << 30, np.int32), np.zeros(n, np.int32)
    at = 0
    for m, total in zip(news, pool.lens):
        for i in range(m):
            p = total - m + i
            whole = max(0, (p + 1) // 4)
            c = min(k_blk, whole)
            if not full and at % 5 == 3:
                c = int(rng.integers(0, c + 1))
            blocks[at, :c] = np.sort(rng.permutation(whole)[:c])
            counts[at] = c
            at += 1
    return blocks, counts


def run(pool, news, H_q, q_dtype, blocks, counts, seed=1, pad=2, scale=None, ld_pad=0, stream=None):
    d = pool.d
    scale = 1 / math.sqrt(d) if scale is None else scale
    rng = np.random.default_rng(seed)
    cu = starts(news)
    n = cu[-1] + pad
    qf = torch.from_numpy(rng.standard_normal((n, H_q * d + ld_pad)).astype(np.float32)).to(DEV).to(q_dtype)
    q = qf[:, :H_q * d].unflatten(1, (H_q, d))
    out = torch.full((n, H_q, d), -7.0, dtype=q_dtype, device=DEV)
    lse = torch.full((n, H_q), -7.0, device=DEV)
    b = np.concatenate([blocks, np.zeros((pad, blocks.shape[1]), np.int32)])
    c = np.concatenate([counts, np.full(pad, 1, np.int32)])
    qsa.paged_sparse_attn(pool.cache, pool.table, i32(cu), pool.kv_len, i32(b), i32(c), q, out, scale, lse=lse, stream=stream)
    torch.cuda.synchronize()
    o, l, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for s, m in enumerate(news):
        for i in range(m):
            t = cu[s] + i
            cells = four.listed_cells(blocks[t], counts[t], pool.lens[s] - m + i)
            units = None if pool.units[s] is None else pool.units[s][cells]
            check_attention(o[t:t + 1], l[t:t + 1], qn[t:t + 1], pool.k[s][cells], pool.v[s][cells], max(len(cells) - 1, 0), scale, len(cells) == 0, q_dtype,
                            kind_of(pool.K.dtype), units) if len(cells) else (np.testing.assert_array_equal(o[t], 0), np.testing.assert_array_equal(l[t], -np.inf))
    assert (o[cu[-1]:] == -7).all() and (l[cu[-1]:] == -7).all()
    return out, lse


CASES = [  # lens, news, H_q, H_kv, page, k_blk
    ([1, 2, 3, 4, 5, 8, 9, 64], [1] * 8, 8, 1, 8, 16),
    ([3000, 700, 0, 41], [1, 1, 0, 1], 32, 4, 64, 128),
    ([513, 64, 3], [4, 3, 3], 32, 4, 16, 40),
    ([333, 90], [2, 1], 12, 1, 32, 30),
    ([333, 90], [2, 1], 32, 1, 128, 30),
    ([90, 2], [2, 2], 4, 4, 32, 9),
    ([2600, 1100], [300, 250], 16, 2, 64, 33),
]


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1, F32])
@pytest.mark.parametrize("lens,news,H_q,H,page,k_blk", CASES)
def test_sparse(lens, news, H_q, H, page, k_blk, dtype, q_dtype):
    pool = any_pool(lens, H, 128, page, dtype, seed=3)
    run(pool, news, H_q, q_dtype, *lists(pool, news, k_blk, seed=4))


@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
@pytest.mark.parametrize("n_seq", [1, 5, 40])
def test_the_selection_of_the_framework(dtype, n_seq):
    """2,048 selected cells and the open block, from one sequence (many parts a token) to more tokens than CTAs."""
    pool = any_pool([9001 + 3 * i for i in range(n_seq)] if n_seq < 40 else [2300] * n_seq, 4 if n_seq < 40 else 1, 128, 64, dtype, seed=3)
    news = [1] * n_seq if n_seq < 40 else [4] * n_seq
    run(pool, news, 8 * pool.H, BF16, *lists(pool, news, 512, seed=4, full=True))


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, E2M1])
@pytest.mark.parametrize("H_q,H,d", [(33, 1, 128), (80, 2, 128), (4, 2, 64), (6, 2, 256), (3, 1, 16)])
def test_other_shapes(H_q, H, d, dtype, q_dtype):
    pool = any_pool([150, 40], H, d, 32, dtype, seed=6)
    run(pool, [3, 2], H_q, q_dtype, *lists(pool, [3, 2], 12, seed=7))


@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
def test_no_lists_and_odd_entries(dtype):
    """k_blk 0, negative counts, counts beyond k_blk, negative and incomplete blocks, a block twice."""
    pool = any_pool([50, 49, 48, 47], 2, 128, 16, dtype, seed=8)
    news = [1] * 4
    run(pool, news, 16, BF16, np.zeros((4, 0), np.int32), np.zeros(4, np.int32))
    run(pool, news, 16, BF16, np.zeros((4, 0), np.int32), np.full(4, 7, np.int32))
    blocks = np.array([[0, -1, 12, 13], [12, 11, 11, 3], [-2 ** 31, 2 ** 31 - 1, 2 ** 29, 1], [5, 5, 5, 5]], np.int32)
    run(pool, news, 16, BF16, blocks, np.array([4, 3, 9, 2], np.int32))
    run(pool, news, 16, BF16, blocks, np.array([-1, -2 ** 31, 0, 1], np.int32))


@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
def test_unlisted_cells_do_not_enter(dtype):
    """Cells that are not listed, and those behind the open block's token, are NaN; a listed NaN makes its token NaN."""
    pool = any_pool([130], 1, 128, 16, dtype, seed=9)
    blocks = np.array([[1, 7, 20]], np.int32)
    keep = np.zeros(130, bool)
    keep[four.listed_cells(blocks[0], 3, 129)] = True
    r = pool.rows(pool.table[0].cpu().numpy(), np.flatnonzero(~keep))
    if dtype == E2M1:
        for t in (pool.Ks, pool.Vs):
            t.view(torch.uint8)[r // 16, :, r % 16] = 0x7f
    else:
        for t in (pool.K, pool.V):
            t.view(torch.uint8 if dtype == E4M3 else dtype)[r] = 0x7f if dtype == E4M3 else float("nan")
    run(pool, [1], 8, BF16, blocks, np.array([3], np.int32))
    out, _ = torch.zeros(1, 8, 128, device=DEV).bfloat16(), None
    q = torch.randn(1, 8, 128, device=DEV).bfloat16()
    qsa.paged_sparse_attn(pool.cache, pool.table, i32([0, 1]), pool.kv_len, i32([[2, 7, 20]]), i32([3]), q, out, 0.1)
    assert torch.isnan(out).all()


@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
def test_bad_pages_and_lengths(dtype):
    pool = any_pool([100, 100, 100], 2, 128, 16, dtype, seed=10)
    t = pool.table.clone()
    t[1, 1] = -1
    kv = i32([100, 100, 16 * 1000])
    q = torch.randn(3, 16, 128, device=DEV).bfloat16()

    def call(first):
        out, lse = torch.zeros_like(q), torch.zeros(3, 16, device=DEV)
        qsa.paged_sparse_attn(pool.cache, t, i32([0, 1, 2, 3]), kv, i32([[first, 12]] * 3), i32([2] * 3), q, out, 0.1, lse=lse)
        return out, lse

    out, lse = call(5)  # a cell on the bad page
    assert torch.isnan(out[1:]).all() and torch.isnan(lse[1:]).all() and torch.isfinite(out[0]).all()
    out, lse = call(0)  # no cell on it
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2]).all()


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_scales(scale, q_dtype):
    for dtype in (BF16, E4M3, E2M1):
        pool = any_pool([300], 2, 128, 32, dtype, seed=11)
        run(pool, [2], 16, q_dtype, *lists(pool, [2], 40, seed=12), scale=scale)


def test_strided_queries_and_another_stream():
    pool = any_pool([300, 40], 2, 128, 32, E2M1, seed=11)
    b = lists(pool, [2, 1], 40, seed=12)
    run(pool, [2, 1], 16, BF16, *b, ld_pad=64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    run(pool, [2, 1], 16, BF16, *b, stream=st)


@pytest.mark.parametrize("dtype", [BF16, E4M3, E2M1])
def test_captured_graph_follows_lists(dtype):
    pool = any_pool([4000, 900], 2, 128, 64, dtype, seed=13)
    q = torch.randn(2, 16, 128, device=DEV).bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(2, 16, device=DEV)
    cu, counts = i32([0, 1, 2]), i32([0, 0])
    blocks = torch.zeros(2, 512, dtype=torch.int32, device=DEV)

    def call(o, l):
        qsa.paged_sparse_attn(pool.cache, pool.table, cu, pool.kv_len, blocks, counts, q, o, 0.09, lse=l)

    call(out, lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, lse)
    for lens, most in (([4000, 900], 512), ([2101, 3], 100), ([8, 899], 1)):
        pool.kv_len.copy_(i32(lens))
        pool.lens = lens
        b, c = lists(pool, [1, 1], most, seed=most)
        blocks[:, :most] = i32(b)
        counts.copy_(i32(c))
        q.normal_()
        want, wl = torch.zeros_like(out), torch.zeros_like(lse)
        call(want, wl)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
