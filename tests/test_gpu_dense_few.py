"""Few query rows over long contexts (qsa_paged_attn with bf16 queries): up to 32 rows a sequence and KV
head, over bf16 cells and over e4m3 cells whose codes are multiplied as they are.  Which kernel a call of
few rows takes follows from the most cells a sequence may have: tables here are widened with entries that
nothing may read.

Tolerances are those of the other dense attention tests (test_gpu_dense.tolerance).  They hold here by:
bf16 weights, and e4m3 weights of nine bits, are off by 2^-9 of themselves, inside the 2^-8; an e4m3 weight
ends at 2^-16 where the largest is at least 2^10, so at 2^-26 of it, inside 2^-25; a query of the item ends
at 2^-31 of the item's largest, so a logit is off by scale * 2^-31 * max|q| * sum|k|, inside the
(d + 16) * 2^-24 of the largest |q||k|.
"""
import math

import numpy as np
import pytest
import torch

import dense_reference as ref
import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, E4M3, F32, Pool, check_attention, i32, run_paged, starts

pytestmark = pytest.mark.gpu


def widen(pool, cells=16384):
    """The pool's table with entries of no page behind each sequence's own, so that a row of it is
    `cells` long."""
    t = pool.table
    n = -(-cells // pool.page)
    if t.shape[1] < n:
        pad = torch.full((t.shape[0], n - t.shape[1]), -1, dtype=torch.int32, device=DEV)
        pool.table = torch.cat([t, pad], 1).contiguous()
    return pool


FEW = [
    # lens, news, H_q, H, page
    ([2050], [1], 8, 2, 64),                                     # four rows
    ([1, 7, 128, 129, 0, 1000], [1, 1, 1, 1, 0, 1], 32, 4, 16),  # eight rows; tiles just full and just begun
    ([700, 33, 5, 260], [4, 4, 4, 1], 32, 4, 64),                # 32 rows
    ([3, 300], [4, 4], 8, 1, 8),                                 # more new tokens than cells
    ([257, 1, 640], [5, 1, 5], 9, 3, 128),                       # three heads a KV head: 15 rows
    ([500, 130], [10, 10], 3, 1, 32),                            # and 30
    ([300, 129], [32, 7], 2, 2, 32),                             # one head a KV head
    ([400], [1], 32, 1, 4096),                                   # 32 heads a KV head
    ([900, 40], [1, 1], 40, 2, 16),                              # twenty
    ([1500, 1400], [2, 3], 10, 2, 64),                           # five
]


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("case", range(len(FEW)))
def test_few_rows(case, kv_dtype):
    lens, news, H_q, H, page = FEW[case]
    run_paged(widen(Pool(lens, H, 128, page, kv_dtype, seed=40 + case)), news, H_q, BF16, seed=60 + case)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news,H_q", [([8, 5, 1, 0], 32), ([16, 3, 9, 2], 16), ([11, 1, 7, 5], 20)])
def test_rows_of_two_tiles(news, H_q, kv_dtype):
    """Up to 64 rows: e4m3 cells are read once for each 32 of them."""
    run_paged(widen(Pool([700, 5, 260, 40], 4, 128, 64, kv_dtype, seed=27)), news, H_q, BF16, seed=28)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_more_tokens_than_the_host_said(kv_dtype):
    """max_q chooses the kernel only: chunks and prompts by the kernel of few rows."""
    run_paged(widen(Pool([400, 90, 61], 2, 128, 64, kv_dtype, seed=29)), [150, 90, 1], 16, BF16, seed=30, max_q=1)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_few_rows_counts_beyond_the_buffers(kv_dtype):
    """cu_q that runs past the buffers, or back, and lengths below zero, are clipped; nothing behind the
    buffers is touched."""
    pool = widen(Pool([300, 200, 100], 2, 128, 64, kv_dtype, seed=31))
    q = torch.randn(12, 16, 128, device=DEV).to(BF16)
    big = torch.full((30, 16, 128), -7.0, dtype=BF16, device=DEV)
    lse = torch.full((30, 16), -7.0, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(12, 3, 4, 16, 2, 128), dtype=torch.uint8, device=DEV)
    for cu, lens in (([0, 4, 2, 90], [300, 200, 100]), ([-5, 4, 2 ** 31 - 1, 3], [300, 200, 100]),
                     ([0, 4, 8, 12], [-1, 2 ** 31 - 1, 100]), ([0, 0, 0, 0], [300, 200, 100])):
        qsa.paged_attn(pool.cache, pool.table, i32(cu), i32(lens), q, big[:12], 0.1, 4, lse=lse[:12], workspace=ws)
        torch.cuda.synchronize()
        assert (big[12:] == -7).all() and (lse[12:] == -7).all()
    # a sequence of no cell gives zeros, one longer than its row of the table NaN
    big.fill_(-7.0)
    qsa.paged_attn(pool.cache, pool.table, i32([0, 4, 8, 12]), i32([-1, 2 ** 31 - 1, 100]), q, big[:12], 0.1, 4, lse=lse[:12],
                   workspace=ws)
    assert (big[:4] == 0).all() and torch.isneginf(lse[:4]).all()
    assert torch.isnan(big[4:8].float()).all() and torch.isfinite(big[8:12].float()).all()


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [[1, 1], [4, 2]])
def test_few_rows_without_causal_mask(news, kv_dtype):
    run_paged(widen(Pool([333, 129], 2, 128, 32, kv_dtype, seed=3)), news, 16, BF16, seed=4, causal=False)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("scale", [8.0, 0.0, -0.2, 1e-20])
@pytest.mark.parametrize("news", [1, 4])
def test_few_rows_scales(news, scale, kv_dtype):
    run_paged(widen(Pool([150, 700], 2, 128, 32, kv_dtype, seed=10)), [news, news], 16, BF16, seed=11, scale=scale)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 4])
def test_few_rows_logits_that_grow(news, kv_dtype):
    """Each tile's largest logit passes the last one's: the references move at every tile."""
    pool = widen(Pool([1900, 700], 2, 128, 64, kv_dtype, seed=12))
    for s, n in enumerate(pool.lens):
        rows = pool.rows(pool.table[s].cpu().numpy(), np.arange(n))
        if kv_dtype == E4M3:
            pool.Ke[rows] = (118 + torch.arange(n, device=DEV) * 12 // n).to(torch.uint8)[:, None]
        else:
            pool.K[rows] *= (2.0 ** (torch.arange(n, device=DEV) * 12 // n - 6))[:, None, None].to(BF16)
        pool.k[s] = pool.values(s, np.arange(n))[0]
    run_paged(pool, [news, news], 16, BF16, seed=13)


@pytest.mark.parametrize("news", [1, 4])
def test_few_rows_exponents_far_apart(news):
    """e4m3 values whose rows' exponents span the whole range, rows of zeros, and a sequence of the
    smallest exponent alone."""
    pool = widen(Pool([300, 700, 260], 2, 128, 32, E4M3, seed=20))
    rng = np.random.default_rng(21)
    for s in range(3):
        rows = pool.rows(pool.table[s].cpu().numpy(), np.arange(pool.lens[s]))
        e = rng.choice([27, 60, 90, 120, 127, 150], (len(rows), 2))
        if s == 1:
            e[200:] = rng.choice([27, 127, 200, 227], (len(rows) - 200, 2))
        if s == 2:
            e[:] = 27
        pool.Ve[rows] = torch.from_numpy(e.astype(np.uint8)).to(DEV)
        pool.V.view(torch.uint8)[rows[10:20]] = 0
        pool.v[s] = pool.values(s, np.arange(pool.lens[s]))[1]
        pool.units[s] = 2.0 ** (e.astype(float) - 127)
    run_paged(pool, [news] * 3, 16, BF16, seed=22)


def test_few_rows_sums_of_the_smallest_exponent():
    """Twenty thousand cells of zeros at the smallest exponent: their sum is far above one in units of the
    weights' reference."""
    n, page = 20000, 128
    pages = -(-n // page)
    K = torch.zeros(pages * page, 1, 128, device=DEV).to(E4M3)
    e = torch.full((pages * page, 1), 27, dtype=torch.uint8, device=DEV)
    cache = qsa.PagedCache(K, K.clone(), page, K_exp=e, V_exp=e)
    q = torch.randn(1, 8, 128, device=DEV).to(BF16)
    out, lse = torch.ones_like(q), torch.zeros(1, 8, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(1, 1, 1, 8, 1, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(cache, torch.arange(pages, device=DEV).int()[None].contiguous(), i32([0, 1]), i32([n]), q, out, 0.1, 1,
                   lse=lse, workspace=ws)
    assert (out == 0).all()
    # (the logarithm of a sum in fp32: log2 of the sum is below 2^5 and off by half of 2^-19 once or twice)
    assert (lse.double() - math.log(n)).abs().max() <= 4 * 2.0 ** -19


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_few_rows_queries_of_every_size(kv_dtype):
    """Heads whose queries differ by 2^30, one with an infinity, one with a NaN: each head alone."""
    pool = widen(Pool([900], 1, 128, 64, kv_dtype, seed=15))
    rng = np.random.default_rng(16)
    size = 2.0 ** np.array([0, -30, -60, 4, -8, -15, 0, 0])
    qn = rng.standard_normal((1, 8, 128)) * size[None, :, None]
    q = torch.from_numpy(qn.astype(np.float32)).to(DEV).to(BF16)
    q[0, 6, 17], q[0, 7, 90] = float("inf"), float("nan")
    out, lse = torch.zeros_like(q), torch.zeros(1, 8, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(1, 1, 1, 8, 1, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32([0, 1]), pool.kv_len, q, out, 0.1, 1, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isnan(out[0, 6:].float()).all() and torch.isnan(lse[0, 6:]).all()
    check_attention(out[:, :6].double().cpu().numpy(), lse[:, :6].double().cpu().numpy(),
                    q[:, :6].double().cpu().numpy(), pool.k[0], pool.v[0], 899, 0.1, True, BF16, kv_dtype, pool.units[0])


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 4])
def test_few_rows_a_page_outside_the_pool_gives_nan(news, kv_dtype):
    pool = widen(Pool([400, 220, 300], 2, 128, 32, kv_dtype, seed=13))
    table = pool.table.clone()
    table[1, 2] = pool.cache.n_pages
    lens = pool.kv_len.clone()
    lens[2] = 32 * table.shape[1] + 1  # longer than its row of the table
    n = 3 * news
    q = torch.randn(n, 16, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(n, 16, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, 3, news, 16, 2, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, table, i32(starts([news] * 3)), lens, q, out, 0.1, news, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:news].float()).all() and torch.isfinite(lse[:news]).all()
    assert torch.isnan(out[news:].float()).all() and torch.isnan(lse[news:]).all()


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_few_rows_cells_not_seen_do_not_matter(kv_dtype):
    """NaN in the keys and values of the third of four new tokens: the first two do not see them."""
    lens, bad = [300, 128, 129], float("nan")
    pool = widen(Pool(lens, 2, 128, 32, kv_dtype, seed=14))
    for s, n in enumerate(lens):
        r = pool.rows(pool.table[s].cpu().numpy(), np.array([n - 2]))
        if kv_dtype == E4M3:
            pool.K.view(torch.uint8)[r, :, 3], pool.V.view(torch.uint8)[r, :, 5] = 0x7f, 0xff
        else:
            pool.K[r, :, 3], pool.V[r, :, 5] = bad, bad
    q = torch.randn(12, 16, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(12, 16, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(12, 3, 4, 16, 2, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32([0, 4, 8, 12]), pool.kv_len, q, out, 0.1, 4, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    o, l, qn = (x.double().cpu().numpy() for x in (out, lse, q))
    for s, n in enumerate(lens):
        a = 4 * s
        check_attention(o[a:a + 2], l[a:a + 2], qn[a:a + 2], pool.k[s][:n - 2], pool.v[s][:n - 2], n - 4, 0.1, True, BF16,
                        kv_dtype, None if kv_dtype == BF16 else pool.units[s][:n - 2])
        assert np.isnan(o[a + 2:a + 4]).all()


def test_few_rows_an_infinite_value_reaches_who_sees_it():
    """bf16: an infinity in the last new token's value is the last token's alone, in its dimension alone."""
    pool = widen(Pool([200], 1, 128, 32, BF16, seed=17), 4096)
    r = pool.rows(pool.table[0].cpu().numpy(), np.array([199]))
    pool.V[r, 0, 7] = float("-inf")
    q = torch.randn(4, 8, 128, device=DEV).to(BF16)
    out = torch.zeros_like(q)
    ws = torch.zeros(qsa.paged_attn_workspace_size(4, 1, 4, 8, 1, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32([0, 4]), pool.kv_len, q, out, 0.1, 4, workspace=ws)
    assert torch.isfinite(out[:3].float()).all()
    assert (out[3, :, 7] == float("-inf")).all()
    out[3, :, 7] = 0
    assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 4])
def test_few_rows_many_short_sequences(news, kv_dtype):
    """A CTA has a score of parts, whole items among them; some sequences have no new token."""
    rng = np.random.default_rng(18)
    lens = [int(x) for x in rng.integers(news, 300, 700)]
    news = [0 if i % 17 == 3 else news for i in range(len(lens))]
    run_paged(widen(Pool(lens, 4, 128, 64, kv_dtype, seed=19), 4096 if kv_dtype == BF16 else 16384), news, 32, BF16, seed=20)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_few_rows_strided_and_on_another_stream(kv_dtype):
    pool = widen(Pool([90, 300], 2, 128, 16, kv_dtype, seed=8, pad_k=64))
    run_paged(pool, [4, 4], 16, BF16, seed=9, ld_pad=40, stream=torch.cuda.Stream())


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_few_rows_captured_and_replayed(kv_dtype):
    """A graph follows lengths and counts that change in place; two calls in it share a workspace."""
    pool = widen(Pool([900, 300], 2, 128, 64, kv_dtype, seed=25))
    scale, cu, lens = 0.1, i32([0, 2, 4]), i32([500, 130])
    q = torch.randn(2, 8, 16, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(2, 8, 16, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(8, 2, 4, 16, 2, 128), dtype=torch.uint8, device=DEV)

    def run(o, l):
        for i in (0, 1):
            qsa.paged_attn(pool.cache, pool.table, cu, lens, q[i], o[i], scale, 2, lse=l[i], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(out, lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, lse)
    for c, l in (([0, 2, 4], [500, 130]), ([0, 4, 5], [900, 1]), ([0, 0, 8], [0, 300]), ([0, 1, 2], [128, 129])):
        cu.copy_(i32(c))
        lens.copy_(i32(l))
        out.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            o, w, qn = (x[i].double().cpu().numpy() for x in (out, lse, q))
            for s in (0, 1):
                a, b = c[s], c[s + 1]
                check_attention(o[a:b], w[a:b], qn[a:b], pool.k[s][:l[s]], pool.v[s][:l[s]], l[s] - (b - a), scale, True,
                                BF16, kv_dtype, None if kv_dtype == BF16 else pool.units[s][:l[s]])
            assert (o[c[2]:] == -7).all()
        again = torch.zeros_like(out), torch.zeros_like(lse)
        run(*again)
        for i in (0, 1):
            assert torch.equal(again[0][i, :c[2]], out[i, :c[2]]) and torch.equal(again[1][i, :c[2]], lse[i, :c[2]])


def test_few_rows_beyond_32_bits():
    """Codes and exponents whose places lie past 2^32."""
    page, H, d, ld = 64, 2, 128, 16384
    n_pages = (1 << 32) // (ld * page) + 4
    K = torch.empty(n_pages * page, ld, dtype=torch.uint8, device=DEV).view(E4M3)
    V = torch.empty(n_pages * page, ld, dtype=torch.uint8, device=DEV).view(E4M3)
    Ke, Ve = (torch.zeros(n_pages * page, H, dtype=torch.uint8, device=DEV) for _ in range(2))
    cache = qsa.PagedCache(K[:, :H * d].unflatten(1, (H, d)), V[:, :H * d].unflatten(1, (H, d)), page, K_exp=Ke, V_exp=Ve)
    table = torch.zeros(1, 256, dtype=torch.int32, device=DEV)
    table[0, :3] = i32([n_pages - 1, 0, n_pages - 3])
    n = 150
    x = torch.randn(2, n, H, d, device=DEV).to(BF16)
    qsa.paged_write(cache, table, i32([0, n]), i32([n]), x[0], x[1])
    back = torch.zeros(2, 1, n, H, d, device=DEV)
    qsa.paged_read(cache, table, i32([n]), i32([n]), n, back[0], back[1])
    q = torch.randn(4, 16, d, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(4, 16, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(4, 1, 4, 16, H, d), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(cache, table, i32([0, 4]), i32([n]), q, out, 0.1, 4, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    k, v = back[:, 0].double().cpu().numpy()
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy(), k, v, n - 4, 0.1, True,
                    BF16, E4M3)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 4])
def test_few_rows_give_up_and_recover(news, kv_dtype):
    """With the limit of its waits at 0 the kernel reports it, leaves NaN and returns its tensor memory;
    the next call is right again."""
    pool = widen(Pool([3000, 700, 90], 2, 128, 64, kv_dtype, seed=26))
    n = 3 * news
    q = torch.randn(n, 16, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(n, 16, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, 3, news, 16, 2, 128), dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run():
        qsa.paged_attn(pool.cache, pool.table, i32(starts([news] * 3)), pool.kv_len, q, out, 0.1, news, lse=lse, workspace=ws)
        torch.cuda.synchronize()

    run()
    want = out.clone(), lse.clone()
    assert torch.isfinite(out.float()).all()
    try:
        qsa.set_wait_options(status, 0)
        out.fill_(3.0)
        run()
        assert int(status.item()) == 4  # QSA_ERR_TIMEOUT
        assert torch.isnan(out.float()).all() and torch.isnan(lse).all()
    finally:
        qsa.set_wait_options(None, qsa.QSA_WAIT_DEFAULT_NS)
    for _ in range(2):
        run()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news,many", [(1, False), (4, False), (90, False), (1, True), (4, True)])
def test_short_limits_give_nan_or_the_result(news, many, kv_dtype):
    """Limits that run out somewhere in the middle: every row is right or NaN, whoever gives up first, and
    the next call is right."""
    lens = [6000, 700, 100] + ([130, 300, 128] * 300 if many else [])  # many: a score of parts a CTA
    pool = widen(Pool(lens, 2, 128, 64, kv_dtype, seed=32))
    n = len(lens) * news
    q = torch.randn(n, 16, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(n, 16, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, len(lens), news, 16, 2, 128), dtype=torch.uint8, device=DEV)
    cu = i32(starts([news] * len(lens)))

    def run():
        qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, q, out, 0.1, news, lse=lse, workspace=ws)
        torch.cuda.synchronize()

    run()
    want = out.clone(), lse.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    try:
        for limit in (1, 300, 1000, 2000, 4000, 8000, 12000, 20000, 30000):
            qsa.set_wait_options(status, limit)
            for _ in range(3):
                status.zero_()
                out.fill_(3.0)
                run()
                same = (out == want[0]).all(-1) & (lse == want[1])
                lost = torch.isnan(out.float()).all(-1) & torch.isnan(lse)
                assert (same | lost).all()
                assert int(status.item()) == 4 or same.all()
    finally:
        qsa.set_wait_options(None, qsa.QSA_WAIT_DEFAULT_NS)
    run()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("H_q,H,d,q_dtype", [(16, 2, 128, BF16), (16, 2, 128, F32), (6, 2, 72, BF16)])
@pytest.mark.parametrize("news", [1, 60])
def test_lengths_that_cannot_be(news, H_q, H, d, q_dtype):
    """The largest length there is, a negative one and a right one, in every kernel: NaN, zeros, the result."""
    pool = Pool([300, 200, 100], H, d, 64, BF16, seed=33)
    n = 3 * news
    q = torch.randn(n, H_q, d, device=DEV).to(q_dtype)
    out, lse = torch.full_like(q, -7.0), torch.full((n, H_q), -7.0, device=DEV)
    ws = torch.zeros(max(16, qsa.paged_attn_workspace_size(n, 3, news, H_q, H, d)), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32(starts([news] * 3)), i32([2 ** 31 - 1, -2 ** 31, 100]), q, out, 0.1, news,
                   lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isnan(out[:news].float()).all() and torch.isnan(lse[:news]).all()
    assert (out[news:2 * news] == 0).all() and torch.isneginf(lse[news:2 * news]).all()
    a = 2 * news
    check_attention(out[a:].double().cpu().numpy(), lse[a:].double().cpu().numpy(), q[a:].double().cpu().numpy(), pool.k[2],
                    pool.v[2], 100 - news, 0.1, True, q_dtype, BF16)
