"""Appends, attention and sparse attention over paged caches as a server uses them together: prompts, then tokens and
drafts some of which are taken back, each step against the 64-bit forms over the cells as they are stored; calls that run
at the same time; captured graphs in turn and at once; cells that lie beyond 32 bits of offset; waits that run out."""
import math

import numpy as np
import pytest
import torch

import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from four_bit_pool import E2M1, Pool4, any_pool, kind_of
from test_gpu_append import append
from test_gpu_dense import BF16, DEV, E4M3, F32, check_attention, i32, starts
from test_gpu_paged_sparse import lists

pytestmark = pytest.mark.gpu


def workspace(n, seqs, max_q, H_q, H, d=128):
    return torch.full((max(16, qsa.paged_attn_workspace_size(n, seqs, max_q, H_q, H, d)),), 255, dtype=torch.uint8, device=DEV)


def units_of(pool, s, cells):
    if pool.units[s] is None:
        return None
    if pool.K.dtype == E2M1:
        return 2.0 ** (pool.Ve.cpu().numpy()[pool.np_rows(pool.table[s].cpu().numpy(), cells)].astype(float) - 127)
    return 2.0 ** (pool.Ve[pool.rows(pool.table[s].cpu().numpy(), cells)].cpu().numpy().astype(float) - 127)


# ------------------------------------------------------------------ a server's steps

class Index:
    """The keys by which blocks are scored, and their pooled rows, of each sequence."""
    H, d = 2, 64

    def __init__(self, caps, rng):
        self.rng = rng
        self.raw = [torch.zeros(c, self.H * self.d, device=DEV) for c in caps]
        self.pooled = [torch.zeros(-(-c // 4), self.H * self.d, device=DEV) for c in caps]
        self.norm = torch.ones(self.d, device=DEV)
        self.n = [0] * len(caps)

    def select(self, s, n, m, k_blk):
        """The last m of n cells of sequence s are new: their keys, and each one's blocks."""
        new = self.rng.standard_normal((m, self.H * self.d)).astype(np.float32)
        self.raw[s][n - m:n] = torch.from_numpy(new).to(DEV)
        keep = min(self.n[s], n - m) // 4  # complete blocks that stay
        qsa.pool_update(self.raw[s], n, self.H, self.d, self.norm, 1e-6, 10000.0, self.pooled[s], keep)
        self.n[s] = n
        rows, whole = -(-n // 4), n // 4
        q = torch.from_numpy(self.rng.standard_normal((m, self.H * self.d)).astype(np.float32)).to(DEV)
        pos = torch.arange(n - m, n, dtype=torch.int32, device=DEV)
        scores = torch.zeros(m, rows, device=DEV)
        qsa.index_score(q, self.pooled[s], rows, self.H, self.d, self.d ** -0.5, scores, q_pos=pos)
        blocks, counts = torch.full((m, k_blk), -5, dtype=torch.int32, device=DEV), torch.zeros(m, dtype=torch.int32, device=DEV)
        if whole:
            qsa.topk_blocks(scores, whole, k_blk, blocks, counts, q_pos=pos)
        return blocks, counts


@pytest.mark.parametrize("dtype", [E2M1, E4M3, BF16])
def test_prompts_tokens_and_drafts(dtype):
    H, H_q, d, k_blk, scale = 2, 16, 128, 24, 128 ** -0.5
    pool = any_pool([330, 140, 20], H, d, 16, dtype, seed=21)
    rng = np.random.default_rng(22)
    index = Index([340, 150, 30], rng)
    lens = [0, 0, 0]
    # prompts; tokens; three drafts and a token, of which the second sequence's last two and the third's three are
    # taken back; a sequence that is left out
    for turn, (news, back) in enumerate([([300, 111, 3], [0, 0, 0]), ([1, 1, 1], [0, 0, 0]), ([4, 4, 4], [0, 2, 3]), ([2, 0, 1], [0, 0, 0]),
                                         ([1, 1, 1], [0, 0, 0])]):
        lens = [a + b for a, b in zip(lens, news)]
        pool.lens, pool.kv_len = lens, i32(lens)
        n, cu = sum(news), starts(news)
        q, _ = append(pool, news, H_q, BF16, seed=30 + turn, pad=0, base=500.0)
        out, sparse = torch.zeros_like(q), torch.zeros_like(q)
        lse, sparse_lse = torch.zeros(n, H_q, device=DEV), torch.zeros(n, H_q, device=DEV)
        qsa.paged_attn(pool.cache, pool.table, i32(cu), pool.kv_len, q, out, scale, max(news), lse=lse, workspace=workspace(n, 3, max(news), H_q, H))
        listed = [index.select(s, lens[s], m, k_blk) for s, m in enumerate(news) if m]
        blocks, counts = (torch.cat(x) for x in zip(*listed))
        qsa.paged_sparse_attn(pool.cache, pool.table, i32(cu), pool.kv_len, blocks, counts, q, sparse, scale, lse=sparse_lse)
        torch.cuda.synchronize()
        o, l, so, sl, qn = (x.double().cpu().numpy() for x in (out, lse, sparse, sparse_lse, q))
        bl, ct = blocks.cpu().numpy(), counts.cpu().numpy()
        for s, m in enumerate(news):
            if not m:
                continue
            a, b = cu[s], cu[s + 1]
            k, v = pool.values(s, np.arange(lens[s]))
            units = units_of(pool, s, np.arange(lens[s]))
            check_attention(o[a:b], l[a:b], qn[a:b], k, v, lens[s] - m, scale, True, BF16, kind_of(dtype), units)
            for i in range(m):
                p = lens[s] - m + i
                assert ct[a + i] == min(k_blk, (p + 1) // 4)
                c = four.listed_cells(bl[a + i], ct[a + i], p)
                check_attention(so[a + i:a + i + 1], sl[a + i:a + i + 1], qn[a + i:a + i + 1], k[c], v[c], len(c) - 1, scale, False, BF16,
                                kind_of(dtype), None if units is None else units[c])
                if (p + 1) // 4 <= k_blk:
                    assert len(c) == p + 1  # every block is listed: the sparse result is the whole one's
        lens = [a - b for a, b in zip(lens, back)]


# ------------------------------------------------------------------ at the same time, and captured

def attn(lens, news, H_q, H, q_dtype, seed, page=64):
    pool = Pool4(lens, H, 128, page, seed=seed)
    cu, n = i32(starts(news)), sum(news)
    q = torch.randn(n, H_q, 128, device=DEV).to(q_dtype)
    out, lse, ws = torch.zeros_like(q), torch.zeros(n, H_q, device=DEV), workspace(n, len(lens), max(news), H_q, H)
    return (lambda: qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, q, out, 0.09, max(news), lse=lse, workspace=ws)), (out, lse)


def sparse(lens, news, H_q, H, dtype, q_dtype, k_blk, seed):
    pool = any_pool(lens, H, 128, 32, dtype, seed=seed)
    blocks, counts = (i32(x) for x in lists(pool, news, k_blk, seed))
    cu, n = i32(starts(news)), sum(news)
    q = torch.randn(n, H_q, 128, device=DEV).to(q_dtype)
    out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device=DEV)
    return (lambda: qsa.paged_sparse_attn(pool.cache, pool.table, cu, pool.kv_len, blocks, counts, q, out, 0.09, lse=lse)), (out, lse)


def store(lens, news, H_q, H, dtype, src, seed):
    pool = any_pool(lens, H, 128, 32, dtype, seed=seed)
    cu, n = i32(starts(news)), sum(news)
    q, k, v = (torch.randn(n, h, 128, device=DEV).to(src) for h in (H_q, H, H))
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    outs = [q_out, k_out, pool.K, pool.V] + [t for t in (pool.Ke, pool.Ve) if t is not None] + ([pool.Ks, pool.Vs] if dtype == E2M1 else [])
    return (lambda: qsa.paged_append(pool.cache, pool.table, cu, pool.kv_len, k, v, 10000.0, q=q, q_out=q_out, k_out=k_out)), outs


def calls():
    torch.manual_seed(4)
    return [
        attn([9000, 700, 1], [1, 1, 1], 32, 4, BF16, 1),           # few rows, cut and joined
        attn([60000], [1], 32, 4, BF16, 2),                       # in many parts: the join of its own
        attn([3000, 500], [4, 2], 16, 2, F32, 3),
        attn([3000, 1200], [200, 90], 16, 2, BF16, 4),             # chunks
        sparse([9000], [1], 32, 4, BF16, BF16, 512, 5),            # one token: clusters
        sparse([900] * 50, [2] * 50, 16, 2, E2M1, BF16, 60, 6),
        sparse([700, 300], [9, 4], 8, 1, E4M3, F32, 40, 7),
        store([400, 90], [300, 1], 8, 2, E2M1, BF16, 8),
        store([400, 90], [300, 1], 8, 2, E4M3, F32, 9),
    ]


def bits(outs):
    return [o.contiguous().view(torch.uint8).clone() for o in outs]


def wipe(outs):
    for o in outs:
        o.view(torch.uint8 if o.element_size() == 1 else o.dtype).fill_(5)


def settled(every):
    """Every call's results when it runs alone on wiped outputs."""
    want = []
    for call, outs in every:
        wipe(outs)
        call()
        torch.cuda.synchronize()
        want.append(bits(outs))
    return want


def test_on_streams_of_their_own():
    every = calls()
    want = settled(every)
    streams = [torch.cuda.Stream() for _ in every]
    for _ in range(4):
        for (call, outs), s in zip(every, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                wipe(outs)
                for _ in range(3):
                    call()
        torch.cuda.synchronize()
        for (_, outs), w in zip(every, want):
            assert all(torch.equal(a, b) for a, b in zip(bits(outs), w))


def test_graphs_in_turn_and_at_once():
    every = calls()
    want = settled(every)
    graphs = []
    for call, _ in every:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for at_once in (False, True):
        for _, outs in every:
            wipe(outs)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() if at_once else torch.cuda.current_stream() for _ in graphs]
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (_, outs), w in zip(every, want):
            assert all(torch.equal(a, b) for a, b in zip(bits(outs), w))


def test_one_graph_of_a_whole_step():
    """Append, attention and sparse attention captured together and replayed as the sequences grow: eager calls' bits."""
    pool = Pool4([900, 300], 2, 128, 32, seed=31)
    q, k, v = (torch.randn(2, h, 128, device=DEV).bfloat16() for h in (16, 2, 2))
    cu, kv_len = i32([0, 1, 2]), i32([890, 290])
    blocks, counts = i32(np.stack([np.arange(20), np.arange(20) * 2])), i32([20, 20])
    ws = [workspace(2, 2, 1, 16, 2) for _ in range(2)]
    held = (pool.K, pool.V, pool.Ke, pool.Ve, pool.Ks.view(torch.uint8), pool.Vs.view(torch.uint8))

    def step(t, w):
        qsa.paged_append(pool.cache, pool.table, cu, kv_len, k, v, 10000.0, q=q, q_out=t[0])
        qsa.paged_attn(pool.cache, pool.table, cu, kv_len, t[0], t[1], 0.09, 1, workspace=w)
        qsa.paged_sparse_attn(pool.cache, pool.table, cu, kv_len, blocks, counts, t[0], t[2], 0.09)

    mine, eager = ([torch.zeros_like(q) for _ in range(3)] for _ in range(2))
    step(mine, ws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(mine, ws[0])
    for i in range(9):
        kv_len += 1
        for x in (q, k, v):
            x.normal_()
        start = [t.clone() for t in held]
        step(eager, ws[1])
        want = [t.clone() for t in (*eager, *held)]
        for t, s in zip(held, start):
            t.copy_(s)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*mine, *held), want))


# ------------------------------------------------------------------ cells far into a pool

@pytest.mark.parametrize("dtype,rows", [(E2M1, 36_000_000), (E4M3, 18_000_000), (BF16, 9_000_000)])
def test_cells_beyond_32_bits(dtype, rows):
    """The last pages of pools of more than 2^32 bytes (codes of 36 million rows of 4 heads, 9.2 GB each for keys and
    values; bf16 values 2^33 bytes) give what the same pages give in a small pool, for every call."""
    H, d, page, lens = 4, 128, 64, [1500, 500]
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    small = any_pool(lens, H, d, page, dtype, seed=41)
    n_small = small.K.shape[0] // page
    n_pages = rows // page
    first = n_pages - n_small

    def grown(t, by_page):
        big = torch.empty((n_pages if by_page else n_pages * page, *t.shape[1:]), dtype=t.dtype, device=DEV)
        view = (lambda x: x.view(torch.uint8)) if t.element_size() == 1 else (lambda x: x)
        view(big)[first * (1 if by_page else page):] = view(t)
        return big

    tensors = dict(K=small.K, V=small.V, K_exp=small.Ke, V_exp=small.Ve)
    if dtype == E2M1:
        tensors.update(K_scale=small.Ks, V_scale=small.Vs)
    big = {x: None if t is None else grown(t, x.endswith("scale")) for x, t in tensors.items()}
    cache = qsa.PagedCache(big["K"], big["V"], page, K_exp=big["K_exp"], V_exp=big["V_exp"], **{x: big[x] for x in big if x.endswith("scale")})
    table = torch.where(small.table >= 0, small.table + first, small.table)
    for turn, news in enumerate(([1, 1], [3, 2], [200, 100])):
        n, cu = sum(news), i32(starts(news))
        g = torch.Generator(device=DEV).manual_seed(turn)
        q, k, v = (torch.randn(n, h, d, device=DEV, generator=g).bfloat16() for h in (32, H, H))
        blocks, counts = (i32(x) for x in lists(small, news, 100, turn))
        results = []
        for c, t, off in ((small.cache, small.table, 0), (cache, table, first)):
            q_out, out, listed = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
            qsa.paged_append(c, t, cu, small.kv_len, k, v, 10000.0, q=q, q_out=q_out)
            qsa.paged_attn(c, t, cu, small.kv_len, q_out, out, 0.09, max(news), workspace=workspace(n, 2, max(news), 32, H))
            qsa.paged_sparse_attn(c, t, cu, small.kv_len, blocks, counts, q_out, listed, 0.09)
            back = [torch.zeros(2, 1500, H, d, device=DEV) for _ in range(2)]
            qsa.paged_read(c, t, small.kv_len, small.kv_len, 1500, *back)
            results.append((q_out, out, listed, *back))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*results))
        assert torch.isfinite(results[0][1].float()).all()
        for x, t in tensors.items():
            if t is not None:
                at = first * (1 if x.endswith("scale") else page)
                a, b = (y.contiguous().view(torch.uint8) for y in (t, big[x][at:]))
                assert torch.equal(a, b)


# ------------------------------------------------------------------ batches of nothing

@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [E2M1, E4M3, BF16])
@pytest.mark.parametrize("max_q", [1, 200])
def test_padding_alone(dtype, q_dtype, max_q):
    """No sequence has a new token: nothing is written."""
    pool = any_pool([70, 0], 2, 128, 16, dtype, seed=61)
    cu, n = i32([0, 0, 0]), 5
    held = [t.clone() for t in (pool.K.view(torch.uint8) if dtype != BF16 else pool.K, pool.V.view(torch.uint8) if dtype != BF16 else pool.V)]
    q, k, v = (torch.randn(n, h, 128, device=DEV).to(q_dtype) for h in (8, 2, 2))
    outs = [torch.full_like(q, -7.0) for _ in range(3)]
    qsa.paged_append(pool.cache, pool.table, cu, pool.kv_len, k, v, 10000.0, q=q, q_out=outs[0])
    qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, q, outs[1], 0.09, max_q, workspace=workspace(n, 2, max_q, 8, 2))
    qsa.paged_sparse_attn(pool.cache, pool.table, cu, pool.kv_len, torch.zeros(n, 3, dtype=torch.int32, device=DEV),
                          torch.full((n,), 3, dtype=torch.int32, device=DEV), q, outs[2], 0.09)
    torch.cuda.synchronize()
    assert all((o == -7).all() for o in outs)
    now = (pool.K.view(torch.uint8), pool.V.view(torch.uint8)) if dtype != BF16 else (pool.K, pool.V)
    assert all(torch.equal(a.nan_to_num() if a.is_floating_point() else a, b.nan_to_num() if b.is_floating_point() else b) for a, b in zip(held, now))


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("news", [[2, 7], [1, 70]])
def test_tokens_before_the_first_cell(news, q_dtype):
    """More new tokens than cells: those at negative positions see nothing, give zero and -inf; the others as ever."""
    lens = [0, 5]
    pool = Pool4(lens, 2, 128, 16, seed=62)
    n, cu = sum(news), starts(news)
    q = torch.randn(n, 16, 128, device=DEV).to(q_dtype)
    blocks, counts = np.zeros((n, 4), np.int32), np.full(n, 1, np.int32)
    for listed in (False, True):
        out, lse = torch.full_like(q, -7.0), torch.full((n, 16), -7.0, device=DEV)
        if listed:
            qsa.paged_sparse_attn(pool.cache, pool.table, i32(cu), pool.kv_len, i32(blocks), i32(counts), q, out, 0.09, lse=lse)
        else:
            qsa.paged_attn(pool.cache, pool.table, i32(cu), pool.kv_len, q, out, 0.09, max(news), lse=lse, workspace=workspace(n, 2, max(news), 16, 2))
        torch.cuda.synchronize()
        o, l, qn = (x.double().cpu().numpy() for x in (out, lse, q))
        for s, m in enumerate(news):
            for i in range(m):
                t, p = cu[s] + i, lens[s] - m + i
                if p < 0:
                    assert (o[t] == 0).all() and np.isneginf(l[t]).all()
                else:
                    check_attention(o[t:t + 1], l[t:t + 1], qn[t:t + 1], pool.k[s][:p + 1], pool.v[s][:p + 1], p, 0.09, True, q_dtype, E4M3, pool.units[s][:p + 1])


# ------------------------------------------------------------------ waits that run out

def test_chunk_gives_up_and_recovers():
    """The tensor-core kernel over 4-bit cells with a limit of 0: every wait gives up without looking, the kernel says
    so, leaves NaN and returns; the next call is right again."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    call, (out, lse) = attn([5000, 300], [100, 40], 16, 2, BF16, 51)
    call()
    torch.cuda.synchronize()
    want = bits((out, lse))
    try:
        qsa.set_wait_options(status, 0)
        wipe((out, lse))
        call()
        torch.cuda.synchronize()
        assert int(status.item()) == 4
        assert torch.isnan(out.float()).all() and torch.isnan(lse).all()
        qsa.set_wait_options(status, qsa.QSA_WAIT_DEFAULT_NS)
        status.zero_()
        for _ in range(2):
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(bits((out, lse)), want))
        assert int(status.item()) == 0
    finally:
        qsa.set_wait_options(None, qsa.QSA_WAIT_DEFAULT_NS)
