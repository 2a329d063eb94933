"""The paged cache (write, read), the attention over it, the attention of packed prompts and the
draft verification, against the 64-bit forms of dense_reference.

Tolerances.  With A = sum_j softmax_j |v_j| (computed in 64 bits), an output is off by at most
  A * (2 * ds + (n + 64) * 2^-24)      fp32 sums over d dims and n cells, ds the logits' error
  + A * 2^-8                           weights rounded to bf16 (the tensor-core forms for bf16
                                       queries: bf16 cells at any number of rows, e4m3 cells at
                                       many; with few rows on e4m3 cells they are fp16, 2^-11)
  + 2^-25 * max_j(softmax_j u_j) * sum_j |v_j| / u_j     fp16 weights below fp16's normal range:
                                       on e4m3 cells a weight multiplies the code v_j / u_j,
                                       u_j = 2^e_j, so it carries u_j; its unit is no larger than
                                       the row's largest softmax_j u_j (the kernel's reference is
                                       some cell's own value), and fp16's spacing there is at most
                                       2^-24 of the unit, half of it the rounding
  + 2^-8 |out|                         the bf16 output's own rounding
with ds = (d + 16) * 2^-24 * scale * max sum|q||k| (d products summed in fp32, a scaling and the
exponential's few units in the last place)."""
import math

import numpy as np
import pytest
import torch

import dense_reference as ref
import gather_qsa_pool_gb300 as qsa

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int)


class Pool:
    """A paged cache of the given type whose sequences hold `lens` cells of normal values; the
    values as stored (64 bits) in self.k[s], self.v[s].  Every row that belongs to no cell is
    NaN."""

    def __init__(self, lens, H, d, page, dtype, seed, spare=2, pad_k=0, extra_cols=1):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.d, self.page = lens, H, d, page
        counts = [-(-n // page) for n in lens]
        n_pages = sum(counts) + spare
        order = rng.permutation(n_pages)
        width = max(counts + [0]) + extra_cols
        table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for i, c in enumerate(counts):
            table[i, :c] = order[at:at + c]
            at += c
        self.table = i32(table)
        rows = n_pages * page
        K = torch.full((rows, H * d + pad_k), float("nan"), device=DEV)
        V = torch.full((rows, H * d), float("nan"), device=DEV)
        self.k, self.v, self.units = [], [], []
        for i, n in enumerate(lens):
            r = self.rows(table[i], np.arange(n))
            x = rng.standard_normal((2, n, H, d)).astype(np.float32)
            K[r, :H * d] = torch.from_numpy(x[0].reshape(n, H * d)).to(DEV)
            V[r] = torch.from_numpy(x[1].reshape(n, H * d)).to(DEV)
        Ke = Ve = None
        if dtype == E4M3:
            # codes of normal values at exponents that differ from row to row
            Ke = torch.from_numpy(rng.integers(118, 127, (rows, H)).astype(np.uint8)).to(DEV)
            Ve = torch.from_numpy(rng.integers(118, 127, (rows, H)).astype(np.uint8)).to(DEV)
            K, V = (64 * K).to(E4M3), (64 * V).to(E4M3)
        else:
            K, V = K.to(dtype), V.to(dtype)
        self.K, self.V, self.Ke, self.Ve = K[:, :H * d].view(rows, H, d) if pad_k == 0 else \
            K[:, :H * d].unflatten(1, (H, d)), V.view(rows, H, d), Ke, Ve
        self.cache = qsa.PagedCache(self.K, self.V, page, K_exp=Ke, V_exp=Ve)
        for i, n in enumerate(lens):
            k, v = self.values(i, np.arange(n))
            self.k.append(k)
            self.v.append(v)
            if dtype == E4M3:
                e = Ve[self.rows(table[i], np.arange(n))].cpu().numpy().astype(float) - 127
                self.units.append(2.0 ** e)
            else:
                self.units.append(None)
        self.kv_len = i32(lens)

    def rows(self, table_row, pos):
        return torch.from_numpy(np.asarray(table_row)[pos // self.page].astype(np.int64) * self.page
                                + pos % self.page).to(DEV)

    def values(self, i, pos):
        """Stored values of cells, 64 bits."""
        r = self.rows(self.table[i].cpu().numpy(), np.asarray(pos))
        out = []
        for x, e in ((self.K, self.Ke), (self.V, self.Ve)):
            if e is None:
                out.append(x[r].double().cpu().numpy())
            else:
                c = x.view(torch.uint8)[r].cpu().numpy()
                out.append(ref.e4m3_values()[c] * 2.0 ** (e[r].cpu().numpy().astype(float) - 127)[..., None])
        return out


def tolerance(q, k, v, first, scale, causal, want, q_dtype, kv_dtype, units=None):
    n, d = max(k.shape[0], 1), q.shape[-1]
    A = ref.attend(q, k, np.abs(v), first, scale, causal)[0]
    qk = np.abs(q).sum(-1).max() * (np.abs(k).max() if k.size else 0.0)
    qk = min(qk, np.sqrt((q ** 2).sum(-1).max()) * (np.sqrt((k ** 2).sum(-1).max()) if k.size else 0))
    ds = (d + 16) * 2.0 ** -24 * abs(scale) * qk * 2  # sum|q||k| <= |q||k| (2: cancellation inside)
    rel = 2 * ds + (n + 64) * 2.0 ** -24
    if q_dtype == BF16:
        rel += 2.0 ** -8
    if kv_dtype == E4M3 and k.shape[0]:
        if units is None:  # rows as the cache writes them
            top = np.abs(v).max(-1)
            units = 2.0 ** np.clip(np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0)), -100, 100)
        A = A + 2.0 ** -25 / rel * small_weights(q, k, v, units, first, scale, causal)
    tol = A * rel + (2.0 ** -8 * np.abs(want) if q_dtype == BF16 else 0.0) + 1e-30
    return tol, ds + (n + 64) * 2.0 ** -24


def small_weights(q, k, v, units, first, scale, causal):
    """max_j(softmax_j u_j) * sum_j |v_j| / u_j over the cells each row sees."""
    m, H_q, d = q.shape
    n, H_kv = k.shape[:2]
    out = np.zeros((m, H_q, d))
    for h in range(H_q):
        g = h * H_kv // H_q
        s = scale * (q[:, h] @ k[:, g].T)
        if causal:
            s = np.where(np.arange(n)[None] > first + np.arange(m)[:, None], -np.inf, s)
        top = s.max(-1, keepdims=True)
        p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
        p = p / np.maximum(p.sum(-1, keepdims=True), 1e-300)
        codes = (p > 0).astype(float) @ (np.abs(v[:, g]) / units[:, g, None])
        out[:, h] = (p * units[None, :, g]).max(-1, keepdims=True) * codes
    return out


def check_attention(got, lse, q, k, v, first, scale, causal, q_dtype, kv_dtype, units=None):
    if q.shape[0] == 0:
        return
    want, wl = ref.attend(q, k, v, first, scale, causal)
    tol, tl = tolerance(q, k, v, first, scale, causal, want, q_dtype, kv_dtype, units)
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"out off by {err.max():.3g}, {(err / tol).max():.3g} of the bound"
    seen = np.isfinite(wl)
    np.testing.assert_array_equal(np.isneginf(lse), ~seen)
    assert (np.abs(lse[seen] - wl[seen]) <= tl + 2.0 ** -22 * np.abs(wl[seen])).all()


def run_paged(pool, news, H_q, q_dtype, seed, causal=True, pad=3, max_q=None, scale=None, ld_pad=0,
              stream=None):
    """paged_attn on queries of `news` tokens a sequence and `pad` tokens behind the last; checks
    every sequence and that nothing behind them was written."""
    d = pool.d
    scale = 1 / math.sqrt(d) if scale is None else scale
    rng = np.random.default_rng(seed)
    cu = starts(news)
    n = cu[-1] + pad
    qf = torch.from_numpy(rng.standard_normal((n, H_q * d + ld_pad)).astype(np.float32)).to(DEV).to(q_dtype)
    q = qf[:, :H_q * d].unflatten(1, (H_q, d))
    out = torch.full((n, H_q, d), -7.0, dtype=q_dtype, device=DEV)
    lse = torch.full((n, H_q), -7.0, device=DEV)
    mq = max(news) if max_q is None else max_q
    ws = torch.full((max(qsa.paged_attn_workspace_size(n, len(news), mq, H_q, pool.H, d), 16),), 255,
                    dtype=torch.uint8, device=DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    qsa.paged_attn(pool.cache, pool.table, i32(cu), pool.kv_len, q, out, scale, max(mq, 1),
                   causal=causal, lse=lse, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    o, l, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for s, m in enumerate(news):
        a, b = cu[s], cu[s + 1]
        check_attention(o[a:b], l[a:b], qn[a:b], pool.k[s], pool.v[s], pool.lens[s] - m, scale,
                        causal, q_dtype, {v: k for k, v in {BF16: 1, F32: 0, E4M3: 2}.items()}.get(
                            pool.cache._struct.dtype), pool.units[s])
    assert (o[cu[-1]:] == -7).all() and (l[cu[-1]:] == -7).all()
    return out, lse


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("src", [BF16, F32])
@pytest.mark.parametrize("dtype", [E4M3, BF16, F32])
@pytest.mark.parametrize("H,d,page", [(4, 128, 64), (1, 8, 8), (3, 72, 16), (2, 256, 128)])
def test_write_then_read(src, dtype, H, d, page):
    """Appends of 0, 1, many tokens and whole sequences; rows of other cells, and exponents of
    other rows, stay as they were; then the cells are read back by range and by list."""
    lens, news = [1, 37, 0, 300, page, 5], [1, 5, 0, 300, 1, 0]
    pool = Pool(lens, H, d, page, dtype, seed=5)
    rng = np.random.default_rng(11)
    n = sum(news)
    x = rng.standard_normal((2, n + 2, H, d)).astype(np.float32) * np.exp(rng.uniform(-8, 8, (2, n + 2, H, 1))).astype(np.float32)
    x[0, 0, 0, :] = 0.0
    x[1, 1, H - 1, 0] = np.nan
    x[1, 1, H - 1, 1] = -np.inf
    x[0, 2, 0, :3] = [448.0, -448.0, 448.0]
    k, v = torch.from_numpy(x[0]).to(DEV).to(src), torch.from_numpy(x[1]).to(DEV).to(src)
    before = [t.view(torch.uint8).clone() if t is not None else None for t in (pool.K, pool.V, pool.Ke, pool.Ve)]
    cu = starts(news)
    qsa.paged_write(pool.cache, pool.table, i32(cu), pool.kv_len, k, v)
    torch.cuda.synchronize()
    written = torch.zeros(pool.K.shape[0], dtype=torch.bool, device=DEV)
    for s, m in enumerate(news):
        pos = np.arange(lens[s] - m, lens[s])
        written[pool.rows(pool.table[s].cpu().numpy(), pos)] = True
        gk, gv = pool.values(s, pos)
        for got, src_t in ((gk, k), (gv, v)):
            want = src_t[cu[s]:cu[s + 1]].double().cpu().numpy()
            if dtype == E4M3:
                for i in range(m):
                    for h in range(H):
                        c, e = ref.encode_row(want[i, h])
                        np.testing.assert_array_equal(got[i, h], c * 2.0 ** e)
            else:
                cast = torch.from_numpy(want).float().to(dtype).double().numpy()
                np.testing.assert_array_equal(got, cast)
    for t, b in zip((pool.K, pool.V, pool.Ke, pool.Ve), before):
        if t is not None:
            assert torch.equal(t.view(torch.uint8)[~written], b[~written])
    # read back: by range, and by list with seq
    most = max(lens) + 2
    for out_t in (BF16, F32):
        K_out = torch.full((len(lens), most, H, d), -3.0, dtype=out_t, device=DEV)
        V_out = torch.full_like(K_out, -3.0)
        qsa.paged_read(pool.cache, pool.table, pool.kv_len, pool.kv_len, most, K_out, V_out)
        torch.cuda.synchronize()
        for s, m in enumerate(lens):
            for got, want in zip((K_out, V_out), pool.values(s, np.arange(m))):
                w = torch.from_numpy(want).float().to(out_t).double().numpy()
                np.testing.assert_array_equal(got[s, :m].double().cpu().numpy(), w)
                assert (got[s, m:] == -3).all()


def test_read_by_list_cells_outside_and_long_lists():
    pool = Pool([100, 40], 2, 64, 16, E4M3, seed=1)
    pos = np.array([[99, 0, 50, 100, -1, 7], [3, 39, 40, 2, 1, 0], [98, 97, 96, 95, 94, 93]], np.int32)
    seq, n = [0, 1, 0], [6, 4, 9]   # the last list is longer than its 6 entries
    K = torch.full((3, 6, 2, 64), -3.0, device=DEV)
    V = torch.full_like(K, -3.0)
    qsa.paged_read(pool.cache, pool.table, pool.kv_len, i32(n), 6, K, V, pos=i32(pos), seq=i32(seq))
    for i in range(3):
        for j in range(6):
            p, s = pos[i, j], seq[i]
            for got, all_ in ((K, pool.k), (V, pool.v)):
                g = got[i, j].double().cpu().numpy()
                if j >= n[i]:
                    assert (g == -3).all()
                elif 0 <= p < pool.lens[s]:
                    np.testing.assert_array_equal(g, all_[s][p])
                else:
                    assert (g == 0).all()
    # a sequence that does not exist, and a page that is not in the pool
    pool.table[1, 0] = 10 ** 6
    qsa.paged_read(pool.cache, pool.table, pool.kv_len, i32([1, 1, 1]), 6, K, V, pos=i32(pos), seq=i32([2, -1, 1]))
    assert (K[:, 0] == 0).all() and (V[:, 0] == 0).all()


def test_write_skips_cells_without_a_page():
    pool = Pool([70, 10], 2, 64, 32, BF16, seed=2)
    table = pool.table.clone()
    table[0, 1] = -1                       # cells 32 .. 63 have no page
    table[1, 0] = pool.cache.n_pages       # nor has sequence 1
    before = pool.K.clone()
    k = torch.ones(80, 2, 64, dtype=BF16, device=DEV)
    # sequence 1 "appends" 12 tokens to 10 cells: two positions are negative
    qsa.paged_write(pool.cache, table, i32([0, 68, 80]), pool.kv_len, k, k)
    torch.cuda.synchronize()
    now = pool.K
    t0 = pool.table[0].cpu().numpy()
    kept = pool.rows(t0, np.r_[0:2, 32:64])
    gone = pool.rows(t0, np.r_[2:32, 64:70])
    assert torch.equal(now[kept], before[kept]) and (now[gone] == 1).all()
    other = torch.ones(now.shape[0], dtype=torch.bool, device=DEV)
    other[gone] = False
    assert torch.equal(now[other].view(torch.int16), before[other].view(torch.int16))


# ------------------------------------------------------------------ paged attention

SHAPES = [
    # lens, news, H_q, H, d, page
    ([2050], [1], 8, 2, 128, 64),
    ([1, 7, 64, 65, 129, 0, 1000], [1, 1, 1, 1, 1, 0, 1], 32, 4, 128, 16),
    ([700, 33, 4, 260], [4, 4, 4, 1], 32, 4, 128, 64),          # drafts; one sequence of drafts only
    ([3, 50], [4, 4], 8, 1, 128, 8),                            # more new tokens than cells
    ([500, 90], [70, 90], 8, 2, 128, 32),                       # a chunk and a whole prompt
    ([257, 1], [200, 1], 12, 4, 128, 128),                      # three heads a KV head
    ([130], [130], 2, 2, 128, 64),                              # one head a KV head
    ([90, 17], [3, 17], 10, 2, 64, 16),                         # d 64, five heads a KV head
    ([40, 21], [2, 5], 6, 2, 72, 8),                            # a head size of no kernel's own
    ([66], [9], 40, 2, 256, 16),                                # twenty heads a KV head
]


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3, F32])
@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_paged_attention(shape, q_dtype, kv_dtype):
    lens, news, H_q, H, d, page = SHAPES[shape]
    pool = Pool(lens, H, d, page, kv_dtype, seed=shape)
    run_paged(pool, news, H_q, q_dtype, seed=100 + shape)


@pytest.mark.parametrize("news", [[1, 1], [40, 3], [300, 129]])
@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_paged_attention_without_causal_mask(news, kv_dtype):
    pool = Pool([333, 129], 2, 128, 32, kv_dtype, seed=3)
    run_paged(pool, news, 16, BF16, seed=4, causal=False)


@pytest.mark.parametrize("news", [1, 4, 150])
@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
def test_max_q_chooses_the_kernel_only(news, kv_dtype):
    """A host that knows no better than 1, or that says far more than there is."""
    pool = Pool([200, 1300], 2, 128, 64, kv_dtype, seed=6)
    for mq in (1, 1000):
        run_paged(pool, [news, news], 16, BF16, seed=7, max_q=mq, pad=0)


@pytest.mark.parametrize("news", [1, 30])
def test_strided_queries_and_keys_other_stream(news):
    pool = Pool([90, 300], 2, 128, 16, BF16, seed=8, pad_k=64)
    run_paged(pool, [news, news], 16, BF16, seed=9, ld_pad=40, stream=torch.cuda.Stream())


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 4, 60])
def test_large_logits_and_scales(news, kv_dtype):
    """Logits of hundreds (one key takes all the weight), and a scale of zero (the mean)."""
    pool = Pool([150, 700], 2, 128, 32, kv_dtype, seed=10)
    run_paged(pool, [news, news], 16, BF16, seed=11, scale=8.0)
    run_paged(pool, [news, news], 16, BF16, seed=12, scale=0.0)


@pytest.mark.parametrize("news", [1, 4, 7, 60])
@pytest.mark.parametrize("q_dtype", [BF16, F32])
def test_exponents_far_apart(news, q_dtype):
    """e4m3 values whose rows' exponents span the whole range, all the large ones in one part of
    the sequence, and rows of zeros (the smallest exponent)."""
    pool = Pool([300, 700], 2, 128, 32, E4M3, seed=20)
    rng = np.random.default_rng(21)
    for s in (0, 1):
        rows = pool.rows(pool.table[s].cpu().numpy(), np.arange(pool.lens[s]))
        e = rng.choice([27, 60, 90, 120, 127, 150], (len(rows), 2))
        e[200:] = rng.choice([27, 127, 200, 227], (len(rows) - 200, 2)) if s else e[200:]
        pool.Ve[rows] = torch.from_numpy(e.astype(np.uint8)).to(DEV)
        pool.V.view(torch.uint8)[rows[10:20]] = 0
        pool.v[s] = pool.values(s, np.arange(pool.lens[s]))[1]
        pool.units[s] = 2.0 ** (e.astype(float) - 127)
    run_paged(pool, [news, news], 16, q_dtype, seed=22)


def test_every_code_comes_back_exactly():
    """One cell: the output is its value, for each of the 256 codes, whichever kernel runs."""
    for news, ex in ((1, 127), (3, 40), (40, 127), (40, 215), (40, 27)):
        K = torch.zeros(2 * 8, 1, 128, device=DEV).to(E4M3)
        V = torch.zeros(2 * 8, 1, 128, dtype=torch.uint8, device=DEV)
        V[0, 0], V[8, 0] = torch.arange(128, device=DEV), torch.arange(128, 256, device=DEV)
        e = torch.full((16, 1), ex, dtype=torch.uint8, device=DEV)
        cache = qsa.PagedCache(K, V.view(E4M3), 8, K_exp=e, V_exp=e)
        q = torch.randn(2 * news, 4, 128, device=DEV).to(BF16)
        out = torch.zeros_like(q)
        ws = torch.zeros(max(16, qsa.paged_attn_workspace_size(2 * news, 2, news, 4, 1, 128)), dtype=torch.uint8, device=DEV)
        qsa.paged_attn(cache, i32([[0], [1]]), i32([0, news, 2 * news]), i32([1, 1]), q, out, 0.1, news, causal=False, workspace=ws)
        want = ref.e4m3_values() * 2.0 ** (ex - 127)
        got = out.double().cpu().numpy()
        for s in (0, 1):
            for i in (0, news - 1):
                for h in range(4):
                    np.testing.assert_array_equal(got[s * news + i, h], want[128 * s:128 * s + 128])


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 4, 60])
def test_negative_scale(news, kv_dtype):
    pool = Pool([150, 300], 2, 128, 32, kv_dtype, seed=23)
    run_paged(pool, [news, news], 16, BF16, seed=24, scale=-0.2)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("news", [1, 5, 100])
def test_a_page_outside_the_pool_gives_nan(news, kv_dtype):
    pool = Pool([400, 220, 300], 2, 128, 32, kv_dtype, seed=13)
    table = pool.table.clone()
    table[1, 2] = pool.cache.n_pages  # a page of the second sequence
    lens = pool.kv_len.clone()
    lens[2] = 32 * table.shape[1] + 1  # longer than its row of the table
    n = 3 * news
    q = torch.randn(n, 16, 128, device=DEV).to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(n, 16, device=DEV)
    ws = torch.zeros(max(16, qsa.paged_attn_workspace_size(n, 3, news, 16, 2, 128)), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, table, i32(starts([news] * 3)), lens, q, out, 0.1, news, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:news].float()).all() and torch.isfinite(lse[:news]).all()
    assert torch.isnan(out[news:].float()).all() and torch.isnan(lse[news:]).all()


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_cells_not_seen_do_not_matter(bad, kv_dtype):
    """NaN or infinities in the keys and values of later tokens reach only the tokens that see
    them; rows of the last page behind the sequence hold NaN in every test here."""
    if kv_dtype == E4M3 and math.isinf(bad):
        pytest.skip("e4m3 has no infinities")
    lens, news = [300, 77], [140, 77]
    pool = Pool(lens, 2, 128, 32, kv_dtype, seed=14)
    t = pool.table.cpu().numpy()
    hit = {0: 220, 1: 40}  # cells: token 60 of the chunk, token 40 of the prompt
    for s, p in hit.items():
        r = pool.rows(t[s], np.array([p]))
        if kv_dtype == E4M3:
            pool.K.view(torch.uint8)[r, :, 3], pool.V.view(torch.uint8)[r, :, 5] = 0x7f, 0x7f
        else:
            pool.K[r, :, 3], pool.V[r, :, 5] = bad, bad
    cu = starts(news)
    q = torch.randn(cu[-1], 16, 128, device=DEV).abs().to(BF16)
    out, lse = torch.zeros_like(q), torch.zeros(cu[-1], 16, device=DEV)
    ws = torch.zeros(max(16, qsa.paged_attn_workspace_size(int(cu[-1]), 2, 140, 16, 2, 128)), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32(cu), pool.kv_len, q, out, 0.1, 140, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    o, l, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for s in (0, 1):
        a, first = cu[s], lens[s] - news[s]
        clean = hit[s] - first  # tokens before it do not see the cell
        check_attention(o[a:a + clean], l[a:a + clean], qn[a:a + clean], pool.k[s][:hit[s]], pool.v[s][:hit[s]],
                        first, 0.1, True, BF16, kv_dtype, None if kv_dtype == BF16 else pool.units[s][:hit[s]])
        assert np.isnan(o[a + clean:cu[s + 1]]).all()


def test_rows_beyond_32_bits():
    """Pages whose elements and bytes lie past 2^32."""
    page, H, d, ld = 64, 2, 128, 8192
    n_pages = (1 << 32) // (ld * page) + 4
    K = torch.empty(n_pages * page, ld, dtype=BF16, device=DEV)
    V = torch.empty(n_pages * page, ld, dtype=BF16, device=DEV)
    Kv, Vv = K[:, :H * d].unflatten(1, (H, d)), V[:, :H * d].unflatten(1, (H, d))
    cache = qsa.PagedCache(Kv, Vv, page)
    table = i32([[n_pages - 1, 0, n_pages - 3]])
    n = 150
    x = torch.randn(2, n, H, d, device=DEV).to(BF16)
    qsa.paged_write(cache, table, i32([0, n]), i32([n]), x[0], x[1])
    for news in (2, 150):
        q = torch.randn(news, 16, d, device=DEV).to(BF16)
        out, lse = torch.zeros_like(q), torch.zeros(news, 16, device=DEV)
        ws = torch.zeros(max(16, qsa.paged_attn_workspace_size(news, 1, news, 16, H, d)), dtype=torch.uint8, device=DEV)
        qsa.paged_attn(cache, table, i32([0, news]), i32([n]), q, out, 0.1, news, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        k, v = x.double().cpu().numpy()
        check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy(), k, v,
                        n - news, 0.1, True, BF16, BF16)
    K_out = torch.zeros(1, n, H, d, dtype=BF16, device=DEV)
    V_out = torch.zeros_like(K_out)
    qsa.paged_read(cache, table, i32([n]), i32([n]), n, K_out, V_out)
    assert torch.equal(K_out[0], x[0]) and torch.equal(V_out[0], x[1])


# ------------------------------------------------------------------ prompts

PROMPTS = [
    ([777], 8, 2, 128), ([1], 32, 4, 128), ([300, 1, 0, 129, 128, 33], 32, 4, 128), ([64, 200], 4, 4, 128),
    ([513, 255], 6, 2, 128), ([150, 90], 10, 2, 64), ([70, 31], 4, 1, 40), ([40], 4, 2, 256), ([100, 260], 40, 1, 128),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompt_attention(case, causal, dtype):
    lens, H_q, H, d = PROMPTS[case]
    rng = np.random.default_rng(case)
    cu = starts(lens)
    n = cu[-1] + 2  # two tokens behind the last sequence

    def draw(h, pad):
        x = torch.from_numpy(rng.standard_normal((n, h * d + pad)).astype(np.float32)).to(DEV).to(dtype)
        x[cu[-1]:] = float("nan")
        return x[:, :h * d].unflatten(1, (h, d))

    q, k, v = draw(H_q, 8), draw(H, 16), draw(H, 0)
    out = torch.full((n, H_q, d), -7.0, dtype=dtype, device=DEV)
    lse = torch.full((n, H_q), -7.0, device=DEV)
    scale = 1 / math.sqrt(d)
    ws = torch.full((max(16, qsa.prompt_attn_workspace_size(n, len(lens), H_q, H, d)),), 255, dtype=torch.uint8, device=DEV)
    qsa.prompt_attn(q, k, v, i32(cu), out, scale, causal=causal, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    qn, kn, vn = (x.double().cpu().numpy() for x in (q, k, v))
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for a, b in zip(cu, cu[1:]):
        check_attention(o[a:b], l[a:b], qn[a:b], kn[a:b], vn[a:b], 0, scale, causal, dtype, dtype)
    assert (o[cu[-1]:] == -7).all() and (l[cu[-1]:] == -7).all()


def test_a_sequence_of_nan_stays_alone():
    """Packed neighbours share tiles; what one holds does not reach the other."""
    lens, H_q, H, d = [100, 60, 200], 8, 2, 128
    cu = starts(lens)
    q, k, v = (torch.randn(cu[-1], h, d, device=DEV).to(BF16) for h in (H_q, H, H))
    for x in (q, k, v):
        x[100:160] = float("nan")
    out, lse = torch.zeros_like(q), torch.zeros(cu[-1], H_q, device=DEV)
    ws = torch.zeros(max(16, qsa.prompt_attn_workspace_size(int(cu[-1]), 3, H_q, H, d)), dtype=torch.uint8, device=DEV)
    qsa.prompt_attn(q, k, v, i32(cu), out, 0.1, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    for a, b in ((0, 100), (160, 360)):
        x = [t[a:b].double().cpu().numpy() for t in (out, lse, q, k, v)]
        check_attention(*x, 0, 0.1, True, BF16, BF16)
    assert torch.isnan(out[100:160].float()).all()


def test_counts_beyond_the_buffers_touch_nothing_else():
    """cu_seq that runs past the buffers, or back, is clipped to them."""
    q = torch.randn(40, 4, 128, device=DEV).to(BF16)
    k = torch.randn(40, 2, 128, device=DEV).to(BF16)
    big = torch.full((60, 4, 128), -7.0, dtype=BF16, device=DEV)
    ws = torch.zeros(max(16, qsa.prompt_attn_workspace_size(40, 3, 4, 2, 128)), dtype=torch.uint8, device=DEV)
    qsa.prompt_attn(q, k, k, i32([0, 10, 5, 90]), big[:40], 0.1, workspace=ws)
    qsa.prompt_attn(q, k, k, i32([-5, 10, 2 ** 31 - 1, 20]), big[:40], 0.1, workspace=ws)
    torch.cuda.synchronize()
    assert (big[40:] == -7).all()


# ------------------------------------------------------------------ draft verification

@pytest.mark.parametrize("n,D,V,greedy", [(1, 3, 50257, False), (5, 4, 1000, False), (3, 0, 300, False), (2, 1, 1, False),
                                          (70, 2, 4096, False), (4, 7, 129, True), (200, 40, 64, False),
                                          (2, 3, 131072, True), (9, 5, 17, False)])
def test_draft_verify(n, D, V, greedy):
    rng = np.random.default_rng(n + D + V)
    for trial in range(4):
        logits = 2 * rng.standard_normal((n, D + 1, V))
        p = np.exp(logits) / np.exp(logits).sum(-1, keepdims=True)
        other = logits[:, :D] + (0.0 if trial == 3 else 0.5) * rng.standard_normal((n, D, V))
        q = np.exp(other) / np.exp(other).sum(-1, keepdims=True) if D else np.zeros((n, 0, V))
        p, q = p.astype(np.float32), q.astype(np.float32)
        tokens = np.zeros((n, D), np.int32)
        for s in range(n):
            for j in range(D):
                tokens[s, j] = other[s, j].argmax() if greedy else rng.choice(V, p=q[s, j].astype(float) / q[s, j].astype(float).sum())
        u = rng.random((n, D + 1)).astype(np.float32)
        u[u == 1.0] = 0.5
        if trial == 1:
            u[:, D] = 0.0
        if trial == 2:
            u[:, D] = 1.0 - 2.0 ** -24
            if D:
                tokens[rng.random((n, D)) < 0.2] = V  # outside the vocabulary
        nd = rng.integers(-1, D + 2, n).astype(np.int32)
        dev = [torch.from_numpy(x).to(DEV) for x in (p, q, tokens, u, nd)]
        out = torch.full((n, D + 1), -9, dtype=torch.int32, device=DEV)
        acc = torch.full((n,), -9, dtype=torch.int32, device=DEV)
        with_n = trial != 0
        qsa.draft_verify(dev[0], None if greedy else dev[1], dev[2], dev[3], out, acc, n_draft=dev[4] if with_n else None)
        for s in range(n):
            want, a = ref.verify(p[s], None if greedy else q[s], tokens[s], nd[s] if with_n else D, u[s])
            assert int(acc[s]) == a
            np.testing.assert_array_equal(out[s].cpu().numpy(), want)


def test_draft_verify_odd_rows_and_no_weight():
    V, D = 131, 2
    t = torch.zeros(3, D + 1, V + 6, device=DEV)[:, :, 1:V + 1]  # rows at an odd offset and stride
    d = torch.zeros(3, D, V + 2, device=DEV)[:, :, :V]
    t[0, 0, 7], d[0, 0, 7] = 1.0, 1.0       # taken for sure; then row 1 without any weight
    t[1, 0, 5], d[1, 0, 9] = 1.0, 1.0       # refused for sure: token 5
    t[2, 0, 130] = float("nan")
    t[2, 0, 129], d[2, 0, 3] = 0.5, 1.0     # NaN counts as nothing
    tokens = i32([[7, 1], [9, 0], [3, 0]])
    u = torch.full((3, D + 1), 0.5, device=DEV)
    out, acc = torch.zeros(3, D + 1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    qsa.draft_verify(t, d, tokens, u, out, acc)
    assert acc.tolist() == [1, 0, 0]
    assert out.tolist() == [[7, -1, -1], [5, -1, -1], [129, -1, -1]]


def test_draft_verify_equal_rows_fall_back_to_the_target():
    """p = q and a refusal (u above 1 cannot be, so a token outside the vocabulary): the
    difference is zero everywhere and the token comes from p."""
    V = 1000
    p = torch.softmax(torch.randn(1, 2, V, device=DEV), -1)
    out, acc = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    u = torch.tensor([[0.3, 0.6]], device=DEV)
    qsa.draft_verify(p, p[:, :1].contiguous(), i32([[V]]), u, out, acc)
    want, a = ref.verify(p[0].cpu().numpy(), p[0, :1].cpu().numpy(), [V], 1, u[0].cpu().numpy())
    assert int(acc[0]) == a == 0 and out[0].tolist() == want.tolist()


# ------------------------------------------------------------------ together

def test_a_server_step_end_to_end():
    """Two sequences through prompts, an 8-bit paged cache, a drafted step and its verification,
    eager and as one captured graph that replays after lengths and tokens changed in place; the
    selected cells of the cache also feed the sparse attention."""
    H_q, H, d, page, D, V = 16, 2, 128, 32, 3, 500
    lens = [150, 70]
    g = torch.Generator(device=DEV).manual_seed(1)

    def rand(*s):
        return torch.randn(*s, device=DEV, generator=g)

    cu = starts(lens)
    q, k, v = (rand(cu[-1], h, d).to(BF16) for h in (H_q, H, H))
    out, lse = torch.zeros_like(q), torch.zeros(cu[-1], H_q, device=DEV)
    scale = 1 / math.sqrt(d)
    ws = torch.zeros(max(16, qsa.prompt_attn_workspace_size(int(cu[-1]), 2, H_q, H, d)), dtype=torch.uint8, device=DEV)
    qsa.prompt_attn(q, k, v, i32(cu), out, scale, lse=lse, workspace=ws)
    n_pages = 16
    K = torch.zeros(n_pages * page, H, d, dtype=E4M3, device=DEV)
    V_ = torch.zeros_like(K)
    Ke = torch.full((n_pages * page, H), 27, dtype=torch.uint8, device=DEV)
    Ve = Ke.clone()
    cache = qsa.PagedCache(K, V_, page, K_exp=Ke, V_exp=Ve)
    table = torch.randperm(n_pages, device=DEV, generator=g).view(2, 8).int()
    kv_len = i32(lens)
    qsa.paged_write(cache, table, i32(cu), kv_len, k, v)

    # one step: D + 1 tokens a sequence
    m = D + 1
    cu_q = i32([0, m, 2 * m])
    kn, vn, qn = rand(2 * m, H, d).to(BF16), rand(2 * m, H, d).to(BF16), rand(2 * m, H_q, d).to(BF16)
    o, l = torch.zeros_like(qn), torch.zeros(2 * m, H_q, device=DEV)
    ws2 = torch.zeros(max(16, qsa.paged_attn_workspace_size(2 * m, 2, m, H_q, H, d)), dtype=torch.uint8, device=DEV)
    p = torch.softmax(2 * rand(2, m, V), -1)
    dr = torch.softmax(2 * rand(2, D, V), -1)
    toks = torch.randint(0, V, (2, D), device=DEV, generator=g).int()
    u = torch.rand(2, m, device=DEV, generator=g)
    t_out, acc = torch.zeros(2, m, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    kv_len += m

    def step():
        qsa.paged_write(cache, table, cu_q, kv_len, kn, vn)
        qsa.paged_attn(cache, table, cu_q, kv_len, qn, o, scale, m, lse=l, workspace=ws2)
        qsa.draft_verify(p, dr, toks, u, t_out, acc)

    def check():
        torch.cuda.synchronize()
        n = kv_len.tolist()
        Kr = torch.zeros(2, max(n), H, d, device=DEV)
        Vr = torch.zeros_like(Kr)
        qsa.paged_read(cache, table, kv_len, kv_len, max(n), Kr, Vr)
        for s in range(2):
            kk, vv = (x[s, :n[s]].double().cpu().numpy() for x in (Kr, Vr))
            # what was written last is what is read (a row within half a step of 4 bits, and the
            # smallest code's half beside the row's largest value)
            last = kn[s * m:(s + 1) * m].double().cpu().numpy()
            top = np.abs(last).max(-1, keepdims=True)
            assert (np.abs(kk[-m:] - last) <= 2.0 ** -4 * np.abs(last) + 2.0 ** -17 * top).all()
            a = s * m
            check_attention(o[a:a + m].double().cpu().numpy(), l[a:a + m].double().cpu().numpy(),
                            qn[a:a + m].double().cpu().numpy(), kk, vv, n[s] - m, scale, True, BF16, E4M3)
            want, w = ref.verify(p[s].cpu().numpy(), dr[s].cpu().numpy(), toks[s].cpu().numpy(), D, u[s].cpu().numpy())
            assert int(acc[s]) == w and t_out[s].tolist() == want.tolist()

    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(2):
        # rejected drafts are rolled back: the lengths follow the tokens that stood
        kv_len.copy_(kv_len - D + acc + m)
        for x in (kn, vn, qn):
            x.copy_(rand(*x.shape).to(BF16))
        u.copy_(torch.rand(2, m, device=DEV, generator=g))
        graph.replay()
        check()

    # the selection of a sparse step, read out of the pages and attended
    cells = 35
    pos = torch.stack([torch.randperm(n, device=DEV, generator=g)[:cells].sort().values for n in kv_len.tolist()]).int()
    n_cells = i32([cells, cells - 4])
    Kc = torch.zeros(2, cells, H, d, dtype=BF16, device=DEV)
    Vc = torch.zeros_like(Kc)
    qsa.paged_read(cache, table, kv_len, n_cells, cells, Kc, Vc, pos=pos)
    q1, o1 = rand(2, H_q, d), torch.zeros(2, H_q, d, device=DEV)
    ws3 = torch.zeros(max(16, qsa.sparse_attn_workspace_size(2, H_q, H, d, cells)), dtype=torch.uint8, device=DEV)
    qsa.sparse_attn(q1, Kc.view(-1, H * d), Vc.view(-1, H * d), n_cells, cells, o1, H, d, d, scale, workspace=ws3)
    torch.cuda.synchronize()
    for s in range(2):
        n = int(n_cells[s])
        want, _ = ref.attend(q1[s:s + 1].double().cpu().numpy(), Kc[s, :n].double().cpu().numpy(),
                             Vc[s, :n].double().cpu().numpy(), n - 1, scale)
        assert np.abs(o1[s:s + 1].double().cpu().numpy() - want).max() < 2e-3
