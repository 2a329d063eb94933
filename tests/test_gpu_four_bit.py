"""The 4-bit paged cache: written, read back, and attended to by a few tokens, drafts and chunks, against the 64-bit
forms.  Codes, scales and exponents have to be equal (every rounding is to nearest, ties to even, of a correctly
rounded quotient); values read back are exact.  The attention's bound is test_gpu_dense's for rows of codes, with the
cells' powers of two as the units of the weights (a code times its scale is exact)."""
import math

import numpy as np
import pytest
import torch

import dense_reference as ref
import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from four_bit_pool import Pool4
from test_gpu_dense import BF16, DEV, E4M3, F32, check_attention, i32, starts

pytestmark = pytest.mark.gpu


def run_attn(pool, news, H_q, q_dtype, seed, causal=True, pad=3, max_q=None, scale=None, ld_pad=0, q_scale=1.0):
    d = pool.d
    scale = 1 / math.sqrt(d) if scale is None else scale
    rng = np.random.default_rng(seed)
    cu = starts(news)
    n = cu[-1] + pad
    qf = torch.from_numpy((q_scale * rng.standard_normal((n, H_q * d + ld_pad))).astype(np.float32)).to(DEV).to(q_dtype)
    q = qf[:, :H_q * d].unflatten(1, (H_q, d))
    out = torch.full((n, H_q, d), -7.0, dtype=q_dtype, device=DEV)
    lse = torch.full((n, H_q), -7.0, device=DEV)
    mq = max(max(news) if max_q is None else max_q, 1)
    ws = torch.full((max(qsa.paged_attn_workspace_size(n, len(news), mq, H_q, pool.H, d), 16),), 255, dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32(cu), pool.kv_len, q, out, scale, mq, causal=causal, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    o, l, qn = out.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for s, m in enumerate(news):
        a, b = cu[s], cu[s + 1]
        check_attention(o[a:b], l[a:b], qn[a:b], pool.k[s], pool.v[s], pool.lens[s] - m, scale, causal, q_dtype, E4M3, pool.units[s])
    assert (o[cu[-1]:] == -7).all() and (l[cu[-1]:] == -7).all()
    return out, lse


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("src", [BF16, F32])
@pytest.mark.parametrize("H,d,page", [(4, 128, 64), (1, 16, 8), (3, 80, 16), (2, 256, 128), (4, 64, 32)])
def test_write_then_read(src, H, d, page):
    """Appends of 0, 1, many tokens and whole sequences: rows as the format says, rows of other cells as they were;
    then the cells are read back by range and by list."""
    lens, news = [1, 37, 0, 300, page, 5], [1, 5, 0, 300, 1, 0]
    pool = Pool4(lens, H, d, page, seed=5, pad=32)
    rng = np.random.default_rng(11)
    n = sum(news)
    x = rng.standard_normal((2, n + 2, H, d)).astype(np.float32) * np.exp(rng.uniform(-12, 12, (2, n + 2, H, 1))).astype(np.float32)
    x[0, 0, 0, :] = 0.0
    x[1, 1, 0, ::3] *= 2.0 ** -12                      # scales that underflow
    x[0, 2, 0, 0], x[1, 3, 0, 1], x[1, 4, 0, 5] = np.nan, np.inf, -np.inf
    x[0, 5] = rng.integers(-12, 13, (H, d)) * 0.25      # ties: with a largest of 6 (and 3, 1.5) quotients of 1/4s
    x[0, 5, :, ::16] = 6.0
    x[0, 6], x[1, 7] = x[0, 6] * np.float32(1e36), x[1, 7] * np.float32(1e-36)
    src_t = torch.from_numpy(x).to(DEV).to(src)
    before = {c: [t.clone() for t in pair] for c, pair in (("K", (pool.K, pool.Ks, pool.Ke)), ("V", (pool.V, pool.Vs, pool.Ve)))}
    qsa.paged_write(pool.cache, pool.table, i32(starts(news)), pool.kv_len, src_t[0], src_t[1])
    torch.cuda.synchronize()
    stored = src_t.double().cpu().numpy()
    written = []
    at = 0
    for s, m in enumerate(news):
        r = pool.np_rows(pool.table[s].cpu().numpy(), np.arange(lens[s] - m, lens[s]))
        written.append(r)
        for is_v, (codes, scale, exp) in enumerate(((pool.K, pool.Ks, pool.Ke), (pool.V, pool.Vs, pool.Ve))):
            c = four.unpack(codes.cpu().numpy()[r])
            sc = scale.view(torch.uint8).cpu().numpy()[r // page, :, r % page]
            e = exp.cpu().numpy()[r]
            for t in range(m):
                for h in range(H):
                    wc, wsc, we = four.encode_row(stored[is_v, at + t, h])
                    np.testing.assert_array_equal(sc[t, h], wsc)
                    assert int(e[t, h]) == we + 127
                    got, want = four.values(c[t, h], sc[t, h], e[t, h]), four.values(wc, wsc, we + 127)
                    np.testing.assert_array_equal(got, want)
                    zero = (wsc == 0) | (wsc == 0x7f)
                    assert (c[t, h].reshape(-1, 16)[zero] == 0).all()
        at += m
    written = np.concatenate(written)
    rest = np.setdiff1d(np.arange(pool.K.shape[0]), written)
    for c, now in (("K", (pool.K, pool.Ks, pool.Ke)), ("V", (pool.V, pool.Vs, pool.Ve))):
        assert torch.equal(now[0][rest], before[c][0][rest]) and torch.equal(now[2][rest], before[c][2][rest])
        a, b = now[1].view(torch.uint8).cpu().numpy(), before[c][1].view(torch.uint8).cpu().numpy()
        np.testing.assert_array_equal(a[rest // page, :, rest % page], b[rest // page, :, rest % page])
    # ---- read back, whole and listed
    for out_t in (BF16, F32):
        most = max(lens)
        K, V = (torch.full((len(lens), most, H, d), -7.0, dtype=out_t, device=DEV) for _ in range(2))
        qsa.paged_read(pool.cache, pool.table, pool.kv_len, pool.kv_len, most, K, V)
        torch.cuda.synchronize()
        for s, m in enumerate(lens):
            k, v = pool.values(s, np.arange(m))
            for got, want in ((K, k), (V, v)):
                g = got[s].double().cpu().numpy()
                np.testing.assert_array_equal(g[:m], torch.from_numpy(want).to(out_t).double().numpy())
                assert (g[m:] == -7).all()
        pos = i32([[0, 299, 7, 300, -1, 123, 5, 1]])
        K, V = (torch.full((1, 8, H, d), -7.0, dtype=out_t, device=DEV) for _ in range(2))
        qsa.paged_read(pool.cache, pool.table, pool.kv_len, i32([7]), 8, K, V, pos=pos, seq=i32([3]))
        torch.cuda.synchronize()
        k, v = pool.values(3, np.array([0, 299, 7, 0, 0, 123, 5]))
        k[3:5] = v[3:5] = 0.0
        for got, want in ((K, k), (V, v)):
            np.testing.assert_array_equal(got[0, :7].double().cpu().numpy(), torch.from_numpy(want).to(out_t).double().numpy())
            assert (got[0, 7] == -7).all()


# ------------------------------------------------------------------ attention

SHAPES = [  # lens, news, H_q, H_kv, page
    ([1, 2, 31, 32, 33, 127, 128, 129, 257], [1] * 9, 8, 1, 8),
    ([4000, 5, 0, 700], [1, 1, 0, 1], 32, 4, 64),
    ([513, 64, 3, 1500], [4, 4, 3, 2], 32, 4, 16),
    ([90, 2, 700], [2, 1, 2], 4, 4, 32),
    ([2050], [1], 8, 2, 64),
    ([333, 41], [3, 1], 24, 2, 128),
    ([333, 41], [1, 1], 32, 1, 32),
    ([900, 17], [5, 3], 14, 2, 16),
    ([300, 260], [70, 9], 16, 2, 64),
    ([1300, 700], [600, 130], 8, 2, 16),
]


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("lens,news,H_q,H,page", SHAPES)
def test_attention(lens, news, H_q, H, page, q_dtype):
    pool = Pool4(lens, H, 128, page, seed=3)
    run_attn(pool, news, H_q, q_dtype, seed=4)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("H_q,H", [(8, 2), (33, 1), (40, 2)])
def test_attention_not_causal_and_many_heads(H_q, H, q_dtype):
    pool = Pool4([150, 40, 7], H, 128, 32, seed=6)
    run_attn(pool, [3, 2, 9], H_q, q_dtype, seed=7, causal=False)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("d", [16, 80, 256])
def test_attention_of_other_sizes(d, q_dtype):
    pool = Pool4([150, 40], 2, d, 32, seed=6)
    run_attn(pool, [3, 2], 6, q_dtype, seed=7)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
def test_long_context_is_split(q_dtype):
    pool = Pool4([20000, 3, 9000], 2, 128, 64, seed=8)
    run_attn(pool, [1, 1, 2], 16, q_dtype, seed=9)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales_of_the_logits(scale):
    pool = Pool4([700], 2, 128, 64, seed=8)
    run_attn(pool, [2], 8, BF16, seed=9, scale=scale)


@pytest.mark.parametrize("news", [[2, 1], [40, 3]])
def test_strided_rows(news):
    pool = Pool4([800, 90], 4, 128, 64, seed=8, pad=64)
    run_attn(pool, news, 32, BF16, seed=9, ld_pad=64)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("news", [[1, 1], [3, 2], [30, 50]])
def test_far_exponents(news, q_dtype):
    """Rows whose powers of two lie far from one, and far from one another: queries scaled so that logits stay in range."""
    pool = Pool4([260, 300], 2, 128, 32, seed=8, exps=(67, 187))
    pool_k = Pool4([260, 300], 2, 128, 32, seed=8, exps=(116, 124))
    # keys of ordinary size, values of exponents in +-60
    pool.Ke.copy_(pool_k.Ke)
    for s in range(2):
        pool.k[s], pool.v[s] = pool.values(s, np.arange(pool.lens[s]))
    run_attn(pool, news, 16, q_dtype, seed=9)


@pytest.mark.parametrize("news", [1, 3, 80])
def test_hidden_cells_do_not_enter(news):
    """NaN scales of V in cells that only later tokens see: tokens before them keep their results, those that see them
    are NaN; cells behind the sequence's end are NaN in every pool here."""
    lens = [200]
    pool = Pool4(lens, 1, 128, 32, seed=10)
    r = pool.np_rows(pool.table[0].cpu().numpy(), np.array([199]))[0]
    pool.Vs.view(torch.uint8)[r // 32, :, r % 32, 3] = 0x7f
    q = torch.randn(news, 8, 128, device=DEV).bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(news, 8, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(news, 1, news, 8, 1, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32([0, news]), pool.kv_len, q, out, 0.09, news, lse=lse, workspace=ws)
    o = out.double().cpu().numpy()
    assert np.isfinite(o[:-1]).all() and np.isfinite(lse.cpu().numpy()).all()
    assert np.isnan(o[-1, :, 48:64]).all()
    assert np.isfinite(o[-1, :, :48]).all() and np.isfinite(o[-1, :, 64:]).all()
    k, v = pool.k[0], pool.v[0].copy()
    v[199] = 0.0
    if news > 1:
        check_attention(o[:-1], lse.double().cpu().numpy()[:-1], q.double().cpu().numpy()[:-1], k[:199], v[:199], 200 - news, 0.09, True, BF16, E4M3, pool.units[0][:199])


@pytest.mark.parametrize("news", [1, 2, 60])
def test_nan_keys_are_their_rows_own(news):
    """A NaN scale of K makes the tokens that see the cell NaN, and no others."""
    pool = Pool4([150, 150], 2, 128, 16, seed=12)
    r = pool.np_rows(pool.table[1].cpu().numpy(), np.array([149]))[0]
    pool.Ks.view(torch.uint8)[r // 16, 1, r % 16, 0] = 0xff
    q = torch.randn(2 * news, 8, 128, device=DEV).bfloat16()
    out = torch.zeros_like(q)
    ws = torch.zeros(qsa.paged_attn_workspace_size(2 * news, 2, news, 8, 2, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, pool.table, i32([0, news, 2 * news]), pool.kv_len, q, out, 0.09, news, workspace=ws)
    o = out.float().cpu().numpy()
    assert np.isnan(o[-1, 4:]).all()
    assert np.isfinite(o[-1, :4]).all() and np.isfinite(o[:-1]).all()


@pytest.mark.parametrize("news", [1, 3, 90])
def test_bad_pages_and_lengths(news):
    """Sequences with a page outside the pool, and longer than the table: NaN; the others as ever."""
    lens = [160, 160, 160, 160]
    pool = Pool4(lens, 2, 128, 16, seed=13)
    t = pool.table.clone()
    t[1, 4], t[2, 2] = 100000, -1
    pool.table = t
    pool.kv_len = i32([160, 160, 160, 160 + 16 * 1000])
    n = 4 * news
    q = torch.randn(n, 8, 128, device=DEV).bfloat16()
    out, lse = torch.zeros_like(q), torch.zeros(n, 8, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, 4, news, 8, 2, 128), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(pool.cache, t, i32(starts([news] * 4)), pool.kv_len, q, out, 0.09, news, lse=lse, workspace=ws)
    o = out.double().cpu().numpy()
    assert np.isnan(o[news:]).all() and torch.isnan(lse[news:]).all()
    check_attention(o[:news], lse.double().cpu().numpy()[:news], q.double().cpu().numpy()[:news], pool.k[0], pool.v[0], 160 - news, 0.09, True, BF16, E4M3, pool.units[0])


@pytest.mark.parametrize("q_dtype,news", [(BF16, 1), (F32, 3), (BF16, 150)])
def test_captured_graph_follows_lengths(q_dtype, news):
    """One capture, replayed with other lengths, tables and queries in place; equal to eager calls, bit for bit."""
    pool = Pool4([5000, 2000], 2, 128, 64, seed=14)
    H_q, n = 16, 2 * news
    q = torch.randn(n, H_q, 128, device=DEV).to(q_dtype)
    out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device=DEV)
    cu = i32([0, news, n])
    ws = [torch.zeros(qsa.paged_attn_workspace_size(n, 2, news, H_q, 2, 128), dtype=torch.uint8, device=DEV) for _ in range(2)]

    def call(o, l, w):
        qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, q, o, 0.09, news, lse=l, workspace=w)

    call(out, lse, ws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, lse, ws[0])
    for lens in ([5000, 2000], [news, 1999], [257, 1024], [4097, max(1, news)]):
        pool.kv_len.copy_(i32(lens))
        q.normal_()
        want, wl = torch.zeros_like(out), torch.zeros_like(lse)
        call(want, wl, ws[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("news,max_q", [([40, 3], 1), ([40, 3], 8), ([1, 2], 500), ([200, 1], 3)])
def test_what_the_host_knows_of_lengths(news, max_q, q_dtype):
    """max_q chooses the kernel; the result is right where it is too small or too large."""
    run_attn(Pool4([300, 90], 2, 128, 32, seed=15), news, 16, q_dtype, seed=16, max_q=max_q)


@pytest.mark.parametrize("q_dtype", [BF16, F32])
@pytest.mark.parametrize("news", [1, 3, 60])
def test_queries_that_are_no_numbers(news, q_dtype):
    """A NaN or an infinity among a row's queries: that row is NaN, the others of its tile are as without it, and so is
    what is left of its head's other tokens."""
    pool = Pool4([150, 150], 2, 128, 16, seed=17)
    n = 2 * news
    q = torch.randn(n, 8, 128, device=DEV).to(q_dtype)
    out, clean = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, 2, news, 8, 2, 128), dtype=torch.uint8, device=DEV)
    cu = i32([0, news, n])
    qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, q, clean, 0.09, news, workspace=ws)
    bad = q.clone()
    bad[0, 1, 5], bad[n - 1, 6, 127], bad[n - 1, 0, 3] = float("nan"), float("inf"), float("-inf")
    qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, bad, out, 0.09, news, workspace=ws)
    odd = torch.zeros(n, 8, dtype=torch.bool, device=DEV)
    odd[0, 1] = odd[n - 1, 6] = odd[n - 1, 0] = True
    assert torch.isnan(out[odd]).all()
    assert torch.isfinite(out[~odd]).all()
    # (the power of two that scales a tile's queries goes by their largest finite magnitude, which may have changed: no
    # bits of the others do but what lies 2^-24 below, so the outputs differ by a rounding, one step of bf16, at most)
    torch.testing.assert_close(out[~odd].float(), clean[~odd].float(), rtol=2.0 ** -7, atol=2.0 ** -9)
