"""Appends with the position rotation on the way, against the 64-bit forms.

Bound of a rotated value a cos t - b sin t: the cosine and sine are off by 2^-23 (2^-25 as one fp32 number, p * 2^-51 from
the angle: counted apart), the two products and their sum by 2^-23 of |a| + |b|; then the output's own rounding, half a
step.  Keys are held to 2^-27 of |a| + |b| (cosine and sine to 2^-29, what the sums of two fp32 numbers lose to less than
2^-29 each) before they are encoded: a stored value is the encoding of the exact one, or of one that far above or
below it.  A group's scale and a row's exponent go by its largest value, so they may differ with that one: an element is
one of what the row's encodings make of it with all its values moved up, not at all, or down.  The angle itself is off by
p * 2^-51 (frequencies to 2^-52 and their rounding), which counts against |a| + |b| too."""
import numpy as np
import pytest
import torch

import dense_reference as ref
import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from four_bit_pool import E2M1, any_pool
from test_gpu_dense import BF16, DEV, E4M3, F32, i32, starts

pytestmark = pytest.mark.gpu


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check_rotated(got, x, pos, rot, base, dtype):
    want = four.rotate(x, pos, rot, base)
    mag = np.abs(x).copy()
    if rot:
        both = np.abs(x[..., :rot // 2]) + np.abs(x[..., rot // 2:rot])
        mag[..., :rot // 2] = mag[..., rot // 2:rot] = both
    over = np.maximum(np.abs(np.asarray(pos, float)) * 2.0 ** -51, 0)[:, None, None]
    tol = np.abs(want) * half_step(dtype)
    tol[..., :rot] += mag[..., :rot] * (2.0 ** -22 + 2.0 ** -23 + over)
    return_ = want, mag[..., :rot] * (2.0 ** -27 + over)
    assert (np.abs(got - want) <= tol * (1 + 1e-6)).all(), (np.abs(got - want) / np.maximum(tol, 1e-300)).max()
    return return_


def encodings(t, row, off):
    """What a row of codes may hold, and its exponent bytes: (values, byte) of the exact row with its values moved up,
    not at all, and down by off."""
    out = []
    for s in (-1, 0, 1):
        x = row.copy()
        x[:len(off)] += s * off * np.where(x[:len(off)] < 0, -1.0, 1.0)
        if t == E4M3:
            w, e = ref.encode_row(x)
            out.append((w * 2.0 ** e, e + 127))
        else:
            c, sc, e = four.encode_row(x)
            out.append((four.values(c, sc, e + 127), e + 127))
    return out


def append(pool, news, H_q, src, seed, rot=None, base=10000.0, pos=None, with_q=True, with_k=True, pad=2, ld_pad=0, in_place=False):
    """The call and all its checks; returns q_out, k_out."""
    H, d, page = pool.H, pool.d, pool.page
    rot = d if rot is None else rot
    rng = np.random.default_rng(seed)
    cu = starts(news)
    n = cu[-1] + pad
    wide = torch.from_numpy(rng.standard_normal((n, (H_q + 2 * H) * d + ld_pad)).astype(np.float32)).to(DEV).to(src)
    q, k, v = wide[:, :(H_q + 2 * H) * d].split([H_q * d, H * d, H * d], 1)
    q, k, v = q.unflatten(1, (H_q, d)), k.unflatten(1, (H, d)), v.unflatten(1, (H, d))
    if in_place:
        q, k = q.contiguous(), k.contiguous()
    qn, kn, vn = (t.double().cpu().numpy() for t in (q, k, v))
    q_out = q if in_place else torch.full((n, H_q, d), -7.0, dtype=src, device=DEV)
    k_out = k if in_place else torch.full((n, H, d), -7.0, dtype=src, device=DEV)
    places = np.concatenate([np.arange(m - x, m) for x, m in zip(news, pool.lens)] + [np.zeros(0, int)])
    turned = places if pos is None else np.asarray(pos)[:len(places)]
    got = qsa.paged_append(pool.cache, pool.table, i32(cu), pool.kv_len, k, v, base, rot, q=q if with_q else None,
                           q_out=q_out if with_q and not in_place else None, k_out=k_out if with_k else None,
                           pos=None if pos is None else i32(pos))
    torch.cuda.synchronize()
    assert got is (q_out if with_q else None)
    at = cu[-1]
    if with_q:
        check_rotated(q_out.double().cpu().numpy()[:at], qn[:at], turned, rot, base, src)
        assert (q_out[at:] == (q[at:] if in_place else -7)).all()
    ko = k_out.double().cpu().numpy()
    exact, off = four.rotate(kn[:at], turned, rot, base), np.zeros((at, H, rot))
    if with_k:
        exact, off = check_rotated(ko[:at], kn[:at], turned, rot, base, src)
    for s, m in enumerate(news):
        if m == 0:
            continue
        cells = np.arange(pool.lens[s] - m, pool.lens[s])
        kc, vc = pool.values(s, cells)
        a, b = cu[s], cu[s + 1]
        r = pool.rows(pool.table[s].cpu().numpy(), cells).cpu().numpy()
        for is_v, (have, x) in enumerate(((kc, exact[a:b]), (vc, vn[a:b]))):
            t = pool.K.dtype
            if t in (E4M3, E2M1):
                exps = (pool.Ve if is_v else pool.Ke).cpu().numpy()[r]
                for i in range(m):
                    for h in range(H):
                        may = encodings(t, x[i, h], np.zeros(0) if is_v else off[a + i, h])
                        assert exps[i, h] in [e for _, e in may]
                        assert np.logical_or.reduce([(have[i, h] == w) | (np.isnan(have[i, h]) & np.isnan(w)) for w, _ in may]).all()
            elif is_v:
                np.testing.assert_array_equal(have, torch.from_numpy(x).to(t).double().numpy())
            else:
                check_rotated(have, kn[a:b], turned[a:b], rot, base, t)
    return q_out, k_out


@pytest.mark.parametrize("src", [BF16, F32])
@pytest.mark.parametrize("dtype", [E2M1, E4M3, BF16, F32])
@pytest.mark.parametrize("H,H_q,d,page,rot", [(4, 32, 128, 64, None), (1, 3, 16, 8, 16), (3, 6, 80, 16, 32), (2, 2, 256, 128, 256),
                                              (4, 4, 64, 32, 48), (5, 35, 128, 16, 64)])
def test_append(src, dtype, H, H_q, d, page, rot):
    pool = any_pool([1, 37, 0, 300, page, 5], H, d, page, dtype, seed=5)
    append(pool, [1, 5, 0, 120, 1, 0], H_q, src, seed=6, rot=rot)


@pytest.mark.parametrize("dtype", [E2M1, E4M3, BF16])
@pytest.mark.parametrize("n_seq,new", [(1, 1), (70, 1), (40, 3), (1, 2500)])
def test_numbers_of_tokens(dtype, n_seq, new):
    """From one token, whose heads go to a warp each, to whole tokens a warp."""
    pool = any_pool([new + (17 * i) % 50 for i in range(n_seq)], 2, 64, 16, dtype, seed=7)
    append(pool, [new] * n_seq, 8, F32, seed=8)


@pytest.mark.parametrize("dtype", [E2M1, BF16])
def test_without_queries_and_without_rotation(dtype):
    pool = any_pool([50, 9], 2, 128, 16, dtype, seed=7)
    append(pool, [7, 9], 8, F32, seed=8, with_q=False)
    append(pool, [7, 9], 8, F32, seed=9, rot=0)
    append(pool, [7, 9], 8, F32, seed=9, rot=0, with_k=False)


@pytest.mark.parametrize("src", [BF16, F32])
def test_strided_and_in_place(src):
    pool = any_pool([50, 9], 2, 128, 16, BF16, seed=7)
    append(pool, [7, 9], 8, src, seed=8, ld_pad=64)
    append(pool, [7, 9], 8, src, seed=8, in_place=True)


def test_positions_of_their_own():
    """Far positions, and negative ones; base 1 (every pair turns alike) and a large base."""
    pool = any_pool([50, 9], 2, 128, 16, F32, seed=7)
    rng = np.random.default_rng(1)
    pos = rng.integers(-2 ** 20, 2 ** 20, 18)
    pos[:6] = 0, 1, 255181, 2 ** 30, -2 ** 30, 2 ** 31 - 1
    for base in (1.0, 10000.0, 5e6):
        append(pool, [7, 9], 8, F32, seed=8, pos=pos, base=base)


def test_tokens_without_a_cell_are_skipped():
    """More new tokens than cells, and a page outside the pool: nothing is written outside the sequence's cells, and
    the queries and keys are rotated all the same."""
    pool = any_pool([3, 40], 2, 128, 16, F32, seed=7)
    t = pool.table.clone()
    t[1, 2] = 1 << 20
    before = pool.K.clone(), pool.V.clone()
    k = torch.randn(13, 2, 128, device=DEV)
    q = torch.randn(13, 4, 128, device=DEV)
    k_out, q_out = torch.zeros_like(k), torch.zeros_like(q)
    qsa.paged_append(pool.cache, t, i32([0, 5, 13]), pool.kv_len, k, k, 10000.0, q=q, q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    pos = np.concatenate([np.arange(-2, 3), np.arange(32, 40)])
    check_rotated(k_out.double().cpu().numpy(), k.double().cpu().numpy(), pos, 128, 10000.0, F32)
    check_rotated(q_out.double().cpu().numpy(), q.double().cpu().numpy(), pos, 128, 10000.0, F32)
    mine = pool.rows(t[0].cpu().numpy(), np.arange(3))
    assert torch.equal(pool.V[mine], k[2:5])
    rest = np.setdiff1d(np.arange(pool.K.shape[0]), mine.cpu().numpy())
    for now, was in zip((pool.K, pool.V), before):  # bits: rows that belong to no cell are NaN
        assert torch.equal(now[rest].view(torch.int32), was[rest].view(torch.int32))


@pytest.mark.parametrize("dtype", [E2M1, E4M3])
def test_values_that_are_no_numbers(dtype):
    """An infinity in a pair makes both NaN or infinite as the rotation does; rows of codes hold NaN there (4 bits: in
    the 16 values around)."""
    pool = any_pool([4], 1, 128, 16, dtype, seed=7)
    k = torch.randn(4, 1, 128, device=DEV)
    k[1, 0, 5], k[2, 0, 70] = float("inf"), float("nan")
    qsa.paged_append(pool.cache, pool.table, i32([0, 4]), pool.kv_len, k, k, 10000.0)
    torch.cuda.synchronize()
    got, v = pool.values(0, np.arange(4))
    span = (lambda i: slice(i // 16 * 16, i // 16 * 16 + 16)) if dtype == E2M1 else (lambda i: slice(i, i + 1))
    for row, i in ((1, 5), (1, 69), (2, 6), (2, 70)):
        assert np.isnan(got[row, 0, span(i)]).all()
    bad = np.isnan(got).sum()
    assert bad == (4 * 16 if dtype == E2M1 else 4) and np.isnan(v).sum() == (2 * 16 if dtype == E2M1 else 2)


@pytest.mark.parametrize("dtype", [E2M1, BF16])
def test_captured_graph(dtype):
    """A capture follows lengths that change in place: the cells and positions are the new ones."""
    pool = any_pool([200, 200], 2, 128, 16, dtype, seed=7)
    k, v, q = (torch.randn(2, h, 128, device=DEV) for h in (2, 2, 8))
    q_out = torch.zeros_like(q)
    cu, state = i32([0, 1, 2]), [t for t in (pool.K, pool.V, pool.Ke, pool.Ve) if t is not None]

    def call():
        qsa.paged_append(pool.cache, pool.table, cu, pool.kv_len, k, v, 10000.0, q=q, q_out=q_out)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([1, 200], [17, 90]):
        pool.kv_len.copy_(i32(lens))
        for t in (k, v, q):
            t.normal_()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone().view(torch.uint8) for t in state], q_out.clone()
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(got[0], state)) and torch.equal(got[1], q_out)
        check_rotated(q_out.double().cpu().numpy(), q.double().cpu().numpy(), [n - 1 for n in lens], 128, 10000.0, F32)
