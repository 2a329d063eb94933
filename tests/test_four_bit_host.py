"""Host-only checks of the 4-bit cache, the append with rotation and the sparse attention over a paged cache: bad
arguments are refused before anything is launched, and the plain forms hold to known values.  No call here reaches
a kernel."""
import ctypes

import numpy as np
import pytest
import torch

import dense_reference as ref
import four_bit_reference as four
import gather_qsa_pool_gb300 as qsa
from gather_qsa_pool_gb300 import _binding as qb
from test_binding_devices import E4M3, every, i32, on

FAKE = 0x10000  # never dereferenced
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return qsa.load()


def struct(**kw):
    f = dict(K=FAKE, V=FAKE, K_exp=FAKE, V_exp=FAKE, dtype=3, H_kv=4, d=128, ld_k=512, ld_v=512, n_pages=10,
             page_size=64, K_scale=FAKE, V_scale=FAKE)
    f.update(kw)
    names = [n for n, _ in qb._PagedCacheStruct._fields_ + qb._PagedCacheScales._fields_]
    return qb._PagedCacheScales(*[f[n] for n in names])


def append_args(c):
    return dict(cache=ctypes.addressof(c), table=FAKE, ld_table=4, n_seq=2, cu=FAKE, kv_len=FAKE, q=FAKE, k=FAKE, v=FAKE,
                dt=1, n_tok=3, H_q=32, ld_q=4096, ld_k=512, ld_v=512, pos=None, rot=128, base=10000.0, q_out=FAKE,
                k_out=None, stream=None)


def sparse_args(c):
    return dict(cache=ctypes.addressof(c), table=FAKE, ld_table=4, n_seq=2, cu=FAKE, kv_len=FAKE, blocks=FAKE, counts=FAKE,
                k_blk=512, q=FAKE, dt=1, n_tok=3, ld_q=4096, H_q=32, scale=1.0, out=FAKE, lse=None, stream=None)


BAD = [(dict(K_exp=None), INVALID), (dict(V_exp=None), INVALID), (dict(K_scale=None), INVALID),
       (dict(V_scale=None), INVALID), (dict(K_scale=FAKE + 8), INVALID), (dict(V_scale=FAKE + 4), INVALID),
       (dict(d=120, ld_k=480, ld_v=480), INVALID), (dict(ld_k=496), INVALID), (dict(ld_k=520), INVALID),
       (dict(ld_v=513), INVALID), (dict(K=FAKE + 8), INVALID), (dict(d=272, ld_k=1088, ld_v=1088), UNSUPPORTED),
       (dict(page_size=4), INVALID), (dict(dtype=4), INVALID)]


@pytest.mark.parametrize("bad,want", BAD, ids=[",".join(b) for b, _ in BAD])
def test_every_call_refuses_a_bad_4_bit_cache(lib, bad, want):
    c = struct(**bad)
    r = ctypes.addressof(c)
    assert lib.qsa_paged_write(r, FAKE, 4, 2, FAKE, FAKE, FAKE, FAKE, 1, 3, 1088, 1088, None) == want
    assert lib.qsa_paged_read(r, FAKE, 4, 2, FAKE, None, None, FAKE, 2, 8, FAKE, FAKE, 1, None) == want
    assert lib.qsa_paged_attn(r, FAKE, 4, 2, FAKE, FAKE, FAKE, 1, 3, 2, 8704, 32, 1.0, 1, FAKE, None, FAKE, 1 << 40,
                              None) == want
    assert lib.qsa_paged_append(*append_args(c).values()) == want
    assert lib.qsa_paged_sparse_attn(*sparse_args(c).values()) == want


def test_append_refuses(lib):
    c = struct()
    base = append_args(c)

    def call(**kw):
        return lib.qsa_paged_append(*{**base, **kw}.values())

    for k in ("cache", "table", "cu", "kv_len", "k", "v", "q_out"):
        assert call(**{k: None}) == INVALID, k
    for k in ("q", "k", "v", "q_out", "k_out"):
        assert call(**{k: FAKE + 8}) == INVALID, k
    assert call(pos=FAKE + 2) == INVALID
    assert call(n_tok=-1) == INVALID and call(n_seq=0) == INVALID and call(ld_table=-1) == INVALID
    for dt in (-1, 2, 3):
        assert call(dt=dt) == INVALID
    for rot in (-16, 8, 72, 144):
        assert call(rot=rot) == INVALID
    for b in (0.5, 0.0, -1.0, float("nan"), float("inf")):
        assert call(base=b) == INVALID
    assert call(H_q=0) == INVALID and call(ld_q=4080) == INVALID and call(ld_q=4100) == INVALID
    assert call(ld_k=504) == INVALID and call(ld_v=516) == INVALID
    far = FAKE + (1 << 20)
    assert call(n_tok=2, q=far, q_out=far, ld_q=8192) == INVALID  # in place, but not packed
    assert call(n_tok=2, k=far, k_out=far, ld_k=1024) == INVALID
    assert call(H_q=1 << 18, ld_q=1 << 26) == UNSUPPORTED and call(n_seq=1 << 31) == UNSUPPORTED
    assert call(n_tok=0) == 0 and call(n_tok=0, q=None, q_out=None, H_q=0, ld_q=0) == 0


def test_sparse_refuses(lib):
    c = struct()
    base = sparse_args(c)

    def call(**kw):
        return lib.qsa_paged_sparse_attn(*{**base, **kw}.values())

    for k in ("cache", "table", "cu", "kv_len", "blocks", "counts", "q", "out"):
        assert call(**{k: None}) == INVALID, k
    assert call(blocks=FAKE + 2) == INVALID and call(counts=FAKE + 1) == INVALID and call(lse=FAKE + 2) == INVALID
    assert call(q=FAKE + 2) == INVALID and call(out=FAKE + 8) == INVALID and call(dt=2) == INVALID
    assert call(k_blk=-1) == INVALID and call(n_tok=-1) == INVALID and call(n_seq=0) == INVALID
    assert call(H_q=33) == INVALID and call(H_q=0) == INVALID and call(ld_q=4088) == INVALID
    assert call(k_blk=(1 << 28) + 1) == UNSUPPORTED and call(n_tok=1 << 27) == UNSUPPORTED
    assert call(n_tok=0) == 0


def test_python_refuses_wrong_4_bit_pools():
    R, H, B = 64, 2, 32
    good = dict(K=torch.zeros(R, H, B, dtype=torch.uint8), V=torch.zeros(R, H, B, dtype=torch.uint8),
                K_exp=torch.zeros(R, H, dtype=torch.uint8), V_exp=torch.zeros(R, H, dtype=torch.uint8),
                K_scale=torch.zeros(4, H, 16, 4).to(E4M3), V_scale=torch.zeros(4, H, 16, 4).to(E4M3))

    def make(**kw):
        t = {**good, **kw}
        return qsa.PagedCache(page_size=16, **{n: None if x is None else on(x) for n, x in t.items()})

    c = make()
    assert c.d == 64 and c._struct.ld_k == H * 64 and c._struct.dtype == 3
    for n in ("K_exp", "V_exp", "K_scale", "V_scale"):
        with pytest.raises(ValueError):
            make(**{n: None})
    with pytest.raises(ValueError):
        make(K_scale=torch.zeros(4, H, 16, 4, dtype=torch.uint8))
    with pytest.raises(ValueError):  # scales row by row: they lie head by head in a page
        make(K_scale=torch.zeros(4, 16, H, 4).to(E4M3))
    with pytest.raises(ValueError):  # 24 values a head
        make(K=good["K"][..., :12].contiguous(), V=good["V"][..., :12].contiguous())


@pytest.fixture
def cache(monkeypatch):
    pool = [on(torch.zeros(32, 2, 16)) for _ in range(2)]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return qsa.PagedCache(*pool, 8)


def test_append_on_another_device(cache):
    every(lambda **a: qsa.paged_append(cache, rope_base=10000.0, **a),
          dict(table=i32(2, 2), cu_q=i32(3), kv_len=i32(2), k=torch.zeros(3, 2, 16), v=torch.zeros(3, 2, 16),
               q=torch.zeros(3, 4, 16), q_out=torch.zeros(3, 4, 16), k_out=torch.zeros(3, 2, 16), pos=i32(3)))


def test_sparse_on_another_device(cache):
    every(lambda **a: qsa.paged_sparse_attn(cache, scale=1.0, **a),
          dict(table=i32(2, 2), cu_q=i32(3), kv_len=i32(2), blocks=i32(3, 4), counts=i32(3), q=torch.zeros(3, 4, 16),
               out=torch.zeros(3, 4, 16), lse=torch.zeros(3, 4)))


def test_python_refuses_wrong_tensors(cache):
    a = dict(table=on(i32(2, 2)), cu_q=on(i32(3)), kv_len=on(i32(2)))
    k, q = on(torch.zeros(3, 2, 16)), on(torch.zeros(3, 4, 16))

    def append(**kw):
        return qsa.paged_append(cache, **{**a, **dict(k=k, v=k, rope_base=10000.0), **kw})

    for bad in (dict(q=on(torch.zeros(2, 4, 16))), dict(q=on(torch.zeros(3, 4, 16).bfloat16())),
                dict(v=on(torch.zeros(2, 2, 16))), dict(q_out=q), dict(q=q, q_out=on(torch.zeros(3, 4, 15))),
                dict(q=on(torch.zeros(3, 8, 16)[:, :4])),               # not packed: there is nowhere to put it
                dict(k_out=on(torch.zeros(3, 4, 16))), dict(pos=on(torch.zeros(2, dtype=torch.int32)))):
        with pytest.raises(ValueError):
            append(**bad)

    def sparse(**kw):
        t = {**a, **dict(blocks=on(i32(3, 4)), counts=on(i32(3)), q=q, out=q, scale=1.0), **kw}
        return qsa.paged_sparse_attn(cache, **t)

    for bad in (dict(blocks=on(i32(2, 4))), dict(blocks=on(torch.zeros(3, 4))), dict(counts=on(i32(2))),
                dict(blocks=on(i32(4, 3)).t()), dict(out=on(torch.zeros(3, 4, 16).bfloat16())),
                dict(lse=on(torch.zeros(3, 3)))):
        with pytest.raises(ValueError):
            sparse(**bad)


def test_reference_rows():
    row = np.zeros(32)
    row[:4] = 2688.0, -224.0, 112.0, 0.0
    row[16:20] = 6.0, 3.5, -2.5, 0.25
    codes, scales, e = four.encode_row(row)
    assert e == 0 and scales[0] == 0x7e and ref.e4m3_values()[scales[1]] == 1.0
    assert list(codes[:4]) == [7, 9, 0, 0]          # 224 / 448 = 0.5; 112 / 448 = 0.25: a tie, to even
    assert list(codes[16:20]) == [7, 6, 12, 0]      # 3.5 -> 4, -2.5 -> -2, 0.25 -> 0: ties to even
    np.testing.assert_array_equal(four.values(codes, scales, e + 127)[16:20], [6.0, 4.0, -2.0, 0.0])
    assert four.encode_row(np.full(16, 2688.5))[2] == 1
    assert four.encode_row(np.full(16, np.nan))[1][0] == 0x7f
    assert four.encode_row(np.zeros(16))[2] == -100
    rng = np.random.default_rng(0)
    x = rng.standard_normal(128)
    c, s, e = four.encode_row(x)
    # a scale is off by at most 2^-4 of itself, a code by at most 1 (half a step) times it, or by what passes 6
    sv = np.repeat(ref.e4m3_values()[s], 16) * 2.0 ** e
    over = np.repeat(np.abs(x).reshape(-1, 16).max(-1), 16) - 6 * sv
    assert (np.abs(four.values(c, s, e + 127) - x) <= sv + np.maximum(over, 0)).all()


def test_reference_rotation():
    x = np.zeros((2, 1, 8))
    x[:, 0, 0] = x[:, 0, 6] = 1.0
    y = four.rotate(x, [0, 3], 4, 100.0)  # pairs (0, 2), (1, 3); value 6 stays
    np.testing.assert_allclose(y[0], x[0])
    np.testing.assert_allclose(y[1, 0], [np.cos(3), 0, np.sin(3), 0, 0, 0, 1, 0], atol=1e-15)


def test_reference_cells():
    assert list(four.listed_cells([0, 2, -1, 3], 4, 13)) == [0, 1, 2, 3, 8, 9, 10, 11, 12, 13]
    assert list(four.listed_cells([1, 1], 1, 7)) == [4, 5, 6, 7]
    assert list(four.listed_cells([0], 1, -1)) == []
