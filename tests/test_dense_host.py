"""Host-only checks of the paged cache, the dense attention and the draft verification: bad
arguments are refused before anything is launched, and the plain forms the GPU tests compare
with hold to known values.  No call here reaches a kernel."""
import ctypes

import numpy as np
import pytest

import dense_reference as ref
import gather_qsa_pool_gb300 as qsa
from gather_qsa_pool_gb300 import _binding as qb

P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return qsa.load()


def cache(**kw):
    f = dict(K=FAKE, V=FAKE, K_exp=None, V_exp=None, dtype=1, H_kv=4, d=128, ld_k=512, ld_v=512,
             n_pages=10, page_size=64)
    f.update(kw)
    c = qb._PagedCacheStruct(*[f[n] for n, _ in qb._PagedCacheStruct._fields_])
    return c


def write(lib, c, **kw):
    a = dict(table=FAKE, ld_table=4, n_seq=2, cu=FAKE, kv_len=FAKE, k=FAKE, v=FAKE, dt=1, n_tok=3,
             ld_k=512, ld_v=512)
    a.update(kw)
    return lib.qsa_paged_write(ctypes.addressof(c) if c else None, a["table"], a["ld_table"],
                               a["n_seq"], a["cu"], a["kv_len"], a["k"], a["v"], a["dt"],
                               a["n_tok"], a["ld_k"], a["ld_v"], None)


BAD_CACHES = [
    (dict(K=None), INVALID), (dict(V=FAKE + 8), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(H_kv=0), INVALID), (dict(d=0), INVALID),
    (dict(d=12, ld_k=48, ld_v=48), INVALID), (dict(ld_k=511), INVALID), (dict(ld_v=516), INVALID),
    (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID), (dict(page_size=4), INVALID),
    (dict(page_size=96), INVALID), (dict(page_size=8192), INVALID),
    (dict(dtype=2, ld_k=512, ld_v=512), INVALID),  # codes without exponents
    (dict(d=264, ld_k=1056, ld_v=1056), UNSUPPORTED), (dict(n_pages=1 << 25), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,want", BAD_CACHES, ids=[",".join(b) for b, _ in BAD_CACHES])
def test_every_call_refuses_a_bad_cache(lib, bad, want):
    c = cache(**bad)
    r = ctypes.addressof(c)
    assert write(lib, c) == want
    assert lib.qsa_paged_read(r, FAKE, 4, 2, FAKE, None, None, FAKE, 2, 8, FAKE, FAKE, 1, None) == want
    assert lib.qsa_paged_attn(r, FAKE, 4, 2, FAKE, FAKE, FAKE, 1, 3, 2, 4096, 32, 1.0, 1, FAKE,
                              None, FAKE, 1 << 40, None) == want


def test_write_refuses(lib):
    c = cache()
    assert write(lib, None) == INVALID
    for k in ("table", "cu", "kv_len", "k", "v"):
        assert write(lib, c, **{k: None}) == INVALID, k
    assert write(lib, c, n_tok=-1) == INVALID
    assert write(lib, c, n_seq=-1) == INVALID
    assert write(lib, c, n_seq=0) == INVALID            # tokens of no sequence
    assert write(lib, c, ld_table=-1) == INVALID
    assert write(lib, c, ld_k=508) == INVALID           # shorter than a row
    assert write(lib, c, ld_v=514) == INVALID           # rows not 16-byte multiples
    assert write(lib, c, k=FAKE + 2) == INVALID
    assert write(lib, c, dt=2) == INVALID               # rows are written from fp32 or bf16
    assert write(lib, c, cu=FAKE + 2) == INVALID
    assert write(lib, c, n_seq=1 << 31, n_tok=1) == UNSUPPORTED
    assert write(lib, c, n_tok=0) == 0                  # nothing to do


def test_read_refuses(lib):
    c = cache()
    r = ctypes.addressof(c)
    base = [r, FAKE, 4, 2, FAKE, None, None, FAKE, 2, 8, FAKE, FAKE, 1, None]

    def call(i, v):
        a = list(base)
        a[i] = v
        return lib.qsa_paged_read(*a)

    for i in (0, 1, 4, 7, 10, 11):
        assert call(i, None) == INVALID, i
    assert call(2, -1) == INVALID
    assert call(3, -1) == INVALID
    assert call(5, FAKE + 1) == INVALID
    assert call(6, FAKE + 2) == INVALID
    assert call(8, -1) == INVALID
    assert call(9, -1) == INVALID
    assert call(10, FAKE + 8) == INVALID
    assert call(12, 2) == INVALID
    assert call(9, 1 << 30) == UNSUPPORTED
    assert call(8, 0) == 0
    assert call(9, 0) == 0


def _attn_args(lib, r):
    need = lib.qsa_paged_attn_workspace_size(3, 2, 2, 32, 4, 128)
    return [r, FAKE, 4, 2, FAKE, FAKE, FAKE, 1, 3, 2, 4096, 32, 1.0, 1, FAKE, None, FAKE, need, None]


def test_paged_attn_refuses(lib):
    c = cache()
    base = _attn_args(lib, ctypes.addressof(c))

    def call(*changes):
        a = list(base)
        for i, v in changes:
            a[i] = v
        return lib.qsa_paged_attn(*a)

    for i in (0, 1, 4, 5, 6, 14):
        assert call((i, None)) == INVALID, i
    assert call((6, FAKE + 2)) == INVALID      # q misaligned
    assert call((7, 2)) == INVALID             # q is fp32 or bf16
    assert call((8, -1)) == INVALID
    assert call((9, -1)) == INVALID
    assert call((9, 0)) == INVALID             # tokens, but none in any sequence
    assert call((10, 4095)) == INVALID
    assert call((10, 4100)) == INVALID         # rows not 16-byte multiples
    assert call((11, 0)) == INVALID
    assert call((11, 33), (10, 33 * 128)) == INVALID
    assert call((14, FAKE + 8)) == INVALID
    assert call((15, FAKE + 2)) == INVALID
    assert call((3, 1 << 31)) == UNSUPPORTED
    assert call((8, 1 << 30)) == UNSUPPORTED   # 4 KV heads of as many tokens
    assert call((8, 0)) == 0


def test_prompt_attn_refuses(lib):
    need = lib.qsa_prompt_attn_workspace_size(100, 2, 32, 4, 128)
    base = [FAKE, FAKE, FAKE, 1, 100, 4096, 512, 512, FAKE, 2, 32, 4, 128, 1.0, 1, FAKE, None,
            FAKE, need, None]

    def call(*changes):
        a = list(base)
        for i, v in changes:
            a[i] = v
        return lib.qsa_prompt_attn(*a)

    for i in (0, 1, 2, 8, 15):
        assert call((i, None)) == INVALID, i
    assert call((3, 2)) == INVALID
    assert call((4, -1)) == INVALID
    assert call((5, 4088)) == INVALID
    assert call((6, 508)) == INVALID
    assert call((7, 516)) == INVALID
    assert call((9, -1)) == INVALID
    assert call((9, 0)) == INVALID
    assert call((10, 30)) == INVALID           # not a multiple of the KV heads
    assert call((11, 0)) == INVALID
    assert call((12, 124)) == INVALID
    assert call((1, FAKE + 4)) == INVALID
    assert call((16, FAKE + 1)) == INVALID
    assert call((12, 264), (5, 8448), (6, 1056), (7, 1056)) == UNSUPPORTED
    assert call((4, 1 << 31)) == UNSUPPORTED
    assert call((4, 0)) == 0


def test_draft_verify_refuses(lib):
    base = [FAKE, 100, FAKE, 100, FAKE, None, FAKE, 2, 3, 100, FAKE, FAKE, None]

    def call(*changes):
        a = list(base)
        for i, v in changes:
            a[i] = v
        return lib.qsa_draft_verify(*a)

    for i in (0, 4, 6, 10, 11):
        assert call((i, None)) == INVALID, i
    assert call((1, 99)) == INVALID
    assert call((3, 99)) == INVALID
    assert call((7, -1)) == INVALID
    assert call((8, -1)) == INVALID
    assert call((9, 0)) == INVALID
    assert call((5, FAKE + 2)) == INVALID
    assert call((0, FAKE + 2)) == INVALID
    assert call((9, (1 << 31) - 1), (1, 1 << 32), (3, 1 << 32)) == UNSUPPORTED
    assert call((8, 1 << 30), (7, 4)) == UNSUPPORTED
    assert call((7, 0)) == 0


def test_python_wrappers_refuse_wrong_tensors():
    import torch

    k = torch.zeros(64, 2, 16)
    with pytest.raises(ValueError):
        qsa.PagedCache(k, k[:, :1], 32)             # different shapes
    with pytest.raises(ValueError):
        qsa.PagedCache(k, k, 48)                    # not whole pages
    with pytest.raises(TypeError):
        qsa.PagedCache(k.half(), k.half(), 32)
    with pytest.raises(ValueError):                 # tensors of the host
        qsa.PagedCache(k, k, 32)
    c = torch.zeros(64, 2, 16, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        qsa.PagedCache(c, c, 32)
    q = torch.zeros(5, 4, 16)
    with pytest.raises(ValueError):
        qsa.prompt_attn(q, k[:5], k[:5], torch.zeros(2, dtype=torch.int32), q.clone(), 1.0)
    with pytest.raises(ValueError):
        qsa.draft_verify(torch.zeros(2, 3, 10), None, torch.zeros(2, 2, dtype=torch.int32),
                         torch.zeros(2, 3), torch.zeros(2, 3, dtype=torch.int32),
                         torch.zeros(2, dtype=torch.int32))


def test_reference_codes_match_the_format():
    v = ref.e4m3_values()
    assert v[0x7e] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7f])
    import torch

    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(np.isnan(t), np.isnan(v))
    np.testing.assert_array_equal(t[~np.isnan(v)], v[~np.isnan(v)])
    # exponents at the border of 448 and roundings to even
    assert ref.encode_row([448.0])[1] == 0 and ref.encode_row([448.5])[1] == 1
    assert ref.encode_row([0.0])[1] == -100
    codes, e = ref.encode_row([256.0, 17.0, 19.0, -1.0 / 1024])
    assert e == 0 and list(codes) == [256.0, 16.0, 20.0, -0.0]
    assert ref.encode_row([2.0 ** 120])[0][0] == 448.0


def test_reference_verification_keeps_the_targets_distribution():
    """Over many draws the first token's frequencies are the target's, whatever the draft is."""
    rng = np.random.default_rng(3)
    V, n = 5, 40000
    p, q = rng.dirichlet(np.ones(V), 2), rng.dirichlet(np.ones(V), 1)
    seen = np.zeros(V)
    for _ in range(n):
        t = rng.choice(V, p=q[0])
        out, a = ref.verify(p, q, [t], 1, rng.random(2))
        assert a == (out[1] >= 0)
        seen[out[0]] += 1
    # five standard deviations of a frequency
    assert np.all(np.abs(seen / n - p[0]) < 5 * np.sqrt(p[0] / n))
