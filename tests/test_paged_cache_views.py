"""Pools given with a leading [n_pages][page_size]: a PagedCache works on the caller's memory, or refuses."""
import pytest
import torch

import gather_qsa_pool_gb300 as qsa

PAGES, PAGE, H, D = 6, 16, 2, 64
E4M3 = torch.float8_e4m3fn


def test_interleaved_pools_are_refused():
    """K and V of a page beside one another: the rows of two pages are not one stride apart."""
    kv = torch.zeros(PAGES, 2, PAGE, H, D)
    with pytest.raises(ValueError, match="without a copy"):
        qsa.PagedCache(kv[:, 0], kv[:, 1], PAGE)
    rows = torch.zeros(PAGES, PAGE, 2, H, D)
    with pytest.raises(ValueError, match="without a copy"):
        qsa.PagedCache(rows[:, :, 0], rows.transpose(0, 1)[:, :, 1], PAGE)


def test_interleaved_exponents_are_refused():
    c = torch.zeros(PAGES, PAGE, H, D, dtype=E4M3)
    e = torch.zeros(PAGES, 2, PAGE, H, dtype=torch.uint8)
    with pytest.raises(ValueError, match="without a copy"):
        qsa.PagedCache(c, c, PAGE, K_exp=e[:, 0], V_exp=e[:, 1])


def test_one_pool_with_pages_and_one_without_is_refused():
    k = torch.zeros(PAGES, PAGE, H, D)
    with pytest.raises(ValueError, match="one type and shape"):
        qsa.PagedCache(k, k.flatten(0, 1), PAGE)


def _write(K, V, Ke=None, Ve=None):
    """Three tokens at cells 14 .. 16 of a sequence of pages 4 and 1."""
    c = qsa.PagedCache(K, V, PAGE, K_exp=Ke, V_exp=Ve)
    assert c.K.data_ptr() == K.data_ptr() and c.V.data_ptr() == V.data_ptr()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    k = torch.arange(3 * H * D, device="cuda").view(3, H, D).bfloat16() + 1
    qsa.paged_write(c, i32([[4, 1]]), i32([0, 3]), i32([17]), k, -k)
    torch.cuda.synchronize()
    return k


@pytest.mark.gpu
@pytest.mark.parametrize("between", [0, 1])
def test_a_write_reaches_the_callers_pool(between):
    """Pages one behind another, and K and V rows in turn (a stride of two rows)."""
    pool = torch.zeros(PAGES, PAGE, 1 + between, H, D, dtype=torch.bfloat16, device="cuda")
    K = pool[:, :, 0]
    V = pool[:, :, 1] if between else torch.zeros_like(K)
    k = _write(K, V)
    for t, want in ((K, k), (V, -k)):
        assert torch.equal(t[4, 14], want[0]) and torch.equal(t[4, 15], want[1]) and torch.equal(t[1, 0], want[2])
        assert int((t != 0).any(-1).any(-1).sum()) == 3


@pytest.mark.gpu
def test_a_write_reaches_the_callers_exponents():
    K = torch.zeros(PAGES, PAGE, H, D, dtype=E4M3, device="cuda")
    V = torch.zeros_like(K)
    Ke = torch.zeros(PAGES, PAGE, H, dtype=torch.uint8, device="cuda")
    Ve = torch.zeros_like(Ke)
    k = _write(K, V, Ke, Ve)
    for t, e in ((K, Ke), (V, Ve)):
        assert int((e != 0).all(-1).sum()) == 3 and (e[4, 14:] != 0).all() and (e[1, 0] != 0).all()
    got = K[1, 0].float() * torch.exp2(Ke[1, 0].float() - 127)[:, None]
    # half a step of four significant bits
    assert ((got - k[2].float()).abs() <= 2.0 ** -4 * k[2].float()).all()
