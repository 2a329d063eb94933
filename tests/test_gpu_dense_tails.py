"""e4m3 cells of small weight beside others of large weight: what a row's many small weights add must not be
cut off.  Every 32nd cell takes nearly all of the weight and has values of zero, so the output is what the
others add, 2^-20 and less of the largest weight each.

Tolerances, with A = sum_j softmax_j |v_j| and ds as in test_gpu_dense; a weight (times its cell's unit u_j)
is off by
  9 bits (bf16 queries, few rows, long contexts)   2^-9 of itself, or 3 * 2^-23 where the largest is >= 2^10
  fp16 (bf16 queries, short contexts)              2^-11 of itself, or 2^-25 where the largest is >= 2^13
  two fp16 terms (fp32 queries)                    2^-22 of itself, or 2^-25 where the largest is >= 2^13
so the output by A * (2 ds + (n + 64) * 2^-24 + rel) + small * max_j(softmax_j u_j) * sum_j |v_j| / u_j, with
small = 3 * 2^-33, 2^-38, 2^-38; and a bf16 output by half its step, 2^-8 |out|."""
import numpy as np
import pytest
import torch

import dense_reference as ref
import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, E4M3, F32, i32, small_weights

pytestmark = pytest.mark.gpu


def _check(n, width, q_dtype, rel, small, unit):
    """One sequence of n cells in a table of `width` cells, one KV head, four heads; unit: the exponent byte
    of the cells of small weight (the others have 127)."""
    page, d, G = 64, 128, 4
    rng = np.random.default_rng(n + unit)
    pages = -(-n // page)
    k, v = np.zeros((pages * page, 1, d), np.float32), np.zeros((pages * page, 1, d), np.float32)
    top = np.arange(0, n, 32)
    k[:n, 0, 1] = rng.random(n)          # logits that differ a little
    k[top, 0, 0] = 1.0
    v[:n, 0] = np.abs(16 * rng.standard_normal((n, d)))
    v[top] = 0.0
    K, V = torch.from_numpy(k).to(DEV).to(E4M3), torch.from_numpy(v).to(DEV).to(E4M3)
    Ke = torch.full((pages * page, 1), 127, dtype=torch.uint8, device=DEV)
    Ve = torch.full((pages * page, 1), unit, dtype=torch.uint8, device=DEV)
    Ve[torch.from_numpy(top).to(DEV)] = 127
    cache = qsa.PagedCache(K, V, page, K_exp=Ke, V_exp=Ve)
    table = torch.full((1, width // page), -1, dtype=torch.int32, device=DEV)
    table[0, :pages] = torch.randperm(pages, device=DEV).int()
    q = torch.zeros(1, G, d, device=DEV)
    q[0, :, 0] = torch.tensor([14.0, 15.5, 17.0, 18.1])   # 2^-20 .. 2^-26 of the largest weight
    q[0, :, 1] = 1.0
    q = q.to(q_dtype)
    out, lse = torch.zeros_like(q), torch.zeros(1, G, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(1, 1, 1, G, 1, d), dtype=torch.uint8, device=DEV)
    qsa.paged_attn(cache, table, i32([0, 1]), i32([n]), q, out, 1.0, 1, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    rows = table[0, :pages].cpu().numpy().astype(int)[np.arange(n) // page] * page + np.arange(n) % page
    kd, vd = K.float()[rows].double().cpu().numpy(), V.float()[rows].double().cpu().numpy()
    u = 2.0 ** (Ve[rows].cpu().numpy().astype(float) - 127)
    vd *= u[..., None]
    qd = q.double().cpu().numpy()
    want, wl = ref.attend(qd, kd, vd, n - 1, 1.0)
    A = ref.attend_weights_abs(qd, kd, vd, n - 1, 1.0)
    ds = (d + 16) * 2.0 ** -24 * np.abs(qd).sum(-1).max() * 2
    tol = A * (2 * ds + (n + 64) * 2.0 ** -24 + rel) + small * small_weights(qd, kd, vd, u, n - 1, 1.0, True)
    if q_dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    err = np.abs(out.double().cpu().numpy() - want)
    worst = (err / tol).max()
    assert worst <= 1, f"{worst:.3g} of the bound, {(err / np.abs(want)).max():.3g} of the output"
    assert (np.abs(lse.double().cpu().numpy() - wl) <= ds + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(wl)).all()


@pytest.mark.parametrize("unit", [127, 117])
@pytest.mark.parametrize("n", [300, 12000])
def test_few_rows_on_the_tensor_cores(n, unit):
    _check(n, 16384, BF16, 2.0 ** -9, 3 * 2.0 ** -33, unit)


@pytest.mark.parametrize("unit", [127, 117])
def test_short_contexts(unit):
    _check(2000, 2048, BF16, 2.0 ** -11, 2.0 ** -38, unit)


@pytest.mark.parametrize("unit", [127, 117])
@pytest.mark.parametrize("n", [300, 12000])
def test_fp32_queries(n, unit):
    _check(n, 16384, F32, 2.0 ** -22, 2.0 ** -38, unit)
