"""Many row tiles of a number of tokens that neither divides a tile of cells nor is a multiple of it (3, 5, 6, 7
heads per KV head), cut between CTAs: where a CTA's share begins is counted over all row tiles before it.
Compared in 64 bits at rows of every part; tolerances are those of test_gpu_dense.tolerance."""
import math

import numpy as np
import pytest
import torch

import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, E4M3, F32, Pool, check_attention, i32, run_paged, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H_q,H,causal", [([6000], 28, 4, True), ([9000], 6, 2, True), ([5000, 3, 700], 10, 2, True),
                                               ([3000, 1500], 12, 2, False)])
def test_long_prompts(lens, H_q, H, causal):
    g = torch.Generator(device=DEV).manual_seed(len(lens))
    cu = starts(lens)
    n, d = cu[-1], 128
    q, k, v = (torch.randn(n, h, d, device=DEV, generator=g).to(BF16) for h in (H_q, H, H))
    out, lse = torch.full_like(q, float("nan")), torch.full((n, H_q), float("nan"), device=DEV)
    ws = torch.full((qsa.prompt_attn_workspace_size(n, len(lens), H_q, H, d),), 255, dtype=torch.uint8, device=DEV)
    scale = 1 / math.sqrt(d)
    qsa.prompt_attn(q, k, v, i32(cu), out, scale, causal=causal, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()  # every row was written
    kn, vn = k.double().cpu().numpy(), v.double().cpu().numpy()
    for a, b in zip(cu, cu[1:]):
        # some rows of each row tile: every 17th token
        for i in np.arange(a, b, 17 if b - a < 2000 else 97):
            o, l, qn = (x[i:i + 1].double().cpu().numpy() for x in (out, lse, q))
            check_attention(o, l, qn, kn[a:b], vn[a:b], i - a, scale, causal, BF16, BF16)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,news,H_q,H", [([6000], [170], 6, 2), ([3000, 100, 2500], [90, 100, 61], 7, 1)])
def test_chunks(lens, news, H_q, H, kv_dtype):
    run_paged(Pool(lens, H, 128, 64, kv_dtype, seed=5), news, H_q, BF16, seed=6)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("H_q,H", [(10, 2), (3, 1)])
def test_fp32_queries(H_q, H, kv_dtype):
    """Row tiles of three and five tokens."""
    run_paged(Pool([1500, 40, 300], H, 128, 32, kv_dtype, seed=7), [200, 40, 111], H_q, F32, seed=8)
