"""Prompts and chunks whose items are not cut between CTAs, up to the longest that are not."""
import math

import pytest
import torch

import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, E4M3, Pool, check_attention, i32, run_paged, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,H_q,H", [([2900], 8, 2), ([1500, 200, 1100], 8, 2), ([1050], 32, 4), ([1400], 4, 4)])
def test_prompts(lens, H_q, H):
    g = torch.Generator(device=DEV).manual_seed(sum(lens))
    cu = starts(lens)
    n = cu[-1]
    q, k, v = (torch.randn(n, h, 128, device=DEV, generator=g).to(BF16) for h in (H_q, H, H))
    out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device=DEV)
    ws = torch.full((qsa.prompt_attn_workspace_size(n, len(lens), H_q, H, 128),), 255, dtype=torch.uint8, device=DEV)
    scale = 1 / math.sqrt(128)
    qsa.prompt_attn(q, k, v, i32(cu), out, scale, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    o, l, qn, kn, vn = (x.double().cpu().numpy() for x in (out, lse, q, k, v))
    for a, b in zip(cu, cu[1:]):
        check_attention(o[a:b], l[a:b], qn[a:b], kn[a:b], vn[a:b], 0, scale, True, BF16, BF16)


@pytest.mark.parametrize("kv_dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,news", [([1900], [390]), ([1400, 300, 1500, 90], [100, 100, 37, 90])])
def test_chunks(lens, news, kv_dtype):
    run_paged(Pool(lens, 4, 128, 64, kv_dtype, seed=1), news, 32, BF16, seed=2)
