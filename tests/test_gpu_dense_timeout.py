"""Bounded waits of the tensor-core dense attention (qsa_set_wait_options): with the limit at 0 every
wait inside its pipeline gives up without looking; the kernel reports it, leaves NaN, returns its tensor
memory, and the next call is right again.  No wait is unbounded and nothing is made to fault."""
import numpy as np
import pytest
import torch

import gather_qsa_pool_gb300 as qsa

pytestmark = pytest.mark.gpu

TIMEOUT = 4  # QSA_ERR_TIMEOUT


@pytest.fixture
def status():
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    yield st
    qsa.set_wait_options(None, qsa.QSA_WAIT_DEFAULT_NS)  # later tests get the defaults


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _case(kind):
    """(run, out, lse): a call that takes the tensor-core kernel, its items whole, cut and joined."""
    g = torch.Generator(device="cuda").manual_seed(5)

    def rand(*s):
        return torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)

    H_q, H, d = 16, 2, 128
    if kind in ("short prompts", "prompts"):
        lens = [300, 1, 77] if kind == "short prompts" else [2500, 700]
        n = sum(lens)
        q, k, v = rand(n, H_q, d), rand(n, H, d), rand(n, H, d)
        cu = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
        ws = torch.zeros(qsa.prompt_attn_workspace_size(n, len(lens), H_q, H, d), dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device="cuda")
        return lambda: qsa.prompt_attn(q, k, v, cu, out, 0.1, lse=lse, workspace=ws), out, lse
    n, cells, page = 100, 5000, 64
    pages = -(-cells // page)
    K, V = rand(pages * page, H, d), rand(pages * page, H, d)
    e = None
    if kind == "e4m3 chunk":
        K, V = (16 * K.float()).to(torch.float8_e4m3fn), (16 * V.float()).to(torch.float8_e4m3fn)
        e = torch.full((pages * page, H), 123, dtype=torch.uint8, device="cuda")
    cache = qsa.PagedCache(K, V, page, K_exp=e, V_exp=e)
    table = torch.randperm(pages, device="cuda", generator=g).int()[None].contiguous()
    q = rand(n, H_q, d)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, 1, n, H_q, H, d), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device="cuda")
    cu, kv_len = _i32([0, n]), _i32([cells])
    return lambda: qsa.paged_attn(cache, table, cu, kv_len, q, out, 0.1, n, lse=lse, workspace=ws), out, lse


@pytest.mark.parametrize("kind", ["short prompts", "prompts", "chunk", "e4m3 chunk"])
def test_gives_up_and_recovers(kind, status):
    run, out, lse = _case(kind)
    run()
    torch.cuda.synchronize()
    want = out.clone(), lse.clone()
    assert torch.isfinite(out.float()).all()
    qsa.set_wait_options(status, 0)
    out.fill_(3.0)
    lse.fill_(3.0)
    run()
    torch.cuda.synchronize()
    assert int(status.item()) == TIMEOUT
    assert torch.isnan(out.float()).all() and torch.isnan(lse).all()
    qsa.set_wait_options(status, qsa.QSA_WAIT_DEFAULT_NS)
    status.zero_()
    for _ in range(2):
        run()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
    assert int(status.item()) == 0
