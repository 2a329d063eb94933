"""Calls that run at the same time on streams of their own, with workspaces of their own, give the bits that
they give alone; so do two captured graphs replayed in turn and at once."""
import math

import pytest
import torch

import gather_qsa_pool_gb300 as qsa
from test_gpu_dense import BF16, DEV, E4M3, F32, Pool, i32, starts
from test_gpu_dense_few import widen

pytestmark = pytest.mark.gpu


def chunk(lens, news, H_q, kv_dtype, q_dtype, seed, width=0):
    pool = Pool(lens, 2, 128, 64, kv_dtype, seed=seed)
    if width:
        widen(pool, width)
    cu = i32(starts(news))
    n = sum(news)
    q = torch.randn(n, H_q, 128, device=DEV).to(q_dtype)
    out, lse = torch.zeros_like(q), torch.zeros(n, H_q, device=DEV)
    ws = torch.zeros(qsa.paged_attn_workspace_size(n, len(lens), max(news), H_q, 2, 128), dtype=torch.uint8, device=DEV)
    call = lambda: qsa.paged_attn(pool.cache, pool.table, cu, pool.kv_len, q, out, 1 / math.sqrt(128), max(news), lse=lse,
                                  workspace=ws)
    return call, (out, lse)


def prompt(lens, seed):
    n = sum(lens)
    q, k, v = (torch.randn(n, h, 128, device=DEV).to(BF16) for h in (8, 2, 2))
    out, lse = torch.zeros_like(q), torch.zeros(n, 8, device=DEV)
    ws = torch.zeros(qsa.prompt_attn_workspace_size(n, len(lens), 8, 2, 128), dtype=torch.uint8, device=DEV)
    cu = i32(starts(lens))
    return (lambda: qsa.prompt_attn(q, k, v, cu, out, 0.1, lse=lse, workspace=ws)), (out, lse)


def verify():
    p, d = (torch.softmax(3 * torch.randn(20, r, 40000, device=DEV), -1) for r in (4, 3))
    tokens = torch.randint(0, 40000, (20, 3), device=DEV).int()
    u = torch.rand(20, 4, device=DEV)
    out, acc = torch.zeros(20, 4, dtype=torch.int32, device=DEV), torch.zeros(20, dtype=torch.int32, device=DEV)
    return (lambda: qsa.draft_verify(p, d, tokens, u, out, acc)), (out, acc)


def calls():
    torch.manual_seed(3)
    return [
        chunk([5000, 900], [300, 200], 16, BF16, BF16, 1, 65536),   # 128 rows, cut and joined
        chunk([3000, 1200, 40], [4, 1, 3], 16, E4M3, BF16, 2, 16384),  # few rows
        chunk([1500, 300], [2, 1], 8, BF16, BF16, 3),               # short contexts
        chunk([2500, 70], [9, 3], 8, E4M3, F32, 4),                 # fp32 queries
        prompt([700, 1, 300], 5),
        verify(),
    ]


def bits(outs):
    return [o.clone().view(torch.uint8) for o in outs]


def test_on_streams_of_their_own():
    every = calls()
    want = []
    for call, outs in every:
        call()
        torch.cuda.synchronize()
        want.append(bits(outs))
    streams = [torch.cuda.Stream() for _ in every]
    for turn in range(5):
        for (call, outs), s in zip(every, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                for o in outs:
                    o.fill_(5)
                for _ in range(3):
                    call()
        torch.cuda.synchronize()
        for (_, outs), w in zip(every, want):
            assert all(torch.equal(a, b) for a, b in zip(bits(outs), w))


def test_graphs_in_turn_and_at_once():
    every = calls()[:5]
    want, graphs = [], []
    for call, outs in every:
        call()
        torch.cuda.synchronize()
        want.append(bits(outs))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for at_once in (False, True):
        for _, outs in every:
            for o in outs:
                o.fill_(5)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() if at_once else torch.cuda.current_stream() for _ in graphs]
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for (_, outs), w in zip(every, want):
            assert all(torch.equal(a, b) for a, b in zip(bits(outs), w))
