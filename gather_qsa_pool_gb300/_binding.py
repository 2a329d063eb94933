"""ctypes binding of ``libqsa.so``: argument marshalling only.

Every function here has the name of the C entry point it calls (without the ``qsa_``
prefix), takes torch tensors that already live on the GPU, passes their data pointers,
sizes and the current CUDA stream, and raises :class:`QSAError` when the call returns a
non-OK status.  All computation happens in the library's CUDA kernels; there is no
fallback of any kind: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libqsa.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "qsa.h")

QSA_OK, QSA_ERR_INVALID_ARG, QSA_ERR_UNSUPPORTED, QSA_ERR_CUDA, QSA_ERR_TIMEOUT = range(5)
QSA_F32, QSA_BF16, QSA_E4M3 = 0, 1, 2
QSA_PREC_F32, QSA_PREC_BF16_TC = 0, 1
QSA_WAIT_DEFAULT_NS = 2_000_000_000

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f = ctypes.c_float
_d = ctypes.c_double
_sz = ctypes.c_size_t

_SIGNATURES = {
    "qsa_status_str": (ctypes.c_char_p, [_int]),
    "qsa_version": (_int, []),
    "qsa_set_wait_options": (None, [_p, ctypes.c_uint64]),
    "qsa_pool_update": (_int, [_p, _int, _i64, _int, _int, _p, _f, _d, _p, _int, _i64, _i64,
                               _p]),
    "qsa_index_score": (_int, [_p, _i64, _i64, _p, _p, _int, _i64, _int, _int, _f, _p, _i64,
                               _int, _p, _sz, _p]),
    "qsa_index_score_workspace_size": (_sz, [_i64, _i64, _int, _int, _int, _int]),
    "qsa_topk_blocks": (_int, [_p, _i64, _i64, _p, _i64, _i64, _p, _p, _p]),
    "qsa_topk_max_candidates": (_i64, []),
    "qsa_index_score_maxima": (_int, [_p, _i64, _i64, _p, _p, _int, _i64, _int, _int, _f, _p,
                                      _i64, _p, _i64, _p, _sz, _p]),
    "qsa_topk_blocks_maxima": (_int, [_p, _i64, _i64, _p, _i64, _i64, _p, _i64, _p, _p, _p,
                                      _sz, _p]),
    "qsa_topk_blocks_maxima_workspace_size": (_sz, [_i64]),
    "qsa_expand_block_scores": (_int, [_p, _i64, _i64, _i64, _p, _i64, _p]),
    "qsa_gather_kv": (_int, [_p, _p, _int, _i64, _int, _int, _int, _i64, _i64, _p, _p, _i64,
                             _i64, _p, _i64, _p, _p, _p, _p, _i64, _p]),
    "qsa_sparse_attn": (_int, [_p, _i64, _int, _int, _int, _int, _f, _p, _p, _int, _i64, _i64,
                               _i64, _p, _p, _i64, _p, _p, _p, _sz, _p]),
    "qsa_sparse_attn_workspace_size": (_sz, [_i64, _int, _int, _int, _i64]),
    "qsa_sparse_attn_union": (_int, [_p, _i64, _int, _int, _int, _f, _p, _p, _int, _i64, _i64,
                                     _i64, _p, _p, _i64, _p, _p, _p, _sz, _p]),
    "qsa_sparse_attn_union_workspace_size": (_sz, [_i64, _i64]),
    "qsa_decode_step": (_int, [_p, _int, _i64, _int, _int, _p, _f, _d, _p, _int, _i64, _i64,
                               _i64, _p, _f, _p, _i64, _p, _p, _p, _p, _int, _i64, _int, _int,
                               _i64, _p, _p, _i64, _p, _int, _f, _p, _p, _p, _sz, _p]),
    "qsa_decode_step_workspace_size": (_sz, [_i64, _int, _int, _int, _i64, _i64]),
    "qsa_decode_step_host": (_int, [_p, _p, _p, _p, _int, _i64, _int, _int, _p, _f, _d, _p, _int,
                                    _i64, _i64, _i64, _f, _p, _i64, _p, _p, _p, _p, _int, _i64,
                                    _int, _int, _i64, _p, _p, _i64, _int, _f, _p, _p, _p, _sz,
                                    _p]),
    "qsa_decode_step_host_layout": (_sz, [_i64, _int, _int, _int, _int, _int, _int, _int, _p]),
    "qsa_decode_step_host_workspace_size": (_sz, [_i64, _int, _int, _int, _i64, _i64, _int, _int,
                                                  _int, _int]),
    "qsa_decode_plan_create": (_int, [ctypes.POINTER(_p), _p, _int, _int, _int, _p, _f, _d, _p,
                                      _int, _i64, _i64, _f, _p, _i64, _p, _p, _p, _p, _int, _i64,
                                      _int, _int, _i64, _p, _p, _i64, _int, _f, _p, _p, _p, _sz]),
    "qsa_decode_plan_destroy": (None, [_p]),
    "qsa_decode_plan_step": (_int, [_p, _i64, _i64, _i64, _p, _p, _p]),
    "qsa_decode_plan_step_host": (_int, [_p, _i64, _i64, _i64, _p, _p, _p, _p]),
    "qsa_mask_to_list": (_int, [_p, _i64, _i64, _i64, _i64, _p, _p, _p, _p]),
    "qsa_mask_sparse_eligible": (_int, [_int, _f, _f, _i64, _i64]),
    "qsa_mask_sparse_attn": (_int, [_p, _i64, _int, _int, _int, _int, _f, _p, _int, _i64, _i64,
                                    _p, _i64, _i64, _p, _p, _p, _p]),
    "qsa_paged_write": (_int, [_p, _p, _i64, _i64, _p, _p, _p, _p, _int, _i64, _i64, _i64, _p]),
    "qsa_paged_read": (_int, [_p, _p, _i64, _i64, _p, _p, _p, _p, _i64, _i64, _p, _p, _int, _p]),
    "qsa_paged_attn": (_int, [_p, _p, _i64, _i64, _p, _p, _p, _int, _i64, _i64, _i64, _int, _f,
                              _int, _p, _p, _p, _sz, _p]),
    "qsa_paged_attn_workspace_size": (_sz, [_i64, _i64, _i64, _int, _int, _int]),
    "qsa_prompt_attn": (_int, [_p, _p, _p, _int, _i64, _i64, _i64, _i64, _p, _i64, _int, _int,
                               _int, _f, _int, _p, _p, _p, _sz, _p]),
    "qsa_prompt_attn_workspace_size": (_sz, [_i64, _i64, _int, _int, _int]),
    "qsa_draft_verify": (_int, [_p, _i64, _p, _i64, _p, _p, _p, _i64, _i64, _i64, _p, _p, _p]),
}

_lib = None


class QSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {status_str(status)}")


def header_functions() -> list[str]:
    """Names of every function that include/qsa.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(qsa_\w+)\s*\(", text, re.M)))


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the library (building it first when its sources are newer)."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        from . import build as _build

        path = _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"QSA CUDA library not found at {path}")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def set_wait_options(status=None, limit_ns=QSA_WAIT_DEFAULT_NS):
    """qsa_set_wait_options: for later launches from this thread, the int32 device tensor a
    kernel whose bounded wait gave up stores QSA_ERR_TIMEOUT into (or None), and the limit of
    the waits inside a kernel's pipeline (0: give up unless already complete)."""
    load().qsa_set_wait_options(_ptr(status), int(limit_ns))


def status_str(status: int) -> str:
    return load().qsa_status_str(status).decode()


def _check(fn: str, status: int):
    if status != QSA_OK:
        raise QSAError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ld(t) -> int:
    """Element stride between rows of a row-major tensor (a single-row tensor may carry an
    arbitrary stride on its size-1 leading dim: use its row length)."""
    if t.dim() < 2 or t.shape[0] <= 1:
        return t[0].numel() if t.dim() >= 2 else t.numel()
    return t.stride(0)


def _dtype(t) -> int:
    import torch

    if t.dtype == torch.float32:
        return QSA_F32
    if t.dtype == torch.bfloat16:
        return QSA_BF16
    raise TypeError(f"QSA tensors are float32 or bfloat16, got {t.dtype}")


# --------------------------------------------------------------------------- entry points

def pool_update(raw_k, n_ctx, H, d, norm_w, eps, rope_base, pooled, n_valid_full, stream=None):
    """qsa_pool_update: recompute pooled rows [n_valid_full, ceil(n_ctx/4)) of a float32 or
    bfloat16 cache."""
    _check("qsa_pool_update", load().qsa_pool_update(
        _ptr(raw_k), _dtype(raw_k), n_ctx, H, d, _ptr(norm_w), eps, rope_base, _ptr(pooled),
        _dtype(pooled), pooled.shape[0], n_valid_full, _stream(stream)))


def index_score_workspace_size(n_q, n_rows, H, d, precision=QSA_PREC_F32,
                               pooled_dtype=QSA_F32) -> int:
    return int(load().qsa_index_score_workspace_size(n_q, n_rows, H, d, pooled_dtype,
                                                     precision))


def index_score(q, pooled, n_rows, H, d, scale, scores, q_pos=None, precision=QSA_PREC_F32,
                workspace=None, stream=None):
    """qsa_index_score: scores[i][b] for b < n_rows (q: [n_q][>= H*d] fp32; pooled float32
    or bfloat16)."""
    n_q = q.shape[0] if q.dim() > 1 else 1
    ld_q = _ld(q) if q.dim() > 1 else H * d
    ld_s = _ld(scores) if scores.dim() > 1 else n_rows
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qsa_index_score", load().qsa_index_score(
        _ptr(q), n_q, ld_q, _ptr(q_pos), _ptr(pooled), _dtype(pooled), n_rows, H, d, scale,
        _ptr(scores), ld_s, precision, _ptr(workspace), ws_bytes, _stream(stream)))


def topk_max_candidates() -> int:
    return int(load().qsa_topk_max_candidates())


def topk_blocks(scores, n_full, k_blk, blocks_out, counts_out, q_pos=None, stream=None):
    """qsa_topk_blocks over the first n_full columns of each score row."""
    n_q = scores.shape[0] if scores.dim() > 1 else 1
    ld = _ld(scores)
    _check("qsa_topk_blocks", load().qsa_topk_blocks(
        _ptr(scores), n_q, ld, _ptr(q_pos), n_full, k_blk, _ptr(blocks_out), _ptr(counts_out),
        _stream(stream)))


def index_score_maxima(q, pooled, n_rows, H, d, scale, scores, maxima, q_pos=None,
                       workspace=None, stream=None):
    """qsa_index_score_maxima: the tensor-core scores plus maxima[i][g], the largest score of
    rows 32g .. 32g+31 of query i (maxima: [n_q][>= ceil(n_rows / 32)] fp32)."""
    n_q = q.shape[0] if q.dim() > 1 else 1
    ld_q = _ld(q) if q.dim() > 1 else H * d
    ld_s = _ld(scores) if scores.dim() > 1 else n_rows
    ld_m = _ld(maxima) if maxima.dim() > 1 else maxima.numel()
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qsa_index_score_maxima", load().qsa_index_score_maxima(
        _ptr(q), n_q, ld_q, _ptr(q_pos), _ptr(pooled), _dtype(pooled), n_rows, H, d, scale,
        _ptr(scores), ld_s, _ptr(maxima), ld_m, _ptr(workspace), ws_bytes, _stream(stream)))


def topk_blocks_maxima_workspace_size(n_q) -> int:
    return int(load().qsa_topk_blocks_maxima_workspace_size(n_q))


def topk_blocks_maxima(scores, maxima, n_full, k_blk, blocks_out, counts_out, workspace,
                       q_pos=None, stream=None):
    """qsa_topk_blocks_maxima: qsa_topk_blocks fed with the score kernel's group maxima
    (workspace: topk_blocks_maxima_workspace_size(n_q) bytes of device memory)."""
    n_q = scores.shape[0] if scores.dim() > 1 else 1
    ld = _ld(scores)
    ld_m = _ld(maxima) if maxima.dim() > 1 else maxima.numel()
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("qsa_topk_blocks_maxima", load().qsa_topk_blocks_maxima(
        _ptr(scores), n_q, ld, _ptr(q_pos), n_full, k_blk, _ptr(maxima), ld_m,
        _ptr(blocks_out), _ptr(counts_out), _ptr(workspace), ws_bytes, _stream(stream)))


def expand_block_scores(scores, n_full, cell_scores, stream=None):
    """qsa_expand_block_scores: cell_scores[i][c] = scores[i][c // 4] for c < 4*n_full."""
    n_q = scores.shape[0] if scores.dim() > 1 else 1
    ld_s = _ld(scores) if scores.dim() > 1 else scores.numel()
    ld_c = _ld(cell_scores) if cell_scores.dim() > 1 else cell_scores.numel()
    _check("qsa_expand_block_scores", load().qsa_expand_block_scores(
        _ptr(scores), n_q, ld_s, n_full, _ptr(cell_scores), ld_c, _stream(stream)))


def gather_kv(blocks, counts, k_blk, pos_out, n_cells_out, max_cells, n_ctx=-1, q_pos=None,
              K=None, V=None, K_out=None, V_out=None, H_kv=0, d_k=0, d_v=0, n_kv=None,
              stream=None):
    """qsa_gather_kv: cell positions (and compact K/V rows when K_out / V_out are given)."""
    n_q = counts.shape[0]
    dt = _dtype(K) if K is not None else QSA_BF16
    if n_kv is None:
        n_kv = K.shape[0] if K is not None else (1 << 62)
    ld_k = _ld(K) if K is not None else H_kv * d_k
    ld_v = _ld(V) if V is not None else H_kv * d_v
    _check("qsa_gather_kv", load().qsa_gather_kv(
        _ptr(K), _ptr(V), dt, n_kv, H_kv, d_k, d_v, ld_k, ld_v, _ptr(blocks), _ptr(counts), n_q,
        k_blk, _ptr(q_pos), n_ctx, _ptr(K_out), _ptr(V_out), _ptr(pos_out), _ptr(n_cells_out),
        max_cells, _stream(stream)))


def sparse_attn_workspace_size(n_q, H_q, H_kv, d_v, max_cells) -> int:
    return int(load().qsa_sparse_attn_workspace_size(n_q, H_q, H_kv, d_v, max_cells))


def sparse_attn(q, K, V, n_cells, max_cells, out, H_kv, d_k, d_v, scale, pos=None, lse=None,
                workspace=None, ld_k=None, ld_v=None, n_kv=None, stream=None):
    """qsa_sparse_attn: q [n_q][H_q][d_k] fp32 over listed cells of K/V."""
    n_q, H_q = q.shape[0], q.shape[1]
    ld_k = _ld(K) if ld_k is None else ld_k
    ld_v = _ld(V) if ld_v is None else ld_v
    n_kv = K.shape[0] if n_kv is None else n_kv
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qsa_sparse_attn", load().qsa_sparse_attn(
        _ptr(q), n_q, H_q, H_kv, d_k, d_v, scale, _ptr(K), _ptr(V), _dtype(K), n_kv, ld_k, ld_v,
        _ptr(pos), _ptr(n_cells), max_cells, _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
        _stream(stream)))


def sparse_attn_union(q, K, V, n_cells, max_cells, out, H_kv, d, scale, pos, lse=None,
                      workspace=None, ld_k=None, ld_v=None, n_kv=None, stream=None):
    """qsa_sparse_attn_union: q [n_q][H_q][d] fp32, groups of 16 consecutive queries over the
    union of their lists (bf16 K/V, d 128, 8 query heads per KV head)."""
    n_q, H_q = q.shape[0], q.shape[1]
    ld_k = _ld(K) if ld_k is None else ld_k
    ld_v = _ld(V) if ld_v is None else ld_v
    n_kv = K.shape[0] if n_kv is None else n_kv
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qsa_sparse_attn_union", load().qsa_sparse_attn_union(
        _ptr(q), n_q, H_q, H_kv, d, scale, _ptr(K), _ptr(V), _dtype(K), n_kv, ld_k, ld_v,
        _ptr(pos), _ptr(n_cells), max_cells, _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
        _stream(stream)))


def sparse_attn_union_workspace_size(n_q, max_cells) -> int:
    return int(load().qsa_sparse_attn_union_workspace_size(n_q, max_cells))


def decode_step(raw_k, n_ctx, H_idx, d_idx, norm_w, eps, rope_base, pooled, n_valid_full,
                q_idx, scale_idx, scores, k_blk, blocks, counts, K, V, H_kv, d, pos, n_cells,
                max_cells, q, H_q, scale, out, lse=None, workspace=None, n_q=1, stream=None):
    """qsa_decode_step: pool update, score, top-k, cell list and attention in one call, for
    the last n_q tokens of the context (packed per-query buffers)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("qsa_decode_step", load().qsa_decode_step(
        _ptr(raw_k), _dtype(raw_k), n_ctx, H_idx, d_idx, _ptr(norm_w), eps, rope_base,
        _ptr(pooled), _dtype(pooled), pooled.shape[0], n_valid_full, n_q, _ptr(q_idx), scale_idx,
        _ptr(scores), k_blk, _ptr(blocks), _ptr(counts), _ptr(K), _ptr(V), _dtype(K), K.shape[0],
        H_kv, d, _ld(K), _ptr(pos), _ptr(n_cells), max_cells, _ptr(q), H_q, scale, _ptr(out),
        _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream)))


def decode_step_workspace_size(H_q, H_kv, d, max_cells, cap_rows, n_q=1) -> int:
    return int(load().qsa_decode_step_workspace_size(n_q, H_q, H_kv, d, max_cells, cap_rows))


def decode_step_host_layout(n_q, raw_dtype, H_idx, d_idx, kv_dtype, H_kv, d, H_q):
    """(total bytes, [5] section offsets) of qsa_decode_step_host's packed input."""
    off = (ctypes.c_int64 * 5)()
    total = int(load().qsa_decode_step_host_layout(n_q, raw_dtype, H_idx, d_idx, kv_dtype, H_kv,
                                                   d, H_q, off))
    return total, list(off)


def decode_step_host_workspace_size(n_q, H_q, H_kv, d, max_cells, cap_rows, raw_dtype, H_idx,
                                    d_idx, kv_dtype) -> int:
    return int(load().qsa_decode_step_host_workspace_size(n_q, H_q, H_kv, d, max_cells, cap_rows,
                                                          raw_dtype, H_idx, d_idx, kv_dtype))


class DecodePlan:
    """A qsa_decode_plan: the fixed arguments of a sequence's decode steps bound once (the
    tensors are kept alive with the plan, which is destroyed with this object)."""

    def __init__(self, raw_k, norm_w, eps, rope_base, pooled, max_queries, scale_idx, scores,
                 k_blk, blocks, counts, K, V, H_idx, d_idx, H_kv, d, pos, n_cells, max_cells, H_q,
                 scale, out, lse, workspace):
        lib = load()
        handle = _p()
        ws_bytes = workspace.numel() * workspace.element_size()
        _check("qsa_decode_plan_create", lib.qsa_decode_plan_create(
            ctypes.byref(handle), _ptr(raw_k), _dtype(raw_k), H_idx, d_idx, _ptr(norm_w), eps,
            rope_base, _ptr(pooled), _dtype(pooled), pooled.shape[0], max_queries, scale_idx,
            _ptr(scores), k_blk, _ptr(blocks), _ptr(counts), _ptr(K), _ptr(V), _dtype(K),
            K.shape[0], H_kv, d, _ld(K), _ptr(pos), _ptr(n_cells), max_cells, H_q, scale,
            _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes))
        self._lib = lib
        self.handle = handle.value
        self._keep = (raw_k, norm_w, pooled, scores, blocks, counts, K, V, pos, n_cells, out, lse,
                      workspace)
        self.step = lib.qsa_decode_plan_step            # (handle, n_ctx, n_valid_full, n_q,
        self.step_host = lib.qsa_decode_plan_step_host  #  ...) -> status, see qsa.h

    def close(self):
        if self.handle:
            self._lib.qsa_decode_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown: the library may already be gone
            pass


def mask_to_list(mask, max_list, pos_out, counts_out, bits_out=None, n_kv=None, stream=None):
    """qsa_mask_to_list over every row of a uint8 mask [n_rows][ld]."""
    n_rows = mask.shape[0]
    n_kv = mask.shape[1] if n_kv is None else n_kv
    _check("qsa_mask_to_list", load().qsa_mask_to_list(
        _ptr(mask), n_rows, n_kv, _ld(mask), max_list, _ptr(pos_out), _ptr(counts_out),
        _ptr(bits_out), _stream(stream)))


def mask_sparse_attn(q, KV, mask, max_list, out, scale, counts_out=None, lse=None, n_kv=None,
                     d_k=576, d_v=512, stream=None):
    """qsa_mask_sparse_attn: q [n_q][16][576] fp32 over the set positions of each query's
    mask row (mask [n_q][ld] uint8), the latent KV rows [n_kv][ld] bf16."""
    n_q, H_q = q.shape[0], q.shape[1]
    n_kv = KV.shape[0] if n_kv is None else n_kv
    _check("qsa_mask_sparse_attn", load().qsa_mask_sparse_attn(
        _ptr(q), n_q, H_q, 1, d_k, d_v, scale, _ptr(KV), _dtype(KV), n_kv, _ld(KV), _ptr(mask),
        _ld(mask), max_list, _ptr(counts_out), _ptr(out), _ptr(lse), _stream(stream)))


def mask_sparse_eligible(has_mask, max_bias, softcap, n_kv, max_list) -> bool:
    st = load().qsa_mask_sparse_eligible(int(bool(has_mask)), max_bias, softcap, n_kv, max_list)
    if st not in (QSA_OK, QSA_ERR_UNSUPPORTED):
        raise QSAError("qsa_mask_sparse_eligible", st)
    return st == QSA_OK


# ------------------------------------------------- paged cache, dense attention, verification

class _PagedCacheStruct(ctypes.Structure):
    _fields_ = [("K", _p), ("V", _p), ("K_exp", _p), ("V_exp", _p), ("dtype", _int),
                ("H_kv", _int), ("d", _int), ("ld_k", _i64), ("ld_v", _i64), ("n_pages", _i64),
                ("page_size", _int)]


# The calls below are made once per layer and step, many of them on tensors that take the GPU a few
# microseconds: their checks are plain comparisons, and messages are made only when one fails.

_torch = None
_raw_stream_of = None


def _use_torch():
    """torch, imported on first use (this module itself loads without it)."""
    global _torch, _raw_stream_of
    import torch

    _torch = torch
    _raw_stream_of = torch._C._cuda_getCurrentRawStream
    return torch


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _dp(t):
    """Data pointer as an integer, or None."""
    return None if t is None else t.data_ptr()


def _gpu(name, t):
    """Index of the GPU that a call works on, by its first tensor; the others have to be there too, as the
    kernels get bare addresses."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor is wanted, got {tuple(t.shape)} on {t.device}")
    return dev


def _raw_stream(stream, dev):
    """The stream's handle: `stream`, or the current stream of the current device, on which the
    tensors must be."""
    here = _torch._C._cuda_getDevice()
    if dev != here:
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{here}")
    if stream is None:
        return _raw_stream_of(here)
    if stream.device_index != here:
        raise ValueError(f"tensors on cuda:{here}, but a stream of cuda:{stream.device_index}")
    return stream.cuda_stream


def _bad_i32(name, t, shape, dev):
    raise ValueError(f"{name}: a packed int32 tensor of shape {shape} or more on cuda:{dev} is wanted, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _i32_vector(name, t, n, dev):
    """int32, on the GPU, contiguous, n entries or more; its address."""
    if t.dtype is not _torch.int32 or t.get_device() != dev or t.dim() != 1 or t.shape[0] < n or \
            not t.is_contiguous():
        _bad_i32(name, t, (n,), dev)
    return t.data_ptr()


def _i32_table(t, n_seq, dev):
    if t.dtype is not _torch.int32 or t.get_device() != dev or t.dim() != 2 or t.shape[0] < n_seq or \
            not t.is_contiguous():
        _bad_i32("table", t, (n_seq, "pages"), dev)
    return t.data_ptr()


def _head_rows(name, t, H, d, dev):
    """[n][H][d] (or [n][H*d]) rows whose heads are contiguous; the stride between rows."""
    if t.get_device() == dev:
        shape, stride = t.shape, t.stride()
        if len(shape) == 3 and shape[1] == H and shape[2] == d:
            if shape[0] == 0:
                return H * d
            if (stride[2] == 1 or d == 1) and (stride[1] == d or H == 1):
                return stride[0] if shape[0] > 1 else H * d
        elif len(shape) == 2 and shape[1] == H * d:
            if shape[0] == 0:
                return H * d
            if stride[1] == 1:
                return stride[0] if shape[0] > 1 else H * d
    raise ValueError(f"{name}: a tensor of shape [n][{H}][{d}] with contiguous rows on cuda:{dev} is wanted, "
                     f"got {tuple(t.shape)} with strides {tuple(t.stride())} on {t.device}")


def _pool_rows(name, t):
    """[n_pages][page_size] rows as [n_pages * page_size] of the same memory: a copy would be a pool
    of its own, which the caller's program neither fills nor reads."""
    try:
        return t.view(t.shape[0] * t.shape[1], *t.shape[2:])
    except RuntimeError:
        raise ValueError(f"{name}: rows at one stride through all pages are wanted (other pools cannot be "
                         f"taken without a copy), got {tuple(t.shape)} with strides {tuple(t.stride())}") from None


class PagedCache:
    """A qsa_paged_cache: a pool of pages in K and V, [n_pages * page_size][H_kv][d] (or with a
    leading [n_pages][page_size] whose rows follow one another at one stride) of float32, bfloat16
    or float8_e4m3fn; the last with its exponent bytes K_exp, V_exp [n_pages * page_size][H_kv]
    uint8.  Holds the tensors, and never a copy of them."""

    def __init__(self, K, V, page_size, K_exp=None, V_exp=None):
        torch = _use_torch()
        if K.dim() == 4 and V.dim() == 4:
            K, V = _pool_rows("K", K), _pool_rows("V", V)
            if K_exp is not None and V_exp is not None:
                K_exp, V_exp = _pool_rows("K_exp", K_exp), _pool_rows("V_exp", V_exp)
        _need(K.dim() == 3 and K.shape == V.shape and K.dtype == V.dtype and K.device == V.device,
              "K and V: two tensors of one type and shape [rows][H_kv][d]")
        types = {torch.float32: QSA_F32, torch.bfloat16: QSA_BF16, torch.float8_e4m3fn: QSA_E4M3}
        if K.dtype not in types:
            raise TypeError(f"a paged cache is float32, bfloat16 or float8_e4m3fn, got {K.dtype}")
        rows, self.H_kv, self.d = K.shape
        _need(page_size > 0 and rows % page_size == 0, "K and V: a whole number of pages")
        dev = _gpu("K", K)
        ld_k = _head_rows("K", K, self.H_kv, self.d, dev)
        ld_v = _head_rows("V", V, self.H_kv, self.d, dev)
        if K.dtype == torch.float8_e4m3fn:
            for e in (K_exp, V_exp):
                _need(e is not None and e.dtype == torch.uint8 and e.is_contiguous()
                      and e.device == K.device and tuple(e.shape) == (rows, self.H_kv),
                      "K_exp and V_exp: contiguous uint8 [rows][H_kv] beside an 8-bit cache")
        self.K, self.V, self.K_exp, self.V_exp = K, V, K_exp, V_exp
        self._dev = dev
        self.page_size, self.n_pages = page_size, rows // page_size
        self._struct = _PagedCacheStruct(_dp(K), _dp(V), _dp(K_exp), _dp(V_exp), types[K.dtype],
                                         self.H_kv, self.d, ld_k, ld_v, self.n_pages, page_size)
        self._ref = ctypes.addressof(self._struct)


def paged_write(cache, table, cu_q, kv_len, k, v, stream=None):
    """qsa_paged_write: rows k, v [n_tok][H_kv][d] (float32 or bfloat16) of the new tokens into
    the pages of their sequences (table [n_seq][>= pages], cu_q [n_seq + 1], kv_len [n_seq])."""
    n_seq, n_tok, dev = kv_len.shape[0], k.shape[0], cache._dev
    tb, cu, kl = (_i32_table(table, n_seq, dev), _i32_vector("cu_q", cu_q, n_seq + 1, dev),
                  _i32_vector("kv_len", kv_len, 0, dev))
    ld_k = _head_rows("k", k, cache.H_kv, cache.d, dev)
    ld_v = _head_rows("v", v, cache.H_kv, cache.d, dev)
    if v.shape[0] != n_tok or v.dtype is not k.dtype:
        raise ValueError("k and v: one type and length")
    if n_tok == 0:
        return  # an empty tensor has no address
    st = load().qsa_paged_write(
        cache._ref, tb, table.shape[1], n_seq, cu, kl, k.data_ptr(), v.data_ptr(), _dtype(k), n_tok,
        ld_k, ld_v, _raw_stream(stream, dev))
    if st:
        raise QSAError("qsa_paged_write", st)


def paged_read(cache, table, kv_len, n_cells, max_cells, K_out, V_out, pos=None, seq=None,
               stream=None):
    """qsa_paged_read: the listed cells (pos [n_list][max_cells], or the first n_cells[i] of each
    sequence) as values, K_out / V_out [n_list][max_cells][H_kv][d] float32 or bfloat16."""
    n_seq, n_list, dev = kv_len.shape[0], n_cells.shape[0], cache._dev
    tb, kl, nc = (_i32_table(table, n_seq, dev), _i32_vector("kv_len", kv_len, 0, dev),
                  _i32_vector("n_cells", n_cells, 0, dev))
    if pos is not None and (pos.dtype is not _torch.int32 or pos.get_device() != dev or
                            tuple(pos.shape) != (n_list, max_cells) or not pos.is_contiguous()):
        _bad_i32("pos", pos, (n_list, max_cells), dev)
    if seq is not None:
        _i32_vector("seq", seq, n_list, dev)
    elif n_list > n_seq:
        raise ValueError("n_cells: one list per sequence unless seq is given")
    size = n_list * max_cells * cache.H_kv * cache.d
    for t in (K_out, V_out):
        if t.get_device() != dev or not t.is_contiguous() or t.numel() < size or t.dtype is not K_out.dtype:
            raise ValueError(f"K_out and V_out: packed [n_list][max_cells][H_kv][d] of one type on cuda:{dev}")
    if size == 0:
        return
    st = load().qsa_paged_read(
        cache._ref, tb, table.shape[1], n_seq, kl, _dp(seq), _dp(pos), nc, n_list, max_cells,
        K_out.data_ptr(), V_out.data_ptr(), _dtype(K_out), _raw_stream(stream, dev))
    if st:
        raise QSAError("qsa_paged_read", st)


def _attn_outputs(q, out, lse, workspace, n_tok, H_q, d, dev):
    """Checks what a call writes; the workspace's address and bytes."""
    if out.dtype is not q.dtype or out.get_device() != dev or not out.is_contiguous() or \
            out.numel() != n_tok * H_q * d:
        raise ValueError(f"out: packed, of q's type and shape, on cuda:{dev}")
    if lse is not None and (lse.dtype is not _torch.float32 or lse.get_device() != dev or
                            not lse.is_contiguous() or lse.numel() != n_tok * H_q):
        raise ValueError(f"lse: packed float32 [n_tok][H_q] on cuda:{dev}")
    if workspace is None:
        return None, 0
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: packed, on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def paged_attn_workspace_size(n_tok, n_seq, max_q, H_q, H_kv, d) -> int:
    return int(load().qsa_paged_attn_workspace_size(n_tok, n_seq, max_q, H_q, H_kv, d))


def paged_attn(cache, table, cu_q, kv_len, q, out, scale, max_q, causal=True, lse=None,
               workspace=None, stream=None):
    """qsa_paged_attn: q [n_tok][H_q][d] (float32 or bfloat16) of the new tokens over the cells
    of their sequences; out like q, lse [n_tok][H_q] float32.  workspace:
    paged_attn_workspace_size() bytes of device memory."""
    n_seq, n_tok, d, dev = kv_len.shape[0], q.shape[0], cache.d, cache._dev
    H_q = q.shape[1] if q.dim() == 3 else q.shape[-1] // d
    tb, cu, kl = (_i32_table(table, n_seq, dev), _i32_vector("cu_q", cu_q, n_seq + 1, dev),
                  _i32_vector("kv_len", kv_len, 0, dev))
    ld_q = _head_rows("q", q, H_q, d, dev)
    ws, ws_bytes = _attn_outputs(q, out, lse, workspace, n_tok, H_q, d, dev)
    if n_tok == 0:
        return
    st = load().qsa_paged_attn(
        cache._ref, tb, table.shape[1], n_seq, cu, kl, q.data_ptr(), _dtype(q), n_tok, max_q, ld_q,
        H_q, scale, 1 if causal else 0, out.data_ptr(), _dp(lse), ws, ws_bytes,
        _raw_stream(stream, dev))
    if st:
        raise QSAError("qsa_paged_attn", st)


def prompt_attn_workspace_size(n_tok, n_seq, H_q, H_kv, d) -> int:
    return int(load().qsa_prompt_attn_workspace_size(n_tok, n_seq, H_q, H_kv, d))


def prompt_attn(q, k, v, cu_seq, out, scale, causal=True, lse=None, workspace=None, stream=None):
    """qsa_prompt_attn: packed prompts q [n_tok][H_q][d], k, v [n_tok][H_kv][d] (float32 or
    bfloat16), sequence s at tokens cu_seq[s] .. cu_seq[s+1] - 1; out like q, lse [n_tok][H_q]
    float32.  workspace: prompt_attn_workspace_size() bytes of device memory."""
    if _torch is None:
        _use_torch()
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k, v: [n_tok][heads][d]")
    n_tok, H_q, d = q.shape
    H_kv = k.shape[1]
    dev = _gpu("q", q)
    cu = _i32_vector("cu_seq", cu_seq, 1, dev)
    ld_q, ld_k, ld_v = (_head_rows("q", q, H_q, d, dev), _head_rows("k", k, H_kv, d, dev),
                        _head_rows("v", v, H_kv, d, dev))
    if k.shape[0] != n_tok or v.shape[0] != n_tok or k.dtype is not q.dtype or v.dtype is not q.dtype:
        raise ValueError("q, k, v: one type and length")
    ws, ws_bytes = _attn_outputs(q, out, lse, workspace, n_tok, H_q, d, dev)
    if n_tok == 0:
        return
    st = load().qsa_prompt_attn(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype(q), n_tok, ld_q, ld_k, ld_v, cu,
        cu_seq.shape[0] - 1, H_q, H_kv, d, scale, 1 if causal else 0, out.data_ptr(), _dp(lse),
        ws, ws_bytes, _raw_stream(stream, dev))
    if st:
        raise QSAError("qsa_prompt_attn", st)


def _prob_rows(name, t, n_seq, n, vocab, dev):
    """float32 [n_seq][n][vocab] with every row at one stride from the one before; the stride."""
    if t.dtype is _torch.float32 and t.get_device() == dev and tuple(t.shape) == (n_seq, n, vocab):
        if n == 0 or n_seq == 0:
            return vocab
        s = t.stride()
        ld = s[1] if n > 1 else (s[0] if n_seq > 1 else vocab)
        if (s[2] == 1 or vocab == 1) and (n_seq == 1 or s[0] == n * ld):
            return ld
    raise ValueError(f"{name}: float32 [{n_seq}][{n}][{vocab}] on cuda:{dev} with contiguous rows at one stride "
                     f"is wanted, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _packed(name, t, dtype, shape, dev):
    if t.dtype is not dtype or t.get_device() != dev or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name}: packed {dtype} {shape} on cuda:{dev}")
    return t.data_ptr()


def draft_verify(target, draft, tokens, u, tokens_out, n_accepted, n_draft=None, stream=None):
    """qsa_draft_verify: target [n_seq][max_draft + 1][vocab] and draft [n_seq][max_draft][vocab]
    (or None) fp32 probabilities, tokens [n_seq][max_draft] and n_draft [n_seq] int32, u
    [n_seq][max_draft + 1] fp32; tokens_out [n_seq][max_draft + 1] and n_accepted [n_seq] int32."""
    if _torch is None:
        _use_torch()
    if target.dim() != 3 or target.shape[1] < 1:
        raise ValueError("target: [n_seq][max_draft + 1][vocab]")
    n_seq, n_rows, vocab = target.shape
    max_draft = n_rows - 1
    i32, f32 = _torch.int32, _torch.float32
    dev = _gpu("target", target)
    ld_t = _prob_rows("target", target, n_seq, n_rows, vocab, dev)
    ld_d = 0 if draft is None else _prob_rows("draft", draft, n_seq, max_draft, vocab, dev)
    tk, to, na, uu = (_packed("tokens", tokens, i32, (n_seq, max_draft), dev),
                      _packed("tokens_out", tokens_out, i32, (n_seq, n_rows), dev),
                      _packed("n_accepted", n_accepted, i32, (n_seq,), dev),
                      _packed("u", u, f32, (n_seq, n_rows), dev))
    nd = None if n_draft is None else _i32_vector("n_draft", n_draft, n_seq, dev)
    if n_seq == 0:
        return
    st = load().qsa_draft_verify(
        target.data_ptr(), ld_t, _dp(draft), ld_d, tk, nd, uu, n_seq, max_draft, vocab, to, na,
        _raw_stream(stream, dev))
    if st:
        raise QSAError("qsa_draft_verify", st)
