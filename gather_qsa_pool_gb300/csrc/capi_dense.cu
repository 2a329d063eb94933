// capi_dense.cu -- the extern "C" entry points of the paged cache, the dense attention and the
// draft verification: argument validation on the host, then one launcher call per operation.
#include <algorithm>
#include <cmath>

#include "dense.cuh"
#include "draft_verify.cuh"
#include "paged.cuh"

using namespace qsa;

namespace {

constexpr int64_t kMaxInt = 0x7fffffffLL;

inline qsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool float_type(qsa_dtype d) { return d == QSA_F32 || d == QSA_BF16; }
// Bytes of `n` values (of QSA_E2M1 an even number).
inline int64_t bytes_of(qsa_dtype d, int64_t n) { return d == QSA_E2M1 ? n / 2 : n * (d == QSA_F32 ? 4 : (d == QSA_BF16 ? 2 : 1)); }

inline int log2_of(int v)
{
    int n = 0;
    while ((1 << n) < v) ++n;
    return n;
}

// Rows of `width` values at a stride of ld, read and written eight values at a time.
inline bool rows_ok(const void *p, int64_t ld, int64_t width, qsa_dtype dt)
{
    return p && aligned(p, 16) && ld >= width && ld % 2 == 0 && bytes_of(dt, ld) % (dt == QSA_E4M3 || dt == QSA_E2M1 ? 8 : 16) == 0;
}

qsa_status check_cache(const qsa_paged_cache *c)
{
    if (!c) return QSA_ERR_INVALID_ARG;
    const bool codes = c->dtype == QSA_E4M3 || c->dtype == QSA_E2M1;
    if (!float_type(c->dtype) && !codes) return QSA_ERR_INVALID_ARG;
    if (c->H_kv < 1 || c->d < 8 || c->d % 8 || c->n_pages < 0 || c->page_size < 8 ||
        c->page_size > 4096 || (c->page_size & (c->page_size - 1)))
        return QSA_ERR_INVALID_ARG;
    const int64_t width = (int64_t)c->H_kv * c->d;
    if (!rows_ok(c->K, c->ld_k, width, c->dtype) || !rows_ok(c->V, c->ld_v, width, c->dtype))
        return QSA_ERR_INVALID_ARG;
    if (codes && (!c->K_exp || !c->V_exp)) return QSA_ERR_INVALID_ARG;
    if (c->dtype == QSA_E2M1 && (c->d % 16 || !c->K_scale || !c->V_scale || !aligned(c->K_scale, 16) ||
                                 !aligned(c->V_scale, 16)))
        return QSA_ERR_INVALID_ARG;
    if (c->d > 256 || width > (1 << 24) || c->n_pages > kMaxInt / c->page_size)
        return QSA_ERR_UNSUPPORTED;
    return QSA_OK;
}

KvView view_of(const qsa_paged_cache *c, const int32_t *table, int64_t ld_table)
{
    KvView v;
    v.K = c->K;
    v.V = c->V;
    v.K_exp = c->K_exp;
    v.V_exp = c->V_exp;
    v.K_scale = c->dtype == QSA_E2M1 ? c->K_scale : nullptr;
    v.V_scale = c->dtype == QSA_E2M1 ? c->V_scale : nullptr;
    v.ld_k = c->ld_k;
    v.ld_v = c->ld_v;
    v.table = table;
    v.ld_table = ld_table;
    v.n_pages = (int32_t)c->n_pages;
    v.page_shift = log2_of(c->page_size);
    v.H_kv = c->H_kv;
    return v;
}

qsa_status check_seqs(const int32_t *table, int64_t ld_table, int64_t n_seq, const int32_t *kv_len,
                      int64_t n_tok)
{
    if (!table || !kv_len || ld_table < 0 || n_seq < 0 || n_tok < 0 || (n_seq < 1 && n_tok > 0) ||
        !aligned(table, 4) || !aligned(kv_len, 4))
        return QSA_ERR_INVALID_ARG;
    if (n_seq >= kMaxInt || n_tok > kMaxInt) return QSA_ERR_UNSUPPORTED;
    return QSA_OK;
}

qsa_status run_attn(const DenseArgs &a, int64_t max_q, void *workspace, size_t workspace_bytes,
                    cudaStream_t st)
{
    const int64_t items = (a.sv.n_tok + a.sv.n_seq) * (int64_t)a.kv.H_kv;
    if (items > kMaxInt || (int64_t)a.H_q * a.d > (1 << 24)) return QSA_ERR_UNSUPPORTED;
    if (dense_few_ok(a, max_q)) {
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < dense_few_workspace())
            return QSA_ERR_INVALID_ARG;
        return launch_dense_few(a, max_q, workspace, st);
    }
    if (few_four_ok(a, max_q)) {
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < few_four_workspace())
            return QSA_ERR_INVALID_ARG;
        return from_cuda(launch_few_four(a, max_q, workspace, st));
    }
    if (dense_decode_ok(a, max_q)) {
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < dense_decode_workspace())
            return QSA_ERR_INVALID_ARG;
        return from_cuda(launch_dense_decode(a, workspace, st));
    }
    if (dense_tc_ok(a)) {
        if (!workspace || !aligned(workspace, 256) || workspace_bytes < dense_tc_workspace())
            return QSA_ERR_INVALID_ARG;
        return launch_dense_tc(a, workspace, st);
    }
    return from_cuda(launch_dense_attn(a, st));
}

// Enough for whichever kernel a call of this shape takes.
size_t attn_workspace(int64_t n_tok, int64_t n_seq, int H_q, int H_kv, int d)
{
    if (n_tok <= 0 || n_seq <= 0 || H_q < 1 || H_kv < 1 || d < 1) return 0;
    return std::max({dense_decode_workspace(), dense_tc_workspace(), dense_few_workspace(), few_four_workspace()});
}

}  // namespace

extern "C" {

qsa_status qsa_paged_write(const qsa_paged_cache *cache, const int32_t *table, int64_t ld_table,
                           int64_t n_seq, const int32_t *cu_q, const int32_t *kv_len,
                           const void *k, const void *v, qsa_dtype src_dtype, int64_t n_tok,
                           int64_t ld_k, int64_t ld_v, qsa_stream_t stream)
{
    qsa_status s = check_cache(cache);
    if (s != QSA_OK) return s;
    s = check_seqs(table, ld_table, n_seq, kv_len, n_tok);
    if (s != QSA_OK) return s;
    const int64_t width = (int64_t)cache->H_kv * cache->d;
    if (!cu_q || !aligned(cu_q, 4) || !float_type(src_dtype) || !rows_ok(k, ld_k, width, src_dtype) ||
        !rows_ok(v, ld_v, width, src_dtype))
        return QSA_ERR_INVALID_ARG;
    if (n_tok == 0) return QSA_OK;
    const SeqView sv = {cu_q, kv_len, (int32_t)n_seq, n_tok};
    if (cache->dtype == QSA_E2M1)
        return from_cuda(launch_paged_append(nullptr, k, v, src_dtype, 0, ld_k, ld_v, 0, cache->d, 0, 1.0, nullptr,
                                             nullptr, nullptr, sv, view_of(cache, table, ld_table), cache->dtype,
                                             (cudaStream_t)stream));
    return from_cuda(launch_paged_write(k, v, src_dtype, ld_k, ld_v, cache->d, sv,
                                        view_of(cache, table, ld_table), cache->dtype,
                                        (cudaStream_t)stream));
}

qsa_status qsa_paged_append(const qsa_paged_cache *cache, const int32_t *table, int64_t ld_table,
                            int64_t n_seq, const int32_t *cu_q, const int32_t *kv_len,
                            const void *q, const void *k, const void *v, qsa_dtype src_dtype,
                            int64_t n_tok, int H_q, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                            const int32_t *pos, int rot, double base, void *q_out, void *k_out,
                            qsa_stream_t stream)
{
    qsa_status s = check_cache(cache);
    if (s != QSA_OK) return s;
    s = check_seqs(table, ld_table, n_seq, kv_len, n_tok);
    if (s != QSA_OK) return s;
    const int64_t width = (int64_t)cache->H_kv * cache->d;
    if (!cu_q || !aligned(cu_q, 4) || !float_type(src_dtype) || !rows_ok(k, ld_k, width, src_dtype) ||
        !rows_ok(v, ld_v, width, src_dtype) || !aligned(pos, 4) || rot < 0 || rot > cache->d || rot % 16 ||
        !(base >= 1.0) || !std::isfinite(base) || !aligned(k_out, 16))
        return QSA_ERR_INVALID_ARG;
    if (q && (H_q < 1 || !q_out || !aligned(q_out, 16) || !rows_ok(q, ld_q, (int64_t)H_q * cache->d, src_dtype)))
        return QSA_ERR_INVALID_ARG;
    if (q && (int64_t)H_q * cache->d > (1 << 24)) return QSA_ERR_UNSUPPORTED;
    // in place only where a token's row lies where its output goes
    if ((q && q == q_out && n_tok > 1 && ld_q != (int64_t)H_q * cache->d) || (k == k_out && n_tok > 1 && ld_k != width))
        return QSA_ERR_INVALID_ARG;
    if (n_tok == 0) return QSA_OK;
    const SeqView sv = {cu_q, kv_len, (int32_t)n_seq, n_tok};
    return from_cuda(launch_paged_append(q, k, v, src_dtype, ld_q, ld_k, ld_v, q ? H_q : 0, cache->d, rot, base, pos,
                                         q_out, k_out, sv, view_of(cache, table, ld_table), cache->dtype,
                                         (cudaStream_t)stream));
}

qsa_status qsa_paged_read(const qsa_paged_cache *cache, const int32_t *table, int64_t ld_table,
                          int64_t n_seq, const int32_t *kv_len, const int32_t *seq,
                          const int32_t *pos, const int32_t *n_cells, int64_t n_list,
                          int64_t max_cells, void *K_out, void *V_out, qsa_dtype out_dtype,
                          qsa_stream_t stream)
{
    qsa_status s = check_cache(cache);
    if (s != QSA_OK) return s;
    s = check_seqs(table, ld_table, n_seq, kv_len, 0);
    if (s != QSA_OK) return s;
    if (!n_cells || !K_out || !V_out || n_list < 0 || max_cells < 0 || !float_type(out_dtype) ||
        !aligned(n_cells, 4) || !aligned(seq, 4) || !aligned(pos, 4) || !aligned(K_out, 16) ||
        !aligned(V_out, 16))
        return QSA_ERR_INVALID_ARG;
    if (n_list == 0 || max_cells == 0) return QSA_OK;
    if (n_list > kMaxInt || max_cells > kMaxInt / n_list) return QSA_ERR_UNSUPPORTED;
    return from_cuda(launch_paged_read(view_of(cache, table, ld_table), cache->dtype, cache->d, seq,
                                       kv_len, n_seq, pos, n_cells, n_list, max_cells, K_out, V_out,
                                       out_dtype, (cudaStream_t)stream));
}

size_t qsa_paged_attn_workspace_size(int64_t n_tok, int64_t n_seq, int64_t max_q, int H_q, int H_kv,
                                     int d)
{
    (void)max_q;
    return attn_workspace(n_tok, n_seq, H_q, H_kv, d);
}

qsa_status qsa_paged_attn(const qsa_paged_cache *cache, const int32_t *table, int64_t ld_table,
                          int64_t n_seq, const int32_t *cu_q, const int32_t *kv_len, const void *q,
                          qsa_dtype q_dtype, int64_t n_tok, int64_t max_q, int64_t ld_q, int H_q,
                          float scale, int causal, void *out, float *lse_out, void *workspace,
                          size_t workspace_bytes, qsa_stream_t stream)
{
    qsa_status s = check_cache(cache);
    if (s != QSA_OK) return s;
    s = check_seqs(table, ld_table, n_seq, kv_len, n_tok);
    if (s != QSA_OK) return s;
    if (!cu_q || !aligned(cu_q, 4) || !float_type(q_dtype) || H_q < 1 || H_q % cache->H_kv ||
        max_q < 0 || (max_q == 0 && n_tok > 0) ||
        !rows_ok(q, ld_q, (int64_t)H_q * cache->d, q_dtype) || !out || !aligned(out, 16) ||
        !aligned(lse_out, 4))
        return QSA_ERR_INVALID_ARG;
    if (n_tok == 0) return QSA_OK;
    DenseArgs a;
    a.kv = view_of(cache, table, ld_table);
    a.sv = {cu_q, kv_len, (int32_t)n_seq, n_tok};
    a.kv_dtype = cache->dtype;
    a.q_dtype = q_dtype;
    a.q = q;
    a.ld_q = ld_q;
    a.out = out;
    a.lse = lse_out;
    a.H_q = H_q;
    a.d = cache->d;
    a.scale = scale;
    a.causal = causal != 0;
    a.pool_rows = cache->n_pages * cache->page_size;
    return run_attn(a, max_q, workspace, workspace_bytes, (cudaStream_t)stream);
}

qsa_status qsa_paged_sparse_attn(const qsa_paged_cache *cache, const int32_t *table, int64_t ld_table,
                                 int64_t n_seq, const int32_t *cu_q, const int32_t *kv_len,
                                 const int32_t *blocks, const int32_t *counts, int64_t k_blk,
                                 const void *q, qsa_dtype q_dtype, int64_t n_tok, int64_t ld_q,
                                 int H_q, float scale, void *out, float *lse_out,
                                 qsa_stream_t stream)
{
    qsa_status s = check_cache(cache);
    if (s != QSA_OK) return s;
    s = check_seqs(table, ld_table, n_seq, kv_len, n_tok);
    if (s != QSA_OK) return s;
    if (!cu_q || !aligned(cu_q, 4) || k_blk < 0 || (k_blk > 0 && !blocks) || !counts || !aligned(blocks, 4) ||
        !aligned(counts, 4) || !float_type(q_dtype) || H_q < 1 || H_q % cache->H_kv ||
        !rows_ok(q, ld_q, (int64_t)H_q * cache->d, q_dtype) || !out || !aligned(out, 16) || !aligned(lse_out, 4))
        return QSA_ERR_INVALID_ARG;
    if (k_blk > (1 << 28) || n_tok > kMaxInt / 8 / cache->H_kv || (int64_t)H_q * cache->d > (1 << 24))
        return QSA_ERR_UNSUPPORTED;
    if (n_tok == 0) return QSA_OK;
    SparseArgs a;
    a.kv = view_of(cache, table, ld_table);
    a.sv = {cu_q, kv_len, (int32_t)n_seq, n_tok};
    a.kv_dtype = cache->dtype;
    a.q_dtype = q_dtype;
    a.blocks = blocks;
    a.counts = counts;
    a.k_blk = k_blk;
    a.q = q;
    a.ld_q = ld_q;
    a.out = out;
    a.lse = lse_out;
    a.H_q = H_q;
    a.d = cache->d;
    a.scale = scale;
    return from_cuda(launch_paged_sparse(a, (cudaStream_t)stream));
}

size_t qsa_prompt_attn_workspace_size(int64_t n_tok, int64_t n_seq, int H_q, int H_kv, int d)
{
    return attn_workspace(n_tok, n_seq, H_q, H_kv, d);
}

qsa_status qsa_prompt_attn(const void *q, const void *k, const void *v, qsa_dtype dtype,
                           int64_t n_tok, int64_t ld_q, int64_t ld_k, int64_t ld_v,
                           const int32_t *cu_seq, int64_t n_seq, int H_q, int H_kv, int d,
                           float scale, int causal, void *out, float *lse_out, void *workspace,
                           size_t workspace_bytes, qsa_stream_t stream)
{
    if (!float_type(dtype) || n_tok < 0 || n_seq < 0 || (n_seq < 1 && n_tok > 0) || H_kv < 1 ||
        H_q < 1 || H_q % H_kv || d < 8 || d % 8 || !cu_seq || !aligned(cu_seq, 4) ||
        !rows_ok(q, ld_q, (int64_t)H_q * d, dtype) || !rows_ok(k, ld_k, (int64_t)H_kv * d, dtype) ||
        !rows_ok(v, ld_v, (int64_t)H_kv * d, dtype) || !out || !aligned(out, 16) ||
        !aligned(lse_out, 4))
        return QSA_ERR_INVALID_ARG;
    if (d > 256 || n_seq >= kMaxInt || n_tok > kMaxInt) return QSA_ERR_UNSUPPORTED;
    if (n_tok == 0) return QSA_OK;
    DenseArgs a = {};
    a.kv.K = k;
    a.kv.V = v;
    a.kv.ld_k = ld_k;
    a.kv.ld_v = ld_v;
    a.kv.H_kv = H_kv;
    a.sv = {cu_seq, nullptr, (int32_t)n_seq, n_tok};
    a.kv_dtype = dtype;
    a.q_dtype = dtype;
    a.q = q;
    a.ld_q = ld_q;
    a.out = out;
    a.lse = lse_out;
    a.H_q = H_q;
    a.d = d;
    a.scale = scale;
    a.causal = causal != 0;
    a.pool_rows = n_tok;
    return run_attn(a, n_tok, workspace, workspace_bytes, (cudaStream_t)stream);
}

qsa_status qsa_draft_verify(const float *target, int64_t ld_target, const float *draft,
                            int64_t ld_draft, const int32_t *tokens, const int32_t *n_draft,
                            const float *u, int64_t n_seq, int64_t max_draft, int64_t vocab,
                            int32_t *tokens_out, int32_t *n_accepted, qsa_stream_t stream)
{
    if (!target || !u || !tokens_out || !n_accepted || n_seq < 0 || max_draft < 0 || vocab < 1 ||
        (!tokens && max_draft > 0) || ld_target < vocab || (draft && ld_draft < vocab) ||
        !aligned(target, 4) || !aligned(draft, 4) || !aligned(tokens, 4) || !aligned(n_draft, 4) ||
        !aligned(u, 4) || !aligned(tokens_out, 4) || !aligned(n_accepted, 4))
        return QSA_ERR_INVALID_ARG;
    if (vocab > kMaxInt - 1024 || max_draft >= kMaxInt || n_seq > kMaxInt / 8 ||
        (n_seq > 0 && max_draft + 1 > kMaxInt / n_seq))
        return QSA_ERR_UNSUPPORTED;
    if (n_seq == 0) return QSA_OK;
    return from_cuda(launch_draft_verify(target, ld_target, draft, ld_draft, tokens, n_draft, u, n_seq,
                                         max_draft, vocab, tokens_out, n_accepted,
                                         (cudaStream_t)stream));
}

}  // extern "C"
