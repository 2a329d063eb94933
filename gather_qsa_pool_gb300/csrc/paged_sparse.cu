// paged_sparse.cu -- attention of each token over the blocks listed for it, in place on a paged cache: the kernel of
// few_cells.cuh, a cluster of CTAs for each token and KV head.
#include "few_cells.cuh"
#include "paged.cuh"

namespace qsa {
namespace {

template <int C, typename TQ, int NB, int NT>
cudaError_t run(const SparseArgs &a, cudaStream_t st)
{
    using P = few::Plan<C, NB, NT>;
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr auto kernel = few::few_cells_kernel<C, TQ, NB, NT, true>;
    // (a head's queries and results take shared memory: four heads' as far as three CTAs fit an SM)
    constexpr int kMost = C == QSA_BF16 || NB * NT > 4 ? 0 : (NB * NT > 2 ? 1 : 2);
    cudaError_t e = ensure_kernel_attrs<few::few_cells_kernel<C, TQ, NB, NT, true>>(few::few_cells_smem<C, NB, NT, true>(1 << kMost));
    if (e != cudaSuccess) return e;
    // CTAs of a token and its heads: as many as fill the GPU, a tile each at most, up to the portable cluster's
    // eight; the heads of a row go to one CTA where that leaves enough CTAs
    const int64_t most = (int64_t)P::kCtas * device_sm_count();
    int hl = kMost;
    while (hl > 0 && a.kv.H_kv % (1 << hl)) --hl;
    while (hl > 0 && (a.sv.n_tok * a.kv.H_kv >> hl) * 8 < most) --hl;
    const int kt = (few::kWarps >> hl) * few::Cell<C>::kKeys;
    const WorkShape ws = {1, kt, 0, a.kv.H_kv >> hl, 1, 0};
    const int64_t items = a.sv.n_tok * ws.H_kv, tiles = a.k_blk / (kt / 4) + 1;
    int64_t parts = most / items;
    if (parts > tiles) parts = tiles;
    if (parts > 8) parts = 8;
    if (parts < 1) parts = 1;
    return launch(kernel, dim3((unsigned)(items * parts)), dim3(few::kThreads), few::few_cells_smem<C, NB, NT, true>(1 << hl), st,
                  (int)parts, a.kv, a.sv, ws, ListView{a.blocks, a.counts, a.k_blk}, static_cast<const TQ *>(a.q), a.ld_q,
                  a.H_q, scale, q_sign, static_cast<TQ *>(a.out), a.lse, (float *)nullptr, (Split *)nullptr, 0, hl, (C == QSA_BF16 ? 6 : 7) - hl);
}

template <int C>
cudaError_t run_cells(const SparseArgs &a, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv;
    constexpr int NT = C == QSA_BF16 ? 3 : 2;
    if (a.q_dtype == QSA_F32) {
        if (G <= 8) return run<C, float, 1, NT>(a, st);
        return G <= 16 ? run<C, float, 2, NT>(a, st) : run<C, float, 4, NT>(a, st);
    }
    if (G <= 8) return run<C, __nv_bfloat16, 1, 1>(a, st);
    return G <= 16 ? run<C, __nv_bfloat16, 2, 1>(a, st) : run<C, __nv_bfloat16, 4, 1>(a, st);
}

}  // namespace

cudaError_t launch_paged_sparse(const SparseArgs &a, cudaStream_t st)
{
    // rows in 16-byte chunks, strides in 32 bits
    const int chunk = a.kv_dtype == QSA_E2M1 ? 32 : (a.kv_dtype == QSA_E4M3 ? 16 : 8);
    const bool fine = a.d == few::kD && a.H_q / a.kv.H_kv <= 32 && a.kv.ld_k % chunk == 0 && a.kv.ld_v % chunk == 0 &&
                      a.kv.ld_k <= (1 << 28) && a.kv.ld_v <= (1 << 28);
    if (fine && a.kv_dtype == QSA_BF16) return run_cells<QSA_BF16>(a, st);
    if (fine && a.kv_dtype == QSA_E4M3) return run_cells<QSA_E4M3>(a, st);
    if (fine && a.kv_dtype == QSA_E2M1) return run_cells<QSA_E2M1>(a, st);
    DenseArgs d;
    d.kv = a.kv;
    d.sv = a.sv;
    d.kv_dtype = a.kv_dtype;
    d.q_dtype = a.q_dtype;
    d.q = a.q;
    d.ld_q = a.ld_q;
    d.out = a.out;
    d.lse = a.lse;
    d.H_q = a.H_q;
    d.d = a.d;
    d.scale = a.scale;
    d.causal = 1;
    d.pool_rows = 0;
    d.list = {a.blocks, a.counts, a.k_blk};
    return launch_dense_attn(d, st);
}

}  // namespace qsa
