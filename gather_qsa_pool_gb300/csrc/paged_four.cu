// paged_four.cu -- attention of a few new tokens per sequence over a 4-bit paged cache: the kernel of few_cells.cuh
// over the flattened list of (sequence, KV head, row tile) items, whose parts dense_join.cuh joins.
#include "few_cells.cuh"

namespace qsa {
namespace {

constexpr int kMaxCtas = 3 * kTargetSMs;

// KV heads of a CTA, as a power of two.
int heads_log2(int H_kv) { return H_kv % 4 == 0 ? 2 : (H_kv % 2 == 0 ? 1 : 0); }

template <typename TQ, int NB, int NT>
cudaError_t run(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    using P = few::Plan<QSA_E2M1, NB, NT>;
    const int G = a.H_q / a.kv.H_kv, hl = heads_log2(a.kv.H_kv), hpc = 1 << hl;
    DenseArgs b = a;  // as the work list and the join see it: hpc KV heads are one
    b.kv.H_kv >>= hl;
    static_assert(few::kWarps * few::Cell<QSA_E2M1>::kKeys == 1 << 7, "a tile of one head");
    const WorkShape ws = work_shape(b, 8 * NB / G, (1 << 7) >> hl, 0);
    // the kernel takes a positive scale: a negative one turns the queries' signs, zero clears them
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr auto kernel = few::few_cells_kernel<QSA_E2M1, TQ, NB, NT, false>;
    cudaError_t e = ensure_kernel_attrs<few::few_cells_kernel<QSA_E2M1, TQ, NB, NT, false>>(
        few::few_cells_smem<QSA_E2M1, NB, NT, false>(few::kWarps));
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count(), ctas = P::kCtas * (sms < kTargetSMs ? sms : kTargetSMs);
    Split *splits = static_cast<Split *>(workspace);
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + kMaxCtas * sizeof(Split));
    e = launch(kernel, dim3((unsigned)ctas), dim3(few::kThreads), few::few_cells_smem<QSA_E2M1, NB, NT, false>(hpc), st, 1, a.kv,
               a.sv, ws, a.list, static_cast<const TQ *>(a.q), a.ld_q, a.H_q, scale, q_sign, static_cast<TQ *>(a.out),
               a.lse, partial, splits, (int)join_by_item(b, ws.rt, ctas), hl, 7 - hl);
    if (e != cudaSuccess) return e;
    return launch_dense_join<TQ>(splits, partial, ctas, 8 * NB * hpc, ws.rt, b, st);
}

}  // namespace

bool few_four_ok(const DenseArgs &a, int64_t max_q)
{
    const int G = a.H_q / a.kv.H_kv;
    if (a.kv_dtype != QSA_E2M1 || a.d != few::kD || !a.kv.table || a.kv.ld_k % 32 || a.kv.ld_v % 32) return false;
    if (a.kv.ld_k > (1 << 28) || a.kv.ld_v > (1 << 28)) return false;  // strides in 32 bits
    // fp32 queries come here however many tokens they are; bf16 queries of more rows are the tcgen05 kernel's
    return G <= (a.q_dtype == QSA_F32 ? 16 : 32) && (a.q_dtype == QSA_F32 || max_q * G <= 64);
}

size_t few_four_workspace()
{
    // 128 rows at two CTAs per SM; of fewer rows three are no more
    return kMaxCtas * sizeof(Split) + (size_t)4 * kTargetSMs * partial_floats(128, few::kD) * sizeof(float);
}

cudaError_t launch_few_four(const DenseArgs &a, int64_t max_q, void *workspace, cudaStream_t st)
{
    const int64_t rows = max_q * (a.H_q / a.kv.H_kv);
    const int G = a.H_q / a.kv.H_kv;
    if (a.q_dtype == QSA_F32)
        return rows <= 8 ? run<float, 1, 2>(a, workspace, st) : run<float, 2, 2>(a, workspace, st);
    if (rows <= 8) return run<__nv_bfloat16, 1, 1>(a, workspace, st);
    if (rows <= 16 && G <= 16) return run<__nv_bfloat16, 2, 1>(a, workspace, st);
    return run<__nv_bfloat16, 4, 1>(a, workspace, st);
}

}  // namespace qsa
