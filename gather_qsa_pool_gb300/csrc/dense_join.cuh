// dense_join.cuh -- the parts of an item that several CTAs of an attention kernel computed,
// joined: with the parts' references m_k, sums l_k and unnormalised outputs o_k of a row,
//   m = max m_k,  l = sum 2^(m_k - m) l_k,  out = sum 2^(m_k - m) o_k / l.
// Reads what the parts wrote once; with few parts bound by the launch.
#pragma once

#include "dense.cuh"
#include "mma_frag.cuh"

namespace qsa {

// An item cut into parts: they are the second record of the CTA where it begins and the first
// records of the CTAs after it.
struct Split {
    int32_t s, g, t;   // sequence (below 0: not cut), KV head, row tile
    int32_t cta;       // where it begins
    int32_t parts;
    int32_t pad[3];
};

// A split's place in the list: the item's number while there are no more items than CTAs (few items
// in many parts: the joining kernel then has work for every CTA it launches), else the CTA where it
// begins (a CTA begins at most one item that it does not end).
inline bool join_by_item(const DenseArgs &a, int rt, int ctas)
{
    return ((a.sv.n_tok + rt - 1) / rt + a.sv.n_seq) * a.kv.H_kv <= ctas;
}

// Called once for each item, by the CTA where it begins.
__device__ __forceinline__ void note_split(Split *splits, int by_item, const WorkItem &it, bool whole, int64_t last_cta)
{
    if (whole && !by_item) return;  // (a CTA's entry was cleared at its start)
    Split sp = {whole ? -1 : it.s, it.g, it.t, (int32_t)blockIdx.x, (int32_t)(last_cta - blockIdx.x) + 1, {0, 0, 0}};
    splits[by_item ? it.index : (int64_t)blockIdx.x] = sp;
}

// One warp per part and row: kParts warps take every kParts-th part of a row (many parts: a long
// context's few rows), 8 / kParts rows at a time.  A record's rows lie in groups of 128, `group`
// tokens each.
template <typename TQ, int kParts>
__global__ void __launch_bounds__(256)
dense_join_kernel(const Split *__restrict__ splits, const float *__restrict__ partial, int rows_max,
                  const SeqView sv, int rt, int group, int H_kv, int G, int by_item, TQ *__restrict__ out,
                  float *__restrict__ lse)
{
    constexpr int kD = 128, kRows = 8 / kParts;
    __shared__ float red_m[8], red_l[8];
    __shared__ float4 red_o[8][32];
    pdl_wait();
    QSA_AFTER_WAIT(splits);
    QSA_AFTER_WAIT(partial);
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = warp % kParts, H_q = H_kv * G;
    if (by_item) {
        // fewer items than the host could tell have no entry
        int64_t items = 0;
        for (int s = lane; s < sv.n_seq; s += 32) {
            int64_t t0;
            int len;
            seq_tokens(sv, s, t0, len);
            items += (len + rt - 1) / rt;
        }
        if ((int64_t)blockIdx.x >= warp_sum_i64(items) * H_kv) return;
    }
    const Split sp = splits[blockIdx.x];
    if (sp.s < 0) return;
    const int c = sp.cta;
    int64_t t0;
    int len;
    seq_tokens(sv, sp.s, t0, len);
    const int64_t rec = partial_floats(rows_max, kD);
    const int r = blockIdx.y * kRows + warp / kParts;
    const int tok = sp.t * rt + (r >> 7) * group + (r & 127) / G;
    const bool live = (r & 127) < group * G && (r >> 7) * group < rt && tok < len;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = part; live && k < sp.parts; k += kParts) {
        const float *p = partial + (2 * (int64_t)(c + k) + (k == 0 ? 1 : 0)) * rec;
        const float pm = p[r], pl = p[rows_max + r];
        const float4 po = *reinterpret_cast<const float4 *>(p + 2 * rows_max + (int64_t)r * kD + 4 * lane);
        const float mn = fmaxf(m, pm), u = mn == -INFINITY ? 0.0f : mn;
        const float a = m == -INFINITY ? 1.0f : exp2f(m - u);  // an unset side is zero or NaN
        const float b = pm == -INFINITY ? 1.0f : exp2f(pm - u);
        l = l * a + pl * b;
        o.x = o.x * a + po.x * b;
        o.y = o.y * a + po.y * b;
        o.z = o.z * a + po.z * b;
        o.w = o.w * a + po.w * b;
        m = mn;
    }
    if constexpr (kParts > 1) {
        if (lane == 0) {
            red_m[warp] = m;
            red_l[warp] = l;
        }
        red_o[warp][lane] = o;
        __syncthreads();
        if (part != 0) return;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kParts; ++w) M = fmaxf(M, red_m[warp + w]);
        const float u = M == -INFINITY ? 0.0f : M;
        l = 0.0f;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kParts; ++w) {
            const float a = red_m[warp + w] == -INFINITY ? 1.0f : exp2f(red_m[warp + w] - u);
            const float4 p = red_o[warp + w][lane];
            l += red_l[warp + w] * a;
            o.x += p.x * a;
            o.y += p.y * a;
            o.z += p.z * a;
            o.w += p.w * a;
        }
        m = M;
    }
    if (!live) return;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // a NaN sum stays NaN
    const int64_t at = (t0 + tok) * H_q + sp.g * G + (r & 127) % G;
    TQ *dst = out + at * kD + 4 * lane;
    if constexpr (sizeof(TQ) == 2) {
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    } else {
        *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
    if (lane == 0 && lse) lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename TQ, int kParts>
cudaError_t launch_join(const Split *splits, const float *partial, int entries, int by_item, int rows_max, int group,
                        const DenseArgs &a, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv, rt = rows_max > 128 ? 2 * group : group;
    constexpr int kRows = 8 / kParts;
    return launch(dense_join_kernel<TQ, kParts>,
                  dim3((unsigned)entries, (unsigned)((rows_max + kRows - 1) / kRows)), dim3(256), 0, st, 1, splits,
                  partial, rows_max, a.sv, rt, group, a.kv.H_kv, G, by_item, static_cast<TQ *>(a.out), a.lse);
}

// ctas: CTAs of the attention kernel; group: tokens of a record's 128 rows (of all its rows where
// it has fewer).  As many warps on a row as the items have parts, about.
template <typename TQ>
cudaError_t launch_dense_join(const Split *splits, const float *partial, int ctas, int rows_max, int group,
                              const DenseArgs &a, cudaStream_t st)
{
    const int rt = rows_max > 128 ? 2 * group : group;
    if (!join_by_item(a, rt, ctas)) return launch_join<TQ, 1>(splits, partial, ctas, 0, rows_max, group, a, st);
    const int items = (int)(((a.sv.n_tok + rt - 1) / rt + a.sv.n_seq) * a.kv.H_kv);
    if (items * 12 <= ctas) return launch_join<TQ, 8>(splits, partial, items, 1, rows_max, group, a, st);
    if (items * 3 <= ctas) return launch_join<TQ, 2>(splits, partial, items, 1, rows_max, group, a, st);
    return launch_join<TQ, 1>(splits, partial, items, 1, rows_max, group, a, st);
}

}  // namespace qsa
