// dense_attn.cu -- attention over every visible cell, any shape: packed sequences with their
// own keys and values, or new tokens over a paged cache, fp32 arithmetic on the CUDA cores.
//
// For query token i of sequence s at position p = cells - tokens + i and head h (KV head
// g = h / G):  o = sum_j softmax_j(scale * q.k_j) v_j over the cells j <= p (all cells when not
// causal), lse = ln sum_j exp(scale * q.k_j).  One pass over the keys with a running maximum m
// and sum l: a tile with maximum m' moves m to max(m, m') and scales l and o by 2^(m - m').
// A row that sees nothing gives o = 0, lse = -inf.  A cell whose page is not in the pool makes
// its rows NaN.  With lists (LIST) a token's cells are those of its listed blocks and of its open block.
//
// One CTA per 16 rows (query tokens x heads of one KV head) and KV head; tiles of 32 cells in
// shared memory as fp32; eight threads per row.  It carries what the tensor-core kernels do
// not: fp32 queries or caches, head sizes other than theirs, any number of heads per KV head.
// Bound by shared-memory reads (one 16-byte read per four multiply-adds).
#include <cuda_fp8.h>

#include "e2m1.cuh"

namespace qsa {
namespace {

constexpr int kRows = 16;
constexpr int kKeys = 32;
constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float load1(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p, int64_t i)
{
    return __bfloat162float(p[i]);
}
__device__ __forceinline__ float load1(const uint8_t *p, int64_t i)
{
    const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)p[i], __NV_E4M3);
    return __half2float(__half(h));
}
// Value `e` of KV head g of pool row `row`, without the row's exponent.
template <typename TK>
__device__ __forceinline__ float load_cell(const KvView &kv, bool is_v, int64_t row, int g, int d, int e)
{
    return load1(static_cast<const TK *>(is_v ? kv.V : kv.K), row * (is_v ? kv.ld_v : kv.ld_k) + (int64_t)g * d + e);
}
struct E2m1Codes {
    uint8_t pair;
};
template <>
__device__ __forceinline__ float load_cell<E2m1Codes>(const KvView &kv, bool is_v, int64_t row, int g, int d, int e)
{
    const int64_t at = row * (is_v ? kv.ld_v : kv.ld_k) + (int64_t)g * d + e;
    const uint32_t h = half_of_codes<0>((uint32_t)static_cast<const uint8_t *>(is_v ? kv.V : kv.K)[at >> 1]);
    const float2 f = __half22float2(reinterpret_cast<const __half2 &>(h));
    return (e & 1 ? f.y : f.x) * scale_value((is_v ? kv.V_scale : kv.K_scale)[scale_row(kv, row, g) * (d / kGroup) + e / kGroup]);
}
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__host__ __device__ constexpr int pitch_of(int d) { return d + 4; }

size_t dense_smem(int d)
{
    return sizeof(float) * ((size_t)(kRows + 2 * kKeys) * pitch_of(d) + kRows * (kKeys + 1));
}

// LIST: each token over the cells of its listed blocks and its open block (an item is one token).
template <typename TQ, typename TK, bool LIST>
__global__ void __launch_bounds__(kThreads)
dense_attn_kernel(KvView kv, SeqView sv, WorkShape ws, ListView lv, const TQ *__restrict__ q, int64_t ld_q, int H_q,
                  int d, float scale_log2, TQ *__restrict__ out, float *__restrict__ lse)
{
    extern __shared__ __align__(16) float sm[];
    const int pitch = pitch_of(d);
    float *Qs = sm, *Ks = Qs + kRows * pitch, *Vs = Ks + kKeys * pitch, *Ps = Vs + kKeys * pitch;
    __shared__ WorkItem item_s;
    __shared__ int bad_s;
    __shared__ bool there_s[kKeys];  // LIST: there is a cell
    pdl_wait();
    QSA_AFTER_WAIT(q);
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = H_q / kv.H_kv;
    if (warp == 0) {
        // one place per item, one item per CTA
        WorkItem it;
        int64_t per, x0, x1;
        if constexpr (LIST) {
            int p, c;
            it.g = (int)(blockIdx.x % (unsigned)kv.H_kv);
            if (!token_place(sv, blockIdx.x / (unsigned)kv.H_kv, it.s, p, c)) it.s = -1;
            it.t = p;
            it.tiles = c;
        } else if (!work_share(sv, ws, blockIdx.x, gridDim.x, per, x0, x1, it)) {
            it.s = -1;
        }
        if (lane == 0) {
            item_s = it;
            bad_s = 0;
        }
    }
    __syncthreads();
    WorkItem it = item_s;
    if (it.s < 0) return;
    int64_t t0;
    int len, cells, n_list = 0, last = 0;
    const int32_t *list = nullptr;
    if constexpr (LIST) {
        t0 = blockIdx.x / (unsigned)kv.H_kv;
        len = 1;
        cells = it.tiles;
        last = it.t;  // the token's position
        it.t = 0;
        n_list = (int)min((int64_t)max(lv.counts[t0], 0), lv.k_blk);
        list = lv.blocks + t0 * lv.k_blk;
    } else {
        seq_tokens(sv, it.s, t0, len);
        cells = seq_cells(sv, it.s, len);
    }
    const bool fits = cells_fit(kv, cells);
    const int n_see = !fits ? 0 : (LIST ? 4 * n_list + 4 : item_cells(ws, len, cells, it.t));
    // rows of one tile may be more than 16 when G > 16: a second grid dimension cuts them
    const int row0 = blockIdx.y * kRows;
    const int rows_item = min(ws.rt, len - it.t * ws.rt) * G;
    if (row0 >= rows_item) return;

    const int r = tid >> 3, sub = tid & 7;  // this thread's row and its place among the row's 8
    const int rr = row0 + r;
    const bool live = rr < rows_item;
    const int tok = it.t * ws.rt + (live ? rr / G : 0);
    const int h = it.g * G + (live ? rr % G : 0);
    // the last cell the row sees
    if constexpr (!LIST) last = live ? (ws.causal ? cells - len + tok : cells - 1) : -1;
    for (int e = tid; e < kRows * d; e += kThreads) {
        const int er = e / d, ed = e - er * d;
        float x = 0.0f;
        if (row0 + er < rows_item)
            x = load1(q, (t0 + it.t * ws.rt + (row0 + er) / G) * ld_q +
                             (int64_t)(it.g * G + (row0 + er) % G) * d + ed);
        Qs[er * pitch + ed] = x;
    }
    float m = -INFINITY, l = 0.0f;
    float o[32];  // dims 4 * sub + 32 * i .. + 3
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
    for (int j0 = 0; j0 < n_see; j0 += kKeys) {
        __syncthreads();
        const int nk = min(kKeys, n_see - j0);
        for (int j = warp; j < kKeys; j += kThreads / 32) {
            int64_t row = -2;
            if constexpr (LIST) {
                const int cell = j < nk ? list_cell(list, n_list, last, j0 + j) : -1;
                if (cell >= 0) row = cell_row(kv, it.s, t0, cell);
                if (lane == 0) there_s[j] = cell >= 0;
            } else {
                if (j < nk) row = cell_row(kv, it.s, t0, j0 + j);
            }
            if (row == -1 && lane == 0) bad_s = 1;
            float km = 1.0f, vm = 1.0f;
            if (sizeof(TK) == 1 && row >= 0) {
                km = two_to(min(max((int)kv.K_exp[row * kv.H_kv + it.g] - kExpBias, kExpMin), kExpMax));
                vm = two_to(min(max((int)kv.V_exp[row * kv.H_kv + it.g] - kExpBias, kExpMin), kExpMax));
            }
            for (int e = lane; e < d; e += 32) {
                Ks[j * pitch + e] = row >= 0 ? load_cell<TK>(kv, false, row, it.g, d, e) * km : 0.0f;
                Vs[j * pitch + e] = row >= 0 ? load_cell<TK>(kv, true, row, it.g, d, e) * vm : 0.0f;
            }
        }
        __syncthreads();
        // logits of keys sub, sub + 8, sub + 16, sub + 24 (log2 units)
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int e = 0; e < d; e += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(&Qs[r * pitch + e]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 b = *reinterpret_cast<const float4 *>(&Ks[(sub + 8 * i) * pitch + e]);
                s[i] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s[i]))));
            }
        }
        float mt = -INFINITY;
        bool seen[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = sub + 8 * i;
            seen[i] = LIST ? there_s[j] && live : j < nk && j0 + j <= last;
            s[i] *= scale_log2;
            if (seen[i]) mt = fmaxf(mt, s[i]);
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
        const float mn = fmaxf(m, mt);
        const float mu = mn == -INFINITY ? 0.0f : mn;
        const float alpha = exp2f(m - mu);  // m = -inf: 0
        float ls = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = seen[i] ? exp2f(s[i] - mu) : 0.0f;
            ls += p;
            // a negative weight marks a cell the row does not see: its value, whatever it
            // holds, is not multiplied
            Ps[r * (kKeys + 1) + sub + 8 * i] = seen[i] ? p : -1.0f;
        }
#pragma unroll
        for (int x = 1; x < 8; x <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, x);
        l = l * alpha + ls;
        m = mn;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= alpha;
        for (int j = 0; j < nk; ++j) {
            const float p = Ps[r * (kKeys + 1) + j];
            if (p < 0.0f) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = 4 * sub + 32 * i;
                if (e < d) {
                    const float4 v = *reinterpret_cast<const float4 *>(&Vs[j * pitch + e]);
                    o[4 * i] = fmaf(p, v.x, o[4 * i]);
                    o[4 * i + 1] = fmaf(p, v.y, o[4 * i + 1]);
                    o[4 * i + 2] = fmaf(p, v.z, o[4 * i + 2]);
                    o[4 * i + 3] = fmaf(p, v.w, o[4 * i + 3]);
                }
            }
        }
    }
    __syncthreads();
    const bool bad = bad_s != 0 || !fits;
    if (!live) return;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // a NaN sum stays NaN
    TQ *dst = out + ((t0 + tok) * H_q + h) * (int64_t)d;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int e = 4 * sub + 32 * (i >> 2) + (i & 3);
        if (e < d) store1(dst + e, bad ? NAN : o[i] * inv);
    }
    if (lse && sub == 0)
        lse[(t0 + tok) * H_q + h] = bad ? NAN : (l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2);
}

template <typename TQ, typename TK, bool LIST>
cudaError_t run(const DenseArgs &a, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv;
    const WorkShape ws = work_shape(a, LIST || G >= kRows ? 1 : kRows / G, 0, 0);
    const size_t smem = dense_smem(a.d);
    cudaError_t e = ensure_kernel_attrs<dense_attn_kernel<TQ, TK, LIST>>(smem);
    if (e != cudaSuccess) return e;
    // no more row tiles than this whatever the lengths are
    const int64_t items = LIST ? a.sv.n_tok * a.kv.H_kv : ((a.sv.n_tok + ws.rt - 1) / ws.rt + a.sv.n_seq) * a.kv.H_kv;
    const int64_t parts = ((int64_t)ws.rt * G + kRows - 1) / kRows;
    return launch(dense_attn_kernel<TQ, TK, LIST>, dim3((unsigned)items, (unsigned)parts), dim3(kThreads), smem,
                  st, 1, a.kv, a.sv, ws, a.list, static_cast<const TQ *>(a.q), a.ld_q, a.H_q, a.d,
                  a.scale * kLog2e, static_cast<TQ *>(a.out), a.lse);
}

template <typename TQ, bool LIST>
cudaError_t run_q(const DenseArgs &a, cudaStream_t st)
{
    switch (a.kv_dtype) {
        case QSA_E2M1: return run<TQ, E2m1Codes, LIST>(a, st);
        case QSA_E4M3: return run<TQ, uint8_t, LIST>(a, st);
        case QSA_BF16: return run<TQ, __nv_bfloat16, LIST>(a, st);
        default: return run<TQ, float, LIST>(a, st);
    }
}

}  // namespace

cudaError_t launch_dense_attn(const DenseArgs &a, cudaStream_t st)
{
    if (a.list.counts) return a.q_dtype == QSA_BF16 ? run_q<__nv_bfloat16, true>(a, st) : run_q<float, true>(a, st);
    return a.q_dtype == QSA_BF16 ? run_q<__nv_bfloat16, false>(a, st) : run_q<float, false>(a, st);
}

}  // namespace qsa
