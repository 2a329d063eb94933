// paged_rw.cu -- the paged key/value cache: rows of new tokens written into their pages
// (quantised to e4m3 on the way when the pool holds 8-bit codes) and listed cells read back.
//
// Mathematics of the 8-bit form: a row is the d values of one token and KV head.  With
// top = max |x| over the row's finite values, e is the least integer with top <= 448 * 2^e
// (448 = the largest e4m3 value), clamped to [-100, 100], and the codes are the e4m3 values
// nearest to x * 2^-e (ties to even; beyond 448 clamped, which only happens at e = 100;
// non-finite x becomes NaN).  A power of two as the row's scale makes x * 2^-e exact, so the
// only rounding is the one to four significant bits, at most 2^-4 of the value from 2^-6 of
// the code range up; a scale of top / 448 would round twice and gain nothing, as the codes are
// floating point themselves.  value = code * 2^e is exact in bf16 and fp32.
#include <cuda_fp8.h>

#include "dense.cuh"
#include "paged.cuh"

namespace qsa {
namespace {

__device__ __forceinline__ void store8(float *p, const float *x)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight e4m3 codes of x * 2^-e (inv = 2^-e), packed little-endian.
__device__ __forceinline__ uint2 encode8(const float *x, float inv)
{
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y0 = x[2 * i] * inv, y1 = x[2 * i + 1] * inv;
        // infinities become NaN (0 * inf); the conversion clamps finite values to 448
        y0 = isfinite(x[2 * i]) ? y0 : NAN;
        y1 = isfinite(x[2 * i + 1]) ? y1 : NAN;
        const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
        w[i >> 1] |= c << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(uint2 c, float mul, float *x)
{
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            (__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * i] = f.x * mul;
        x[2 * i + 1] = f.y * mul;
    }
}

// Exponent of a row from its largest finite magnitude.
__device__ __forceinline__ int row_exponent(float top)
{
    // top = m * 2^x with m in [1, 2): top <= 448 * 2^e = 1.75 * 2^(e + 8)
    const uint32_t u = __float_as_uint(top);
    const int x = (int)(u >> 23) - 127;  // subnormals and zero give -127: clamped below
    const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);
}

// ------------------------------------------------------------------ write
// Eight values per lane, d / 8 lanes per row (a power of two up to 32): a warp holds several
// rows at once, and a row's largest magnitude is a shuffle over its lanes.  One task is a
// token's row of K or of V for one KV head; consecutive tasks are consecutive in memory.
// Bound by the bytes of the rows (a source row read once, its codes written once); with few
// tokens by the launch.
template <typename TS, typename TD>
__global__ void __launch_bounds__(256)
paged_write_kernel(const TS *__restrict__ k, const TS *__restrict__ v, int64_t ld_k, int64_t ld_v,
                   int H, int d, int lanes_log2, SeqView sv, KvView kv, TD *K, TD *V,
                   uint8_t *K_exp, uint8_t *V_exp)
{
    pdl_wait();
    QSA_AFTER_WAIT(k);
    QSA_AFTER_WAIT(v);
    pdl_trigger();
    const int lanes = 1 << lanes_log2;  // lanes of a row; those beyond d / 8 idle
    const int64_t gt = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = (int)(gt & (lanes - 1));
    const bool on = c * 8 < d;
    const int64_t n_tasks = sv.n_tok * 2 * H;
    const int64_t stride = ((int64_t)gridDim.x * blockDim.x) >> lanes_log2;
    // every lane of a warp makes the same number of turns: the shuffles need all of them
    const int64_t first = gt >> lanes_log2;
    const int64_t turns = (n_tasks + stride - 1) / stride;
    for (int64_t i = 0; i < turns; ++i) {
        const int64_t task = first + i * stride;
        const bool live = task < n_tasks;
        const int64_t tok = live ? task / (2 * H) : 0;
        const int r = live ? (int)(task - tok * 2 * H) : 0;
        const bool is_v = r >= H;
        const int h = is_v ? r - H : r;
        // the token's sequence: the last s with cu[s] <= tok (binary search)
        int lo = 0, hi = sv.n_seq;  // answer in [lo, hi)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)sv.cu[mid] <= tok) lo = mid;
            else hi = mid;
        }
        int64_t row = -1;
        if (live) {
            const int64_t a = sv.cu[lo], b = sv.cu[lo + 1];
            const int64_t p = (int64_t)sv.kv_len[lo] - (b - tok);
            if (tok >= a && tok < b && p >= 0 && p < (int64_t)sv.kv_len[lo])
                row = cell_row(kv, lo, 0, (int)p);
        }
        float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (live && on)
            load8((is_v ? v + tok * ld_v : k + tok * ld_k) + (int64_t)h * d + 8 * c, x);
        TD *dst = (is_v ? V + row * kv.ld_v : K + row * kv.ld_k) + (int64_t)h * d + 8 * c;
        if constexpr (sizeof(TD) == 1) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, isfinite(x[j]) ? fabsf(x[j]) : 0.0f);
            for (int o = lanes >> 1; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int e = row_exponent(top);
            if (row >= 0 && on) *reinterpret_cast<uint2 *>(dst) = encode8(x, two_to(-e));
            if (row >= 0 && c == 0) (is_v ? V_exp : K_exp)[row * H + h] = (uint8_t)(e + kExpBias);
        } else {
            if (row >= 0 && on) store8(dst, x);
        }
    }
}

// ------------------------------------------------------------------ read
// One warp per listed cell, looping over the list: the cell's K and V rows of all KV heads are
// contiguous, so the lanes stream them 8 values each.  Bound by the bytes.
template <typename TS, typename TD>
__global__ void __launch_bounds__(256)
paged_read_kernel(KvView kv, int H, int d, const int32_t *__restrict__ seq,
                  const int32_t *__restrict__ kv_len, int64_t n_seq, const int32_t *__restrict__ pos,
                  const int32_t *__restrict__ n_cells, int64_t n_list, int64_t max_cells,
                  TD *__restrict__ K_out, TD *__restrict__ V_out)
{
    pdl_wait();
    QSA_AFTER_WAIT(seq);
    QSA_AFTER_WAIT(kv_len);
    QSA_AFTER_WAIT(pos);
    QSA_AFTER_WAIT(n_cells);
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int hd = H * d;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < n_list * max_cells;
         w += warps) {
        const int64_t i = w / max_cells, j = w - i * max_cells;
        if (j >= (int64_t)n_cells[i]) continue;
        const int64_t s = seq ? (int64_t)seq[i] : i;
        int64_t row = -1;
        if (s >= 0 && s < n_seq) {
            const int64_t p = pos ? (int64_t)pos[w] : j;
            if (p >= 0 && p < (int64_t)kv_len[s]) row = cell_row(kv, (int)s, 0, (int)p);
        }
        const TS *K = static_cast<const TS *>(kv.K), *V = static_cast<const TS *>(kv.V);
        for (int e = 8 * lane; e < 2 * hd; e += 256) {
            const bool is_v = e >= hd;
            const int at = is_v ? e - hd : e;
            float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (row >= 0) {
                const TS *src = (is_v ? V + row * kv.ld_v : K + row * kv.ld_k) + at;
                if constexpr (sizeof(TS) == 1) {
                    const int b = (is_v ? kv.V_exp : kv.K_exp)[row * H + at / d];
                    const int ex = min(max(b - kExpBias, kExpMin), kExpMax);
                    decode8(*reinterpret_cast<const uint2 *>(src), two_to(ex), x);
                } else {
                    load8(src, x);
                }
            }
            store8((is_v ? V_out : K_out) + w * hd + at, x);
        }
    }
}

template <typename TS>
cudaError_t write_to(const void *k, const void *v, int64_t ld_k, int64_t ld_v, int d, const SeqView &sv,
                     const KvView &kv, qsa_dtype cache_dtype, cudaStream_t st)
{
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < d) ++lanes_log2;
    const int64_t threads = sv.n_tok * 2 * kv.H_kv << lanes_log2;
    int64_t grid = (threads + 255) / 256;
    const int64_t most = (int64_t)device_sm_count() * 16;
    if (grid > most) grid = most;
    const TS *ks = static_cast<const TS *>(k), *vs = static_cast<const TS *>(v);
    uint8_t *ke = const_cast<uint8_t *>(kv.K_exp), *ve = const_cast<uint8_t *>(kv.V_exp);
    void *K = const_cast<void *>(kv.K), *V = const_cast<void *>(kv.V);
    const dim3 g((unsigned)grid), b(256);
    switch (cache_dtype) {
        case QSA_E4M3:
            return launch(paged_write_kernel<TS, uint8_t>, g, b, 0, st, 1, ks, vs, ld_k, ld_v, kv.H_kv, d,
                          lanes_log2, sv, kv, static_cast<uint8_t *>(K), static_cast<uint8_t *>(V), ke, ve);
        case QSA_BF16:
            return launch(paged_write_kernel<TS, __nv_bfloat16>, g, b, 0, st, 1, ks, vs, ld_k, ld_v,
                          kv.H_kv, d, lanes_log2, sv, kv, static_cast<__nv_bfloat16 *>(K),
                          static_cast<__nv_bfloat16 *>(V), ke, ve);
        default:
            return launch(paged_write_kernel<TS, float>, g, b, 0, st, 1, ks, vs, ld_k, ld_v, kv.H_kv, d,
                          lanes_log2, sv, kv, static_cast<float *>(K), static_cast<float *>(V), ke, ve);
    }
}

template <typename TS, typename TD>
cudaError_t read_to(const KvView &kv, int d, const int32_t *seq, const int32_t *kv_len, int64_t n_seq,
                    const int32_t *pos, const int32_t *n_cells, int64_t n_list, int64_t max_cells,
                    void *K_out, void *V_out, cudaStream_t st)
{
    int64_t grid = (n_list * max_cells + 7) / 8;
    const int64_t most = (int64_t)device_sm_count() * 8;
    if (grid > most) grid = most;
    return launch(paged_read_kernel<TS, TD>, dim3((unsigned)grid), dim3(256), 0, st, 1, kv, kv.H_kv, d,
                  seq, kv_len, n_seq, pos, n_cells, n_list, max_cells, static_cast<TD *>(K_out),
                  static_cast<TD *>(V_out));
}

}  // namespace

cudaError_t launch_paged_write(const void *k, const void *v, qsa_dtype src_dtype, int64_t ld_k,
                               int64_t ld_v, int d, const SeqView &sv, const KvView &kv,
                               qsa_dtype cache_dtype, cudaStream_t st)
{
    return src_dtype == QSA_BF16
               ? write_to<__nv_bfloat16>(k, v, ld_k, ld_v, d, sv, kv, cache_dtype, st)
               : write_to<float>(k, v, ld_k, ld_v, d, sv, kv, cache_dtype, st);
}

cudaError_t launch_paged_read(const KvView &kv, qsa_dtype cache_dtype, int d, const int32_t *seq,
                              const int32_t *kv_len, int64_t n_seq, const int32_t *pos,
                              const int32_t *n_cells, int64_t n_list, int64_t max_cells, void *K_out,
                              void *V_out, qsa_dtype out_dtype, cudaStream_t st)
{
    const bool f32 = out_dtype == QSA_F32;
    switch (cache_dtype) {
        case QSA_E4M3:
            return f32 ? read_to<uint8_t, float>(kv, d, seq, kv_len, n_seq, pos, n_cells, n_list,
                                                 max_cells, K_out, V_out, st)
                       : read_to<uint8_t, __nv_bfloat16>(kv, d, seq, kv_len, n_seq, pos, n_cells,
                                                         n_list, max_cells, K_out, V_out, st);
        case QSA_BF16:
            return f32 ? read_to<__nv_bfloat16, float>(kv, d, seq, kv_len, n_seq, pos, n_cells, n_list,
                                                       max_cells, K_out, V_out, st)
                       : read_to<__nv_bfloat16, __nv_bfloat16>(kv, d, seq, kv_len, n_seq, pos, n_cells,
                                                               n_list, max_cells, K_out, V_out, st);
        default:
            return f32 ? read_to<float, float>(kv, d, seq, kv_len, n_seq, pos, n_cells, n_list,
                                               max_cells, K_out, V_out, st)
                       : read_to<float, __nv_bfloat16>(kv, d, seq, kv_len, n_seq, pos, n_cells, n_list,
                                                       max_cells, K_out, V_out, st);
    }
}

}  // namespace qsa
