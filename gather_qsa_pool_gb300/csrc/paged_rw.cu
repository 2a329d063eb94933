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

// Eight consecutive source values as they lie in memory.
template <typename T>
struct Src8;
template <>
struct Src8<float> {
    uint32_t w[8];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const float *p)
    {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
    // the largest magnitude, as bits (an order of its own: NaN and infinities come out on top)
    __device__ __forceinline__ uint32_t top() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
        return m;
    }
};
template <>
struct Src8<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0u; }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
    __device__ __forceinline__ float at(int i) const
    {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ uint32_t top() const
    {
        const uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                    __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        return max(m & 0xffff0000u, m << 16);
    }
};
constexpr uint32_t kInfBits = 0x7f800000u;

// Eight e4m3 codes of x * 2^-e (inv = 2^-e), packed little-endian; the conversion clamps finite
// values to 448 and keeps NaN.  all: every value is finite; else infinities become NaN too.
template <typename T>
__device__ __forceinline__ uint2 encode8(const Src8<T> &x, float inv, bool all)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float2 z = mul2(make_float2(x.at(4 * i + j), x.at(4 * i + j + 1)), make_float2(inv, inv));
            y[j] = z.x;
            y[j + 1] = z.y;
        }
        if (!all) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = isfinite(x.at(4 * i + j)) ? y[j] : NAN;
        }
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = __byte_perm(lo, hi, 0x5410);
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

// Exponent of a row from the bits of its largest finite magnitude.
__device__ __forceinline__ int row_exponent(uint32_t u)
{
    // top = m * 2^x with m in [1, 2): top <= 448 * 2^e = 1.75 * 2^(e + 8)
    const int x = (int)(u >> 23) - 127;  // subnormals and zero give -127: clamped below
    const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, kExpMin), kExpMax);
}

// ------------------------------------------------------------------ write
// The largest of a head's magnitudes (as bits), of K and of V: over its `lanes` lanes.  bf16 values have
// both in one word.
template <typename TS>
__device__ __forceinline__ void head_max(uint32_t (&top)[2], int lanes)
{
    if constexpr (sizeof(TS) == 2) {
        uint32_t m = top[0] | top[1] >> 16;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < lanes) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        top[0] = m & 0xffff0000u;
        top[1] = m << 16;
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < lanes) {
                top[0] = max(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
                top[1] = max(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
            }
    }
}

// The sequence of token tok: the number of s with cu[s + 1] <= tok, 32 of them at a time.
__device__ __forceinline__ int token_seq(const SeqView &sv, int64_t tok)
{
    const int lane = threadIdx.x & 31;
    for (int s0 = 0;; s0 += 32) {
        const int s = s0 + lane;
        const bool behind = s < sv.n_seq && (int64_t)sv.cu[s + 1] <= tok;
        const int n = __popc(__ballot_sync(0xffffffffu, behind));
        if (n < 32) return s0 + n;
    }
}

// One warp per `group` consecutive tokens: its lanes look their cells up at once, then the warp takes
// the tokens' K and V rows of all KV heads, eight values a lane, d / 8 lanes per head (a power of two
// of them, up to 32), so a head's largest magnitude is a shuffle over its lanes (K's and V's of bf16
// rows in one word); four loads are in flight.  Prompts (26,900 tokens, 4 heads of 128, bf16 to e4m3):
// 19.8 us, 0.61 of the copy bandwidth; neither the memory nor issue slots (61%) nor a pipe (ALU 57%) is full:
// a warp's loads and its long encoding alternate, with nothing loaded ahead and 38% of the warps resident.
// With few tokens bound by the launch and the look-up's dependent loads.
template <typename TS, typename TD>
__global__ void __launch_bounds__(128, sizeof(TS) == 4 && sizeof(TD) == 1 ? 6 : 8)
paged_write_kernel(const TS *__restrict__ k, const TS *__restrict__ v, int64_t ld_k, int64_t ld_v,
                   int H, int d, int lanes_log2, int group, SeqView sv, KvView kv, TD *K, TD *V,
                   uint8_t *K_exp, uint8_t *V_exp)
{
    pdl_wait();
    QSA_AFTER_WAIT(k);
    QSA_AFTER_WAIT(v);
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int c = lane & ((1 << lanes_log2) - 1);    // this lane's eight values of a head
    const int heads = 32 >> lanes_log2;              // heads of a step
    const int per = (H + heads - 1) / heads;         // steps of a row
    const bool on = c * 8 < d;
    const int head = lane >> lanes_log2;             // of a step
    const int stride = heads * d, lane_at = head * d + 8 * c;
    const bool two = per == 1;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int64_t groups = (sv.n_tok + group - 1) / group;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < groups; w += warps) {
        const int64_t tok0 = w * group;
        const int n = (int)min((int64_t)group, sv.n_tok - tok0);
        int32_t mine = -1;  // pool row of token tok0 + lane
        const int first = token_seq(sv, tok0);
        if (lane < n) {
            const int64_t tok = tok0 + lane;
            int s = first;
            while (s < sv.n_seq && (int64_t)sv.cu[s + 1] <= tok) ++s;
            if (s < sv.n_seq && (int64_t)sv.cu[s] <= tok) {
                const int64_t len = sv.kv_len[s], p = len - ((int64_t)sv.cu[s + 1] - tok);
                if (p >= 0 && p < len) mine = (int32_t)cell_row(kv, s, 0, (int)p);
            }
        }
        for (int at = 0; at < n; at += two ? 2 : 1)
            for (int p = 0; p < per; p += 2) {
                // K and V of two steps of a token, or of two tokens with one step
                Src8<TS> x[2][2];
                bool live[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int tok = at + (two ? j : 0), step = p + (two ? 0 : j);
                    live[j] = on && tok < n && step * heads + head < H;
                    x[j][0].clear();
                    x[j][1].clear();
                    if (live[j]) {
                        x[j][0].load(k + (tok0 + tok) * ld_k + step * stride + lane_at);
                        x[j][1].load(v + (tok0 + tok) * ld_v + step * stride + lane_at);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int tok = at + (two ? j : 0), step = p + (two ? 0 : j);
                    const int64_t row = __shfl_sync(0xffffffffu, mine, tok);
                    const bool here = live[j] && row >= 0;
                    uint32_t top[2];
                    bool all = true;
                    if constexpr (sizeof(TD) == 1) {
                        top[0] = x[j][0].top();
                        top[1] = x[j][1].top();
                        all = !__any_sync(0xffffffffu, max(top[0], top[1]) >= kInfBits);
                        if (!all) {  // some value of the step is no number: the finite ones decide
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (i % 8 == 0) top[i / 8] = 0;
                                const uint32_t b = __float_as_uint(x[j][i / 8].at(i % 8)) & 0x7fffffffu;
                                top[i / 8] = b < kInfBits ? max(top[i / 8], b) : top[i / 8];
                            }
                        }
                        head_max<TS>(top, 1 << lanes_log2);
                    }
#pragma unroll
                    for (int is_v = 0; is_v < 2; ++is_v) {
                        const Src8<TS> &y = x[j][is_v];
                        TD *dst = (is_v ? V + row * kv.ld_v : K + row * kv.ld_k) + step * stride + lane_at;
                        if constexpr (sizeof(TD) == 1) {
                            const int e = row_exponent(top[is_v]);
                            if (here) *reinterpret_cast<uint2 *>(dst) = encode8(y, two_to(-e), all);
                            if (here && c == 0)
                                (is_v ? V_exp : K_exp)[row * H + step * heads + head] = (uint8_t)(e + kExpBias);
                        } else {
                            float f[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] = y.at(i);
                            if (here) store8(dst, f);
                        }
                    }
                }
            }
    }
}

// ------------------------------------------------------------------ read
// One warp per `group` listed cells: its lanes look the cells up at once, then the warp streams their
// K and V rows (all KV heads contiguous), kVec values a lane, four steps in flight.  With eight codes
// a lane the instructions of the conversion bound it (72% of issue slots at 74 us for whole sequences
// of 61,789 cells); with sixteen (d a multiple of 16) the bytes do.  With few cells: the look-up's
// dependent loads and one step's latency.
template <typename T, int kVec>
struct Raw {
    static constexpr int kWords = (int)sizeof(T) * kVec / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (kWords == 2) {
            const uint2 a = *reinterpret_cast<const uint2 *>(p);
            w[0] = a.x; w[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 a = reinterpret_cast<const uint4 *>(p)[i / 4];
                w[i] = a.x; w[i + 1] = a.y; w[i + 2] = a.z; w[i + 3] = a.w;
            }
        }
    }
    // values 8 i .. 8 i + 7, times mul where they are codes
    __device__ __forceinline__ void eight(int i, float mul, float *x) const
    {
        if constexpr (sizeof(T) == 1) {
            decode8(make_uint2(w[2 * i], w[2 * i + 1]), mul, x);
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = __uint_as_float(w[4 * i + j] << 16);
                x[2 * j + 1] = __uint_as_float(w[4 * i + j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[8 * i + j]);
        }
    }
};

template <typename TS, typename TD, int kVec>
__global__ void __launch_bounds__(128, 8)
paged_read_kernel(KvView kv, int H, int d, int d_log2, int group, const int32_t *__restrict__ seq,
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
    constexpr int kStep = 32 * kVec;
    const int lane = threadIdx.x & 31;
    const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
    const int hd = H * d;
    const int64_t groups = (max_cells + group - 1) / group;  // of a list
    const TS *K = static_cast<const TS *>(kv.K), *V = static_cast<const TS *>(kv.V);
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < n_list * groups; w += warps) {
        const int64_t i = div_pos(w, groups), j0 = (w - i * groups) * group;
        // (the list's entry is loaded beside its length, not behind it)
        const int64_t s = seq ? (int64_t)seq[i] : i;
        int64_t p = -1;
        if (lane < group && j0 + lane < max_cells) p = pos ? (int64_t)pos[i * max_cells + j0 + lane] : j0 + lane;
        const int32_t len = s >= 0 && s < n_seq ? kv_len[s] : 0;
        const int64_t many = min((int64_t)n_cells[i], max_cells);
        const int n = (int)min((int64_t)group, many - j0);
        if (n <= 0) continue;
        int32_t mine = -1;  // pool row of cell j0 + lane
        if (lane < n && p >= 0 && p < (int64_t)len) mine = (int32_t)cell_row(kv, (int)s, 0, (int)p);
        // a step: kStep values of a cell's K or V row
        const int per = (hd + kStep - 1) / kStep, steps = n * 2 * per;
        int cell = 0, part = 0;  // of the next step to load
        for (int s0 = 0; s0 < steps; s0 += 4) {
            Raw<TS, kVec> raw[4];
            float mul[4];
            TD *to[4];  // NULL: nothing of this lane's
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int32_t row = __shfl_sync(0xffffffffu, mine, cell);
                const bool is_v = part >= per;
                const int e = (is_v ? part - per : part) * kStep + kVec * lane;
                to[u] = nullptr;
                mul[u] = 0.0f;  // a cell that is not there: zeros
                raw[u].clear();
                if (s0 + u < steps && e < hd) {
                    to[u] = (is_v ? V_out : K_out) + (i * max_cells + j0 + cell) * hd + e;
                    if (row >= 0) {
                        raw[u].load((is_v ? V + row * kv.ld_v : K + row * kv.ld_k) + e);
                        if constexpr (sizeof(TS) == 1) {
                            const int h = d_log2 >= 0 ? e >> d_log2 : e / d;
                            mul[u] = two_to(min(max((int)(is_v ? kv.V_exp : kv.K_exp)[(int64_t)row * H + h] -
                                                        kExpBias, kExpMin), kExpMax));
                        }
                    }
                }
                if (++part == 2 * per) {
                    part = 0;
                    cell = cell + 1 < n ? cell + 1 : cell;
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (!to[u]) continue;
#pragma unroll
                for (int k = 0; k < kVec / 8; ++k) {
                    float x[8];
                    raw[u].eight(k, mul[u], x);
                    store8(to[u] + 8 * k, x);
                }
            }
        }
    }
}

// Rows a warp looks up together: of one to eight, so that 32 warps per SM have the same number of turns
// (prompts of 26,900 tokens, 4 heads, e4m3: six in one turn 21.8 us, four in one or two 22.9).
int rows_group(int64_t rows)
{
    const int64_t warps = (int64_t)device_sm_count() * 32;
    const int64_t turns = (rows + 8 * warps - 1) / (8 * warps);
    const int64_t group = turns ? (rows + turns * warps - 1) / (turns * warps) : 1;
    return group < 1 ? 1 : (int)group;
}

template <typename TS>
cudaError_t write_to(const void *k, const void *v, int64_t ld_k, int64_t ld_v, int d, const SeqView &sv,
                     const KvView &kv, qsa_dtype cache_dtype, cudaStream_t st)
{
    int lanes_log2 = 0;
    while ((8 << lanes_log2) < d) ++lanes_log2;
    const int group = rows_group(sv.n_tok);
    int64_t grid = ((sv.n_tok + group - 1) / group + 3) / 4;
    const int64_t most = (int64_t)device_sm_count() * 16;
    if (grid > most) grid = most;
    const TS *ks = static_cast<const TS *>(k), *vs = static_cast<const TS *>(v);
    uint8_t *ke = const_cast<uint8_t *>(kv.K_exp), *ve = const_cast<uint8_t *>(kv.V_exp);
    void *K = const_cast<void *>(kv.K), *V = const_cast<void *>(kv.V);
    const dim3 g((unsigned)grid), b(128);
    switch (cache_dtype) {
        case QSA_E4M3:
            return launch(paged_write_kernel<TS, uint8_t>, g, b, 0, st, 1, ks, vs, ld_k, ld_v, kv.H_kv, d,
                          lanes_log2, group, sv, kv, static_cast<uint8_t *>(K), static_cast<uint8_t *>(V), ke, ve);
        case QSA_BF16:
            return launch(paged_write_kernel<TS, __nv_bfloat16>, g, b, 0, st, 1, ks, vs, ld_k, ld_v,
                          kv.H_kv, d, lanes_log2, group, sv, kv, static_cast<__nv_bfloat16 *>(K),
                          static_cast<__nv_bfloat16 *>(V), ke, ve);
        default:
            return launch(paged_write_kernel<TS, float>, g, b, 0, st, 1, ks, vs, ld_k, ld_v, kv.H_kv, d,
                          lanes_log2, group, sv, kv, static_cast<float *>(K), static_cast<float *>(V), ke, ve);
    }
}

template <typename TS, typename TD, int kVec>
cudaError_t read_vec(const KvView &kv, int d, const int32_t *seq, const int32_t *kv_len, int64_t n_seq,
                     const int32_t *pos, const int32_t *n_cells, int64_t n_list, int64_t max_cells,
                     void *K_out, void *V_out, cudaStream_t st)
{
    const int group = rows_group(n_list * max_cells);
    int64_t grid = (n_list * ((max_cells + group - 1) / group) + 3) / 4;
    const int64_t most = (int64_t)device_sm_count() * 16;
    if (grid > most) grid = most;
    int d_log2 = -1;
    for (int i = 3; i <= 8; ++i)
        if (d == 1 << i) d_log2 = i;
    return launch(paged_read_kernel<TS, TD, kVec>, dim3((unsigned)grid), dim3(128), 0, st, 1, kv, kv.H_kv, d,
                  d_log2, group, seq, kv_len, n_seq, pos, n_cells, n_list, max_cells,
                  static_cast<TD *>(K_out), static_cast<TD *>(V_out));
}

template <typename TS, typename TD>
cudaError_t read_to(const KvView &kv, int d, const int32_t *seq, const int32_t *kv_len, int64_t n_seq,
                    const int32_t *pos, const int32_t *n_cells, int64_t n_list, int64_t max_cells,
                    void *K_out, void *V_out, cudaStream_t st)
{
    if constexpr (sizeof(TS) == 1) {
        // sixteen codes of one head, 16-byte aligned
        if (d % 16 == 0 && kv.ld_k % 16 == 0 && kv.ld_v % 16 == 0)
            return read_vec<TS, TD, 16>(kv, d, seq, kv_len, n_seq, pos, n_cells, n_list, max_cells, K_out, V_out, st);
    }
    return read_vec<TS, TD, 8>(kv, d, seq, kv_len, n_seq, pos, n_cells, n_list, max_cells, K_out, V_out, st);
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
