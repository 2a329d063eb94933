// paged_append.cu -- new tokens appended to a paged cache in one pass: queries and keys rotated by their positions,
// keys and values stored in the cache's type (fp32, bf16, e4m3 codes, e2m1 codes), rotated queries and keys stored
// beside.  Also the plain write (no rotation) into a 4-bit cache.
//
// Mathematics.  Values i and i + rot / 2 of a head, i < rot / 2, turn by the angle p * base^(-2 i / rot) of the
// token's position p:  (a, b) -> (a cos - b sin, b cos + a sin).  The angle is formed as a fraction of a turn in 64
// bits: with f_i = 2^64 base^(-2 i / rot) / (2 pi), rounded, p * f_i modulo 2^64 is the angle's fraction of a turn
// with an error of p / 2 units of 2^-64, and the whole turns drop out exactly, whatever p is.  In 64-bit
// floating point the same product and its reduction would be bound by this GPU's few fp64 units.  The nearest quarter
// turn is taken off, and cosine and sine of the rest (at most pi / 4) are sums of two fp32 numbers, from their power
// series: the first terms in both, the rest, below 2^-6, in one; together right to 2^-29.
// Keys are rotated with both numbers, and the sum of the products carried in two as well: what is then cut down to
// few bits, a code or a bf16 number, is the exact value's but for 2^-28 of it, where an fp32 result would fall to the
// other side of a border fifty times as often.  (The fp32 number on the way is rounded to odd: its last bit says
// whether anything was left, so the second rounding goes by the exact value.)  Queries take the first numbers alone.
// The quantised forms are paged_rw.cu's (8 bits) and e2m1.cuh's (4 bits).
//
// Shape.  A warp takes some heads of a token, eight values a lane and d / 8 lanes a head (a power of two of them);
// the other value of a pair lies in the lane rot / 16 away.  The warp's lanes make the token's angles once, two a
// lane, and hand them round through shared memory.  A token's heads go to as many warps as keep the GPU full.
// Bound by the bytes with many tokens, by the look-up's dependent loads and the launch with few.
#include "e2m1.cuh"
#include "paged.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;

template <typename T>
struct Eight;
template <>
struct Eight<float> {
    uint32_t w[8];
    __device__ __forceinline__ void load(const float *p)
    {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
};
template <>
struct Eight<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
    __device__ __forceinline__ float at(int i) const
    {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

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

__device__ __forceinline__ uint32_t finite_bits(float x)
{
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// A cell's place for one lane's eight values, and their store.  DT: 0 fp32, 1 bf16, 2 e4m3, 3 e2m1 (qsa_dtype).
// here: this lane writes; the others take part in the shuffles.  lanes: of a head.  All lanes of the warp call it.
template <int DT>
__device__ __forceinline__ void store_cell(const KvView &kv, bool is_v, int64_t row, int head, int c, int lanes, int d,
                                           bool here, const float (&x)[8])
{
    const int64_t at = row * (is_v ? kv.ld_v : kv.ld_k) + (int64_t)head * d + 8 * c;
    void *const base = const_cast<void *>(is_v ? kv.V : kv.K);
    if constexpr (DT == QSA_F32) {
        if (here) store8(static_cast<float *>(base) + at, x);
    } else if constexpr (DT == QSA_BF16) {
        if (here) store8(static_cast<__nv_bfloat16 *>(base) + at, x);
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, finite_bits(x[i]));
        if (!here) top = 0;  // (lanes behind the head's last value)
        uint32_t pair = top;  // e2m1: of this lane's group of sixteen
        if constexpr (DT == QSA_E2M1) {
            pair = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = pair;
        }
#pragma unroll
        for (int o = DT == QSA_E2M1 ? 2 : 1; o < 32; o <<= 1)
            if (o < lanes) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        bool all = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = all && isfinite(x[i]);
        uint8_t *const exps = const_cast<uint8_t *>(is_v ? kv.V_exp : kv.K_exp);
        if constexpr (DT == QSA_E4M3) {
            // as paged_rw.cu: top = m * 2^e', top <= 448 * 2^e
            const int ex = (int)(top >> 23) - 127;
            const int e = min(max(ex - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), kExpMin), kExpMax);
            const float inv = two_to(-e);
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = all || isfinite(x[4 * i + j]) ? x[4 * i + j] * inv : NAN;
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
                w[i] = __byte_perm(lo, hi, 0x5410);
            }
            if (here) {
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(base) + at) = make_uint2(w[0], w[1]);
                if (c == 0) exps[row * kv.H_kv + head] = (uint8_t)(e + kExpBias);
            }
        } else {
            const int e = row_exponent4(top);
            const float inv = two_to(-e);
            const bool fine = __shfl_xor_sync(0xffffffffu, (int)all, 1) && all;
            const uint8_t code = fine ? group_scale(__uint_as_float(pair) * inv) : (uint8_t)0x7f;
            const float s = scale_value(code);
            const float r = __frcp_rn(s);
            uint32_t w = 0;
            if (fine && code != 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w |= code_pair(x[2 * i] * inv, x[2 * i + 1] * inv, s, r) << (8 * i);
            }
            if (here) {
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(base) + (at >> 1)) = w;
                if (c == 0) exps[row * kv.H_kv + head] = (uint8_t)(e + kExpBias);
                if (!(c & 1))
                    const_cast<uint8_t *>(is_v ? kv.V_scale : kv.K_scale)[scale_row(kv, row, head) * (d / kGroup) + (c >> 1)] = code;
            }
        }
    }
}

// 2^64 times the turns of one position, for each pair of values.
struct Turns {
    uint64_t f[128];
};

struct AppendArgs {
    const void *q, *k, *v;
    void *q_out, *k_out;
    int64_t ld_q, ld_k, ld_v;
    const int32_t *pos;  // NULL: a token's place in its sequence
    int32_t H_q, d, rot;
    int32_t lanes_log2;  // of a head
    int32_t per_warp;    // units of a warp
};

// Cosine and sine of a fraction of a turn (in 2^-64), each as the sum of two numbers: c.x + c.y, s.x + s.y.
__device__ __forceinline__ void turn_of(uint64_t frac, float2 &c, float2 &s)
{
    const uint32_t quarter = (uint32_t)((frac + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(frac - ((uint64_t)quarter << 62));  // of [-2^61, 2^61)
    const float rh = (float)rest, rl = (float)(rest - (int64_t)rh);
    constexpr double kStep = 6.283185307179586 / 18446744073709551616.0;  // radians
    constexpr float ph = (float)kStep, pl = (float)(kStep - (double)ph);
    const float xh = __fmul_rn(rh, ph), xl = fmaf(rh, ph, -xh) + fmaf(rh, pl, rl * ph);  // |x| <= pi / 4
    const float th = __fmul_rn(xh, xh), tl = fmaf(xh, xh, -th) + 2.0f * xh * xl;          // x^2
    // cos x = 1 - x^2 / 2 + x^4 (1 / 24 - ...)
    const float uh = fmaf(th, -0.5f, 1.0f);
    const float t2 = fmaf(th, th, 2.0f * th * tl);
    float u = t2 * fmaf(th, fmaf(th, fmaf(th, -1.0f / 3628800.0f, 1.0f / 40320.0f), -1.0f / 720.0f), 1.0f / 24.0f);
    u += fmaf(th, -0.5f, 1.0f - uh) - 0.5f * tl;
    float2 co = make_float2(uh + u, 0.0f);
    co.y = u - (co.x - uh);
    // sin x = x (1 - x^2 / 6 + x^4 (1 / 120 - ...))
    constexpr float k6h = (float)(1.0 / 6.0), k6l = (float)(1.0 / 6.0 - (double)k6h);
    const float mh = __fmul_rn(th, k6h), ml = fmaf(th, k6h, -mh) + fmaf(th, k6l, tl * k6h), vh = __fsub_rn(1.0f, mh);
    const float v = ((1.0f - vh) - mh) - ml +
                    t2 * fmaf(th, fmaf(th, fmaf(th, -1.0f / 39916800.0f, 1.0f / 362880.0f), -1.0f / 5040.0f), 1.0f / 120.0f);
    const float sh = __fmul_rn(xh, vh), sl = fmaf(xh, vh, -sh) + fmaf(xh, v, xl * vh);
    float2 si = make_float2(sh + sl, 0.0f);
    si.y = sl - (si.x - sh);
    const bool swap = quarter & 1;
    c = swap ? si : co;
    s = swap ? co : si;
    if (quarter == 1 || quarter == 2) c = make_float2(-c.x, -c.y);
    if (quarter >= 2) s = make_float2(-s.x, -s.y);
}

// a (c.x + c.y) + b (s.x + s.y), rounded to fp32 (even), and to odd in `odd`.
__device__ __forceinline__ float turned(float a, float b, float2 c, float2 s, float &odd)
{
    // (no product is fused into a sum unasked: what each rounding leaves is counted)
    const float p = __fmul_rn(a, c.x), q = __fmul_rn(b, s.x), h = __fadd_rn(p, q), z = __fsub_rn(h, p);
    const float e = (p - (h - z)) + (q - z);  // p + q = h + e
    const float l = e + (fmaf(a, c.x, -p) + fmaf(b, s.x, -q)) + fmaf(a, c.y, b * s.y);
    const float y = h + l, rest = l - (y - h);
    odd = y;
    if (!isfinite(y)) return odd = h;  // (an infinity times a rest is none)
    const uint32_t bits = __float_as_uint(y);
    if (rest != 0.0f && !(bits & 1u)) odd = __uint_as_float((rest > 0.0f) == (y > 0.0f) ? bits + 1u : bits - 1u);
    return y;
}

// A unit: the heads of a step (32 lanes) of q, or of both k and v.
template <typename TS, int DT>
__global__ void __launch_bounds__(32 * kWarps, 6)
paged_append_kernel(const AppendArgs a, const __grid_constant__ Turns turns, const SeqView sv, const KvView kv)
{
    __shared__ float4 cs_s[kWarps][128];  // cosine, sine, and what they leave
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = 1 << a.lanes_log2, heads = 32 >> a.lanes_log2;  // of a step
    const int c = lane & (lanes - 1), head = lane >> a.lanes_log2;
    const int d = a.d, H = kv.H_kv;
    const bool on = 8 * c < d;
    const int q_units = a.q ? (a.H_q + heads - 1) / heads : 0, units = q_units + (H + heads - 1) / heads;
    const int per_tok = (units + a.per_warp - 1) / a.per_warp;
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t tok = div_pos(w, per_tok);
    if (tok >= sv.n_tok) return;
    const int u0 = (int)(w - tok * per_tok) * a.per_warp, u1 = min(units, u0 + a.per_warp);
    // ---- the token's sequence, position and cell
    int s = 0;
    for (;; s += 32) {
        const bool behind = s + lane < sv.n_seq && (int64_t)sv.cu[s + lane + 1] <= tok;
        const int n = __popc(__ballot_sync(0xffffffffu, behind));
        if (n < 32) {
            s += n;
            break;
        }
    }
    if (s >= sv.n_seq || (int64_t)sv.cu[s] > tok) return;  // of no sequence: nothing is read or written
    const int64_t len = sv.kv_len[s], place = len - ((int64_t)sv.cu[s + 1] - tok);
    const int64_t row = u1 > q_units && place >= 0 && place < len ? cell_row(kv, s, 0, (int)place) : -1;
    // ---- its angles: this lane's eight, as its values need them
    const int hr = a.rot >> 4;  // lanes of half the rotated values
    const bool turn = c < 2 * hr;
    const int other = c < hr ? lane + hr : (turn ? lane - hr : lane);
    const int first = turn ? 8 * (c < hr ? c : c - hr) : 0;  // of its angles
    float4 *const cs = cs_s[warp];
    float co[8], si[8];
    if (hr > 0) {
        const int64_t p = a.pos ? (int64_t)a.pos[tok] : place;
        for (int i = lane; i < 8 * hr; i += 32) {
            float2 c2, s2;
            turn_of((uint64_t)p * turns.f[i], c2, s2);
            cs[i] = make_float4(c2.x, s2.x, c2.y, s2.y);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 t = cs[first + i];
            co[i] = t.x;
            si[i] = c < hr ? -t.y : t.y;
        }
    }
    auto rotated = [&](const Eight<TS> &x, float (&y)[8]) {
        Eight<TS> p;
        constexpr int kWords = sizeof(x.w) / 4;
#pragma unroll
        for (int i = 0; i < kWords; ++i) p.w[i] = __shfl_sync(0xffffffffu, x.w[i], other);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = turn ? fmaf(x.at(i), co[i], p.at(i) * si[i]) : x.at(i);
    };
    // ---- queries, four units in flight
    const TS *const q = static_cast<const TS *>(a.q), *const k = static_cast<const TS *>(a.k), *const v = static_cast<const TS *>(a.v);
    TS *const q_out = static_cast<TS *>(a.q_out), *const k_out = static_cast<TS *>(a.k_out);
    for (int u = u0; u < u1 && u < q_units; u += 4) {
        Eight<TS> x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = (u + j) * heads + head;
            if (on && h < a.H_q && u + j < u1) {
                x[j].load(q + tok * a.ld_q + (int64_t)h * d + 8 * c);
            } else {
#pragma unroll
                for (int i = 0; i < (int)sizeof(x[j].w) / 4; ++i) x[j].w[i] = 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int h = (u + j) * heads + head;
            float y[8];
            rotated(x[j], y);
            if (on && h < a.H_q && u + j < u1) store8(q_out + (tok * a.H_q + h) * d + 8 * c, y);
        }
    }
    // ---- keys and values
    for (int u = max(u0, q_units); u < u1; ++u) {
        const int h = (u - q_units) * heads + head;
        const bool mine = on && h < H;
        Eight<TS> x[2];
        if (mine) {
            x[0].load(k + tok * a.ld_k + (int64_t)h * d + 8 * c);
            x[1].load(v + tok * a.ld_v + (int64_t)h * d + 8 * c);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(x[0].w) / 4; ++i) x[0].w[i] = x[1].w[i] = 0u;
        }
        float y[8], z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = x[0].at(i);
            z[i] = x[1].at(i);
        }
        if (hr > 0) {
            Eight<TS> pw;
#pragma unroll
            for (int i = 0; i < (int)sizeof(x[0].w) / 4; ++i) pw.w[i] = __shfl_sync(0xffffffffu, x[0].w[i], other);
            float even[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 t = cs[first + i];
                even[i] = y[i];
                if (turn)
                    even[i] = turned(y[i], pw.at(i), make_float2(t.x, t.z), c < hr ? make_float2(-t.y, -t.w) : make_float2(t.y, t.w), y[i]);
            }
            // (fp32 results are the nearest; what is rounded again goes on from the odd ones)
            if (k_out && mine) store8(k_out + (tok * H + h) * d + 8 * c, sizeof(TS) == 4 ? even : y);
            if constexpr (DT == QSA_F32) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = even[i];
            }
        } else if (k_out && mine) {
            store8(k_out + (tok * H + h) * d + 8 * c, y);
        }
        store_cell<DT>(kv, false, row, h, c, lanes, d, mine && row >= 0, y);
        store_cell<DT>(kv, true, row, h, c, lanes, d, mine && row >= 0, z);
    }
}

// f_i to about 2^-52 of itself: the exponent i * (2 / rot) log2(base) in two parts, the first exact.
void fill_turns(Turns &t, double base, int rot)
{
    if (rot == 0) return;
    const long double step = log2l((long double)base) * 2.0L / rot;
    const double hi = (double)(float)step, lo = (double)(step - (long double)hi);
    for (int i = 0; i < rot / 2; ++i) {
        const double z = -(i * lo) * 0.6931471805599453;
        // 2^64 / (2 pi), at most: base >= 1
        t.f[i] = (uint64_t)(exp2(-(i * hi)) * (1.0 + z + 0.5 * z * z) * 2935890503282001226.0);
    }
}

template <typename TS>
cudaError_t append_to(AppendArgs &a, const Turns &t, const SeqView &sv, const KvView &kv, qsa_dtype dt, cudaStream_t st)
{
    const int heads = 32 >> a.lanes_log2;
    const int units = (a.q ? (a.H_q + heads - 1) / heads : 0) + (kv.H_kv + heads - 1) / heads;
    // a warp takes one unit while there are few, else whole tokens (a token's angles are made once a warp)
    const int64_t warps = (int64_t)device_sm_count() * 32;
    const int64_t per = (sv.n_tok * units + warps - 1) / warps;
    a.per_warp = (int)(per < 1 ? 1 : (per < units ? per : units));
    const int64_t n = sv.n_tok * ((units + a.per_warp - 1) / a.per_warp);
    const dim3 grid((unsigned)((n + kWarps - 1) / kWarps)), block(32 * kWarps);
    switch (dt) {
        case QSA_E2M1: return launch(paged_append_kernel<TS, QSA_E2M1>, grid, block, 0, st, 1, a, t, sv, kv);
        case QSA_E4M3: return launch(paged_append_kernel<TS, QSA_E4M3>, grid, block, 0, st, 1, a, t, sv, kv);
        case QSA_BF16: return launch(paged_append_kernel<TS, QSA_BF16>, grid, block, 0, st, 1, a, t, sv, kv);
        default: return launch(paged_append_kernel<TS, QSA_F32>, grid, block, 0, st, 1, a, t, sv, kv);
    }
}

}  // namespace

cudaError_t launch_paged_append(const void *q, const void *k, const void *v, qsa_dtype src_dtype, int64_t ld_q,
                                int64_t ld_k, int64_t ld_v, int H_q, int d, int rot, double base, const int32_t *pos,
                                void *q_out, void *k_out, const SeqView &sv, const KvView &kv, qsa_dtype cache_dtype,
                                cudaStream_t st)
{
    AppendArgs a = {q, k, v, q_out, k_out, ld_q, ld_k, ld_v, pos, H_q, d, rot, 0, 1};
    while ((8 << a.lanes_log2) < d) ++a.lanes_log2;
    Turns t;
    fill_turns(t, base, rot);
    return src_dtype == QSA_BF16 ? append_to<__nv_bfloat16>(a, t, sv, kv, cache_dtype, st)
                                 : append_to<float>(a, t, sv, kv, cache_dtype, st);
}

}  // namespace qsa
