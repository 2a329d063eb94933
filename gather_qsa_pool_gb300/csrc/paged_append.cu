// paged_append.cu -- new tokens appended to a paged cache in one pass: queries and keys rotated by their positions,
// keys and values stored in the cache's type (fp32, bf16, e4m3 codes, e2m1 codes), rotated queries and keys stored
// beside.  Also the plain write (no rotation) into a 4-bit cache.
//
// Mathematics.  Values i and i + rot / 2 of a head, i < rot / 2, turn by the angle p * base^(-2 i / rot) of the
// token's position p:  (a, b) -> (a cos - b sin, b cos + a sin).  The angle is formed as a fraction of a turn in 64
// bits: with f_i = 2^64 base^(-2 i / rot) / (2 pi), a double's 53 bits of it, p * f_i modulo 2^64 is the angle's fraction
// of a turn, and the whole turns drop out exactly, whatever p is.  What f_i lacks (up to 650 units of 2^-64 over bases of
// 1 to 10^12, 274 with base 10,000 and 128 values) makes the angle right to p * 2^-52 radians.  In 64-bit floating
// point the same product and its reduction would be bound by this GPU's few fp64 units.  The nearest quarter
// turn is taken off, and cosine and sine of the rest (at most pi / 4) are sums of two fp32 numbers, from their power
// series: the first terms in both, the rest, below 2^-6, in one; together right to 2^-29 for that angle.
// Keys are rotated with both numbers, and the sum of the products carried in two as well: what is then cut down to
// few bits, a code or a bf16 number, is the exact value's but for 2^-28 of it (and p * 2^-52, which passes that from
// positions of 2^24 on).  Of the 13.7 million key codes of 26,792 bf16 tokens none differs from the exact value's;
// with the rotation in fp32 19 e4m3 and 3 e2m1 codes fell to the other side of a border.  (The fp32 number on the way
// is rounded to odd: its last bit says whether anything was left, so the second rounding goes by the exact value.)
// Queries take the first numbers alone.
// The quantised forms are paged_rw.cu's (8 bits) and e2m1.cuh's (4 bits).
//
// Shape.  A warp takes some heads of a token, eight values a lane and d / 8 lanes a head (a power of two of them).  A
// lane's values are four and their four partners, rot / 2 on, so a rotation needs no other lane; lanes behind the
// rotated values have eight in a row.  The warp's lanes make the token's angles once, two a lane, and hand them round
// through shared memory.  A token's heads go to as many warps as keep the GPU full.
// Loads run ahead of the arithmetic: the first are on their way while the token's sequence and cell are looked up, the
// next while these are turned and stored (registers for five CTAs an SM then, four with fp32 sources, which hold twice
// as much: with six and nothing ahead the same took 105 us, with six and loads ahead 101 us and spills).
// Bound by the bytes with many tokens: 26,792 tokens of 32 query and 4 KV heads of d 128 into e4m3 94 us, 5.6 TB/s.  With
// few by the look-up's dependent loads and the launch: 64 tokens 11 to 13 us.
#include "e2m1.cuh"
#include "paged.cuh"

#include <type_traits>

namespace qsa {
namespace {

constexpr int kWarps = 4;

// Four consecutive values as they lie in memory.
template <typename T>
struct Four;
template <>
struct Four<float> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const float *p)
    {
        const uint4 a = *reinterpret_cast<const uint4 *>(p);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
    __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
};
template <>
struct Four<__nv_bfloat16> {
    uint32_t w[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        const uint2 a = *reinterpret_cast<const uint2 *>(p);
        w[0] = a.x; w[1] = a.y;
    }
    __device__ __forceinline__ float at(int i) const
    {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};
template <typename T>
__device__ __forceinline__ void clear(Four<T> &x)
{
#pragma unroll
    for (int i = 0; i < (int)sizeof(x.w) / 4; ++i) x.w[i] = 0u;
}

__device__ __forceinline__ void store4(float *p, const float2 *x)
{
    *reinterpret_cast<float4 *>(p) = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float2 *x)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0].x, x[0].y), b = __floats2bfloat162_rn(x[1].x, x[1].y);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

__device__ __forceinline__ uint32_t finite_bits(float x)
{
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// A lane's place in a head: values d0 .. d0 + 3 and d1 .. d1 + 3.
struct Place {
    int d0, d1;
    bool pair;  // d1 is rot / 2 behind d0 (else four)
    bool on;    // there are such values
};

// A cell's store: this lane's values x[0], x[1] (at d0) and x[2], x[3] (at d1).  here: this lane writes; the others take
// part in the exchange.  lanes: of a head; chunks: words of shared memory for the warp, one for four values of a step
// (4 bits with groups that lanes share unevenly: rot no multiple of 32).  All lanes of the warp call it.
template <int DT>
__device__ __forceinline__ void store_cell(const KvView &kv, bool is_v, int64_t row, int head, const Place &at, int lanes, int d, bool here,
                                           const float2 (&x)[4], bool uneven, uint32_t *chunks)
{
    const int64_t first = row * (is_v ? kv.ld_v : kv.ld_k) + (int64_t)head * d;
    void *const base = const_cast<void *>(is_v ? kv.V : kv.K);
    if constexpr (DT == QSA_F32 || DT == QSA_BF16) {
        using T = std::conditional_t<DT == QSA_F32, float, __nv_bfloat16>;
        if (here) {
            store4(static_cast<T *>(base) + first + at.d0, x);
            store4(static_cast<T *>(base) + first + at.d1, x + 2);
        }
    } else {
        // the largest finite magnitudes of both fours, of the groups they lie in, of the row
        uint32_t m[2];
        bool fine[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u[4] = {finite_bits(x[2 * h].x), finite_bits(x[2 * h].y), finite_bits(x[2 * h + 1].x), finite_bits(x[2 * h + 1].y)};
            m[h] = max(max(u[0], u[1]), max(u[2], u[3]));
            const float s = (x[2 * h].x - x[2 * h].x) + (x[2 * h].y - x[2 * h].y) + (x[2 * h + 1].x - x[2 * h + 1].x) + (x[2 * h + 1].y - x[2 * h + 1].y);
            fine[h] = s == 0.0f;  // no infinity, no NaN
        }
        if (!at.on) m[0] = m[1] = 0;  // (lanes behind the head's last value)
        uint32_t top = max(m[0], m[1]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            if (o < lanes) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        uint8_t *const exps = const_cast<uint8_t *>(is_v ? kv.V_exp : kv.K_exp);
        if constexpr (DT == QSA_E4M3) {
            // as paged_rw.cu: top = m * 2^e', top <= 448 * 2^e
            const int ex = (int)(top >> 23) - 127;
            const int e = min(max(ex - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0), kExpMin), kExpMax);
            const float inv = two_to(-e);
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float2 y[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    y[i] = mul2(x[2 * h + i], make_float2(inv, inv));
                    if (!fine[h]) {
                        y[i].x = isfinite(x[2 * h + i].x) ? y[i].x : NAN;
                        y[i].y = isfinite(x[2 * h + i].y) ? y[i].y : NAN;
                    }
                }
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(y[0], __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(y[1], __NV_SATFINITE, __NV_E4M3);
                w[h] = __byte_perm(lo, hi, 0x5410);
            }
            if (here) {
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(base) + first + at.d0) = w[0];
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(base) + first + at.d1) = w[1];
                if (at.d0 == 0) exps[row * kv.H_kv + head] = (uint8_t)(e + kExpBias);
            }
        } else {
            // (a value that is no number: larger than any)
#pragma unroll
            for (int h = 0; h < 2; ++h) m[h] = fine[h] ? m[h] : 0x7fffffffu;
            if (!uneven) {
                if (!at.pair) m[0] = m[1] = max(m[0], m[1]);
                m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
                m[1] = max(m[1], __shfl_xor_sync(0xffffffffu, m[1], 1));
                const uint32_t a = __shfl_xor_sync(0xffffffffu, m[0], 2), b = __shfl_xor_sync(0xffffffffu, m[1], 2);
                if (at.pair) {
                    m[0] = max(m[0], a);
                    m[1] = max(m[1], b);
                }
            } else {
                // by way of the step's fours
                uint32_t *const mine = chunks + ((threadIdx.x & 31) / lanes) * (2 * lanes);
                __syncwarp();
                if (at.on) {
                    mine[at.d0 >> 2] = m[0];
                    mine[at.d1 >> 2] = m[1];
                }
                __syncwarp();
                if (at.on) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        m[0] = max(m[0], mine[(at.d0 >> 2 & ~3) + i]);
                        m[1] = max(m[1], mine[(at.d1 >> 2 & ~3) + i]);
                    }
                }
            }
            const int e = row_exponent4(top);
            const float inv = two_to(-e);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool good = m[h] < 0x7f800000u;
                const uint8_t code = good ? group_scale(__uint_as_float(m[h]) * inv) : (uint8_t)0x7f;
                const float s = scale_value(code), r = __frcp_rn(s);
                uint32_t w = 0;
                if (good && code != 0) {
                    const float2 y0 = mul2(x[2 * h], make_float2(inv, inv)), y1 = mul2(x[2 * h + 1], make_float2(inv, inv));
                    w = code_pair(y0.x, y0.y, s, r) | code_pair(y1.x, y1.y, s, r) << 8;
                }
                if (here) {
                    const int dim = h ? at.d1 : at.d0;
                    *reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(base) + ((first + dim) >> 1)) = (uint16_t)w;
                    if (dim % kGroup == 0)
                        const_cast<uint8_t *>(is_v ? kv.V_scale : kv.K_scale)[scale_row(kv, row, head) * (d / kGroup) + dim / kGroup] = code;
                }
            }
            if (here && at.d0 == 0) exps[row * kv.H_kv + head] = (uint8_t)(e + kExpBias);
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

__device__ __forceinline__ float2 neg2(float2 a) { return make_float2(-a.x, -a.y); }

// Of two pairs at once, a (c + cl) + b (s + sl), rounded to fp32 (even), and to odd in `odd`.
__device__ __forceinline__ float2 turned2(float2 a, float2 b, float2 c, float2 s, float2 cl, float2 sl, float2 &odd)
{
    // (no product is fused into a sum unasked: what each rounding leaves is counted)
    const float2 p = mul2(a, c), q = mul2(b, s), h = add2(p, q), z = add2(h, neg2(p));
    const float2 e = add2(add2(p, neg2(add2(h, neg2(z)))), add2(q, neg2(z)));  // p + q = h + e
    const float2 l = add2(add2(e, add2(fma2(a, c, neg2(p)), fma2(b, s, neg2(q)))), fma2(a, cl, mul2(b, sl)));
    const float2 y = add2(h, l), rest = add2(l, neg2(add2(y, neg2(h))));
    float2 even;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float yi = i ? y.y : y.x, ri = i ? rest.y : rest.x, hi = i ? h.y : h.x;
        const uint32_t bits = __float_as_uint(yi);
        // towards the exact value where the last bit is 0 and something is left
        const uint32_t step = ri == 0.0f || (bits & 1u) ? 0u : ((__float_as_uint(ri) ^ bits) >> 31 ? 0xffffffffu : 1u);
        const bool fine = isfinite(yi);  // (an infinity times a rest is none)
        (i ? even.y : even.x) = fine ? yi : hi;
        (i ? odd.y : odd.x) = fine ? __uint_as_float(bits + step) : hi;
    }
    return even;
}

// A unit: the heads of a step (32 lanes) of q, or of both k and v.
template <typename TS, int DT>
__global__ void __launch_bounds__(32 * kWarps, sizeof(TS) == 4 ? 4 : 5)
paged_append_kernel(const AppendArgs a, const __grid_constant__ Turns turns, const SeqView sv, const KvView kv)
{
    __shared__ float2 cs_s[kWarps][4][64];  // of each pair of angles: cosines, sines, and what they leave
    __shared__ uint32_t chunk_s[kWarps][64];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = 1 << a.lanes_log2, heads = 32 >> a.lanes_log2;  // of a step
    const int c = lane & (lanes - 1), head = lane >> a.lanes_log2;
    const int d = a.d, H = kv.H_kv;
    Place at;
    at.pair = 8 * c < a.rot;
    at.on = 8 * c < d;
    at.d0 = at.pair ? 4 * c : 8 * c;
    at.d1 = at.pair ? a.rot / 2 + 4 * c : 8 * c + 4;
    const bool on = at.on, uneven = a.rot % 32 != 0;
    const int q_units = a.q ? (a.H_q + heads - 1) / heads : 0, units = q_units + (H + heads - 1) / heads;
    const int per_tok = (units + a.per_warp - 1) / a.per_warp;
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t tok = div_pos(w, per_tok);
    if (tok >= sv.n_tok) return;
    const int u0 = (int)(w - tok * per_tok) * a.per_warp, u1 = min(units, u0 + a.per_warp);
    // ---- what is loaded first is on its way while the token is looked up and its angles are made: four units of queries,
    // one of keys and values; then always the next ones ahead
    const TS *const q = static_cast<const TS *>(a.q), *const k = static_cast<const TS *>(a.k), *const v = static_cast<const TS *>(a.v);
    TS *const q_out = static_cast<TS *>(a.q_out), *const k_out = static_cast<TS *>(a.k_out);
    // (a lane's units of each end behind the last head, or at once)
    const int step = heads * d, d10 = at.d1 - at.d0, heads_log2 = 5 - a.lanes_log2;
    const int end_q = on ? min(u1, (a.H_q - head + heads - 1) >> heads_log2) : 0;
    const int end_kv = on ? min(u1, q_units + ((H - head + heads - 1) >> heads_log2)) : 0;
    const TS *const q0 = q + tok * a.ld_q + head * d + at.d0;
    TS *const q1 = q_out + tok * a.H_q * d + head * d + at.d0;
    const TS *const k0 = k + tok * a.ld_k + head * d + at.d0, *const v0 = v + tok * a.ld_v + head * d + at.d0;
    Four<TS> xq[4][2], xkv[2][2];
    auto load_q = [&](int u) {
        const TS *from = q0 + (int64_t)u * step;
#pragma unroll
        for (int j = 0; j < 4; ++j, from += step)
            if (u + j < end_q) {
                xq[j][0].load(from);
                xq[j][1].load(from + d10);
            }
    };
    auto load_kv = [&](int u) {
        if (u < end_kv) {
            const int64_t off = (int64_t)(u - q_units) * step;
            xkv[0][0].load(k0 + off);
            xkv[0][1].load(k0 + off + d10);
            xkv[1][0].load(v0 + off);
            xkv[1][1].load(v0 + off + d10);
        }
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        clear(xq[j][0]);
        clear(xq[j][1]);
        clear(xkv[j & 1][j >> 1]);
    }
    load_q(u0);
    load_kv(max(u0, q_units));
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
    if (s >= sv.n_seq || (int64_t)sv.cu[s] > tok) return;  // of no sequence: nothing is written
    const int64_t len = sv.kv_len[s], place = len - ((int64_t)sv.cu[s + 1] - tok);
    const int64_t row = u1 > q_units && place >= 0 && place < len ? cell_row(kv, s, 0, (int)place) : -1;
    // ---- its angles: this lane's four, as two pairs
    float2 (*const cs)[64] = cs_s[warp];
    float2 co[2] = {make_float2(1.0f, 1.0f), make_float2(1.0f, 1.0f)}, si[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
    if (a.rot > 0) {
        const int64_t p = a.pos ? (int64_t)a.pos[tok] : place;
        // (a plain load: lanes that read different places of the constant bank take turns)
        const uint64_t *freq = turns.f;
        asm volatile("" : "+l"(freq));
        for (int i = lane; i < a.rot / 2; i += 32) {
            float2 c2, s2;
            turn_of((uint64_t)p * freq[i], c2, s2);
            reinterpret_cast<float *>(cs[0])[i] = c2.x;
            reinterpret_cast<float *>(cs[1])[i] = s2.x;
            reinterpret_cast<float *>(cs[2])[i] = c2.y;
            reinterpret_cast<float *>(cs[3])[i] = s2.y;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (at.pair) {
                co[i] = cs[0][2 * c + i];
                si[i] = cs[1][2 * c + i];
            }
    }
    auto values = [&](const Four<TS> &x, float2 *y) {
        y[0] = make_float2(x.at(0), x.at(1));
        y[1] = make_float2(x.at(2), x.at(3));
    };
    // ---- queries
    for (int u = u0; u < u1 && u < q_units; u += 4) {
        Four<TS> x[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[j][0] = xq[j][0];
            x[j][1] = xq[j][1];
        }
        load_q(u + 4);
        TS *to = q1 + (int64_t)u * step;
#pragma unroll
        for (int j = 0; j < 4; ++j, to += step) {
            float2 lo[2], hi[2];
            values(x[j][0], lo);
            values(x[j][1], hi);
            if (at.pair) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 y = fma2(lo[i], co[i], neg2(mul2(hi[i], si[i])));
                    hi[i] = fma2(hi[i], co[i], mul2(lo[i], si[i]));
                    lo[i] = y;
                }
            }
            if (u + j < end_q) {
                store4(to, lo);
                store4(to + d10, hi);
            }
        }
    }
    // ---- keys and values
    for (int u = max(u0, q_units); u < u1; ++u) {
        const int h = (u - q_units) * heads + head;
        const bool mine = u < end_kv;
        Four<TS> x[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i][0] = xkv[i][0];
            x[i][1] = xkv[i][1];
        }
        load_kv(u + 1);
        float2 y[4], z[4];
        values(x[0][0], y);
        values(x[0][1], y + 2);
        values(x[1][0], z);
        values(x[1][1], z + 2);
        float2 even[4] = {y[0], y[1], y[2], y[3]};
        if (at.pair) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 cl = cs[2][2 * c + i], sl = cs[3][2 * c + i], lo = y[i], hi = y[2 + i];
                even[i] = turned2(lo, hi, co[i], neg2(si[i]), cl, neg2(sl), y[i]);
                even[2 + i] = turned2(hi, lo, co[i], si[i], cl, sl, y[2 + i]);
            }
        }
        // (fp32 results are the nearest; what is rounded again goes on from the odd ones)
        if (k_out && mine) {
            TS *const to = k_out + (tok * H + h) * d;
            store4(to + at.d0, sizeof(TS) == 4 ? even : y);
            store4(to + at.d1, sizeof(TS) == 4 ? even + 2 : y + 2);
        }
        store_cell<DT>(kv, false, row, h, at, lanes, d, mine && row >= 0, DT == QSA_F32 ? even : y, uneven, chunk_s[warp]);
        store_cell<DT>(kv, true, row, h, at, lanes, d, mine && row >= 0, z, uneven, chunk_s[warp]);
    }
}

// f_i to about 2^-51 of itself: the exponent i * (2 / rot) log2(base) in two parts, the first exact.
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
