// few_cells.cuh -- attention of a few query rows over cells of a paged cache, any row type, d 128: the kernel that
// the 4-bit cache's attention of a few tokens (paged_four.cu) and the sparse attention over listed blocks
// (paged_sparse.cu) share.  Only those two include this header.
//
// Mathematics: as dense_decode.cu, a part of a row's cells gives (m, l, o) = (reference, sum 2^(s_j - m),
// sum 2^(s_j - m) v_j), m moves only when a logit passes it by more than the room left, and parts join by scaling
// to a common m.  Rows of codes: v_j = c_j 2^e_j with c_j exact in fp16 (4 bits: the code times its scale), so the
// weight that multiplies c_j is 2^(s_j + e_j - m), and the sum adds 2^-e_j times it.
//
// Shape: operands are swapped, so that the cells are the 16 rows of mma.m16n8k16 and eight query rows its columns:
//   S' [cell][row] = K Q'        A = 16 cells x 16 dims, from the cells' rows
//   O' [dim][row] += V' P'       A = 16 dims x 16 cells, from the same cells' values
// NB blocks of eight rows (tokens x heads of a KV head) use a converted A fragment together, and one token's eight
// heads waste nothing: with rows as the 16 rows of A half of each instruction would be empty.  (The tensor cores
// take 0.5 of these instructions a cycle and SM; the conversion of a 4-bit fragment's two registers, two
// conversions and two multiplications, runs beside it.)  Weights pass from the accumulators of S' to the B fragments
// of the second product by a transposing move of 8 x 8 registers halves.
// A warp takes 16 (bf16) or 32 (codes) cells of a tile at a time and has sums and references of its own.  The warps of
// a CTA take one or more KV heads of the same cells (`hpc` heads of a CTA), so that the heads of a row are read
// together: L2 fetches more than a head's 64 bytes of 4-bit codes, and with the heads in different CTAs 306 MB of
// cells took 510 MB of reads.
//   rows of codes and values lie swizzled in shared memory, and the cells of a fragment are numbered, such that
//   both the reads along a cell (keys) and across four cells (values) touch every bank once.
#pragma once

#include "dense_join.cuh"
#include "e2m1.cuh"
#include "mma_frag.cuh"
#include "umma.cuh"

namespace qsa {
namespace few {

constexpr int kD = 128;
constexpr int kPitch = kD + 4;

// C: QSA_BF16, QSA_E4M3 or QSA_E2M1.
template <int C>
struct Cell {
    static constexpr bool kF16 = C != QSA_BF16;            // the products' 16-bit type
    static constexpr int kRowBytes = C == QSA_BF16 ? 256 : (C == QSA_E4M3 ? 128 : 64);
    static constexpr int kKeys = C == QSA_BF16 ? 16 : 32;  // a warp's cells of a tile
    static constexpr int kGroups = kKeys / 16;
    static constexpr int kE = C == QSA_BF16 ? 8 : (C == QSA_E4M3 ? 16 : 32);  // values of 16 bytes
    static constexpr uint32_t kTile = kKeys * kRowBytes;   // bytes of K (and of V) of a stage
    static constexpr uint32_t kScales = C == QSA_E2M1 ? kKeys * 8 : 0;
    static constexpr uint32_t kStage = 2 * kTile + 2 * kScales;  // K, V, K's scales, V's
    // A reference lies kBelow under the maximum where it is set and moves once a logit is kMove above it: fp16
    // weights end at 2^-25 and 2^16
    static constexpr float kBelow = kF16 ? 13.0f : 0.0f, kMove = kF16 ? 15.0f : 8.0f;
};
// Exponents of V beyond this: the sums are taken from exponentials of their own.
constexpr float kFar = 50.0f;

// Bytes of one head's queries as fragments.
template <int NB, int NT>
__host__ __device__ constexpr size_t q_bytes() { return (size_t)NT * NB * 4 * 32 * 16; }

// `bytes` (0, 8, 16) of 16 from global memory, zeros behind.
// (a head's 4-bit row is 64 bytes: L2 fetches no more, as the other heads' bytes would go again unused)
template <int C>
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes)
{
    if constexpr (C == QSA_E2M1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool F16>
__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1)
{
    if constexpr (F16) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        mma_16816(c, a, b0, b1);
    }
}

// Two values as a 16-bit pair (fp16 or bf16), and what the rounding left of each.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float &x, float &y)
{
    uint32_t u;
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        x -= f.x;
        y -= f.y;
        u = *reinterpret_cast<const uint32_t *>(&h);
    } else {
        u = pack_bf16(x, y);
        x -= __uint_as_float(u << 16);
        y -= __uint_as_float(u & 0xffff0000u);
    }
    return u;
}

// The warp's 8 x 8 matrix of 16-bit values (lane 4 r + c: columns 2 c, 2 c + 1 of row r), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Two e4m3 codes (low or high half) as two fp16 values, exact.
template <int kHigh>
__device__ __forceinline__ uint32_t half_of_e4m3(uint32_t codes)
{
    uint32_t r;
    if constexpr (kHigh)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(codes));
    else
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

// Offset of 16-byte chunk c of row r of a tile.
template <int C>
__device__ __forceinline__ uint32_t cell_off(int r, int c)
{
    const int x = C == QSA_E2M1 ? (r >> 1) & 3 : (C == QSA_E4M3 ? (r & 6) ^ ((r & 1) << 2) : ((r & 1) << 2) | ((r >> 1) & 3));
    return (uint32_t)r * Cell<C>::kRowBytes + (uint32_t)((c ^ x) << 4);
}
// The cell that is row f (of eight) of a fragment: 4-bit rows, two to a line of banks, are taken as 0, 3, 1, 2, ...
template <int C>
__device__ __forceinline__ int frag_cell(int f)
{
    return C == QSA_E2M1 ? (f & 4) | ((0x2130 >> (4 * (f & 3))) & 3) : f;
}
constexpr float kUnset = -3.0e38f;  // a reference before the first cell: any finite logit moves it

// The first of the dims (and the step to the second) that rows g8 and g8 + 8 of the fragment of dims number t hold.
template <int C>
__device__ __forceinline__ int frag_dim(int t, int g8, int half)
{
    return C == QSA_BF16 ? 16 * t + 8 * half + g8 : 16 * g8 + 2 * t + half;
}

// ------------------------------------------------------------------ queries
// The queries' fragments of hpc heads to shared memory by W warps (tid: a thread's number among them; all call it),
// k permuted as the key rows are read: lane (g8, c4) holds row g8 of a block, and kE values of each 4 kE.  Row r of a
// head: token r / G, query head r mod G.  from: the first token's values of the first head.  fp16 holds a row's queries
// times a power of two of its own (one for the tile would let a large query of one token or head take the bits of
// another's); undo: scale over that, what makes the row's products logits, 8 NB rows a head.  The caller's barrier follows.
template <int C, typename TQ, int NB, int NT, int W>
__device__ __forceinline__ void stage_queries(int tid, const TQ *from, int64_t ld_q, int G, int rows, int hpc, float q_sign, float scale,
                                              uint4 *q_all, float *undo)
{
    constexpr bool F16 = Cell<C>::kF16;
    constexpr int E = Cell<C>::kE, kWords = sizeof(TQ) == 2 ? 16 : 32;
    const int warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, c4 = lane & 3;
    // unit u: block u mod NB of head u / NB; warp w takes units w, w + W, ...
    constexpr int kMost = NB * 4 <= W ? 1 : NB * 4 / W;  // of a warp, with up to four heads
    const int units = hpc * NB;
    uint32_t raw[kMost][kWords];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int u = warp + W * i, r = 8 * (u % NB) + g8;
        const int tk = r < G ? 0 : (int)((uint32_t)r / (uint32_t)G);
        const uint4 *const src = reinterpret_cast<const uint4 *>(from + tk * ld_q + (int64_t)((u / NB) * G + r - tk * G) * kD + c4 * E);
        constexpr int kStep = 4 * E * (int)sizeof(TQ) / 16, kOf = E * (int)sizeof(TQ) / 16;  // of 16 bytes
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k) {
            uint4 y = make_uint4(0u, 0u, 0u, 0u);
            if (u < units && r < rows) y = src[(k / kOf) * kStep + k % kOf];
            raw[i][4 * k] = y.x;
            raw[i][4 * k + 1] = y.y;
            raw[i][4 * k + 2] = y.z;
            raw[i][4 * k + 3] = y.w;
        }
    }
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        const int u = warp + W * i;
        if (u >= units) break;
        float mul = q_sign;
        if constexpr (F16) {
            // the row's largest finite magnitude, by its bits, becomes at least 2^7 and less than 2^8
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                const uint32_t a = (sizeof(TQ) == 2 ? raw[i][k] << 16 : raw[i][k]) & 0x7fffffffu;
                const uint32_t b = sizeof(TQ) == 2 ? raw[i][k] & 0x7fff0000u : 0u;
                top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int sh = top > 0u ? min(max(134 - (int)(top >> 23), -120), 100) : 0;
            mul = q_sign * two_to(sh);
            if (c4 == 0) undo[8 * u + g8] = scale * two_to(-sh);
        }
        uint4 *const to = q_all + (u / NB) * (int)(q_bytes<NB, NT>() / 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // two steps of 16 dims
            float xa[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t w = sizeof(TQ) == 2 ? raw[i][(4 * k + e / 2) % kWords] : raw[i][(8 * k + e) % kWords];
                xa[e] = __uint_as_float(sizeof(TQ) == 4 ? w : (e & 1 ? w & 0xffff0000u : w << 16)) * mul;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint4 f;
                f.x = pack16<F16>(xa[0], xa[1]);
                f.y = pack16<F16>(xa[2], xa[3]);
                f.z = pack16<F16>(xa[4], xa[5]);
                f.w = pack16<F16>(xa[6], xa[7]);
                to[((n * NB + u % NB) * 4 + k) * 32 + lane] = f;
            }
        }
    }
}

// ------------------------------------------------------------------ a warp's rows over its cells
// NB: blocks of eight rows.  NT: 16-bit terms of a query and a weight.  Rows 8 n + 2 c4 + e (e = 0, 1) are lane
// (g8, c4)'s, with the dims frag_dim(t, g8, 0 and 1) of each.
template <int C, int NB, int NT>
struct Rows {
    using S = Cell<C>;
    static constexpr bool F16 = S::kF16;
    static constexpr int kGroups = S::kGroups;
    // mx: the rows' reference; l: the sums in its units.  Exponents far apart (wide): l in units of ms, a reference of
    // the logits alone.
    float o[8][NB][4], ms[NB][2], mx[NB][2], l[NB][2];
    bool wide;

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][n][e] = 0.0f;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ms[n][e] = mx[n][e] = kUnset;
                l[n][e] = 0.0f;
            }
        wide = false;
    }

    // The cells of one stage: sk: K, V (codes' scales behind them); ex: per cell 2^ke, the exponent e of the value,
    // 2^-e (codes only); far: some e is beyond kFar; qf: the queries' fragments, undo: what makes their products
    // logits (codes; bf16: key_scale); edge: hide(c, n, e) says whether row (n, e) does not see cell c.
    template <typename Hide>
    __device__ __forceinline__ void tile(const unsigned char *sk, const float4 *ex, const uint4 *qf, const float *undo, float key_scale,
                                         bool far, bool edge, Hide hide)
    {
        const unsigned char *const sv = sk + S::kTile, *const ks = sv + S::kTile, *const vs = ks + S::kScales;
        const int lane = threadIdx.x & 31, g8 = lane >> 2, c4 = lane & 3;
        // where this thread's parts of a fragment lie: key rows f0 (+ 8, + 16 kg), values of cells va, vb (likewise)
        const int f0 = frag_cell<C>(g8), va = frag_cell<C>(2 * c4), vb = frag_cell<C>(2 * c4 + 1);
        const uint32_t at_k = cell_off<C>(f0, c4);
        // ---- logits: fragments of 16 cells x 8 rows
        float s[kGroups][NB][4];
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[kg][n][e] = 0.0f;
        if constexpr (C == QSA_E2M1) {
            uint4 kr[kGroups][2];
            __half2 sc[kGroups][2];  // scales of the lane's two groups of a cell
#pragma unroll
            for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    kr[kg][hf] = *reinterpret_cast<const uint4 *>(sk + at_k + (16 * kg + 8 * hf) * S::kRowBytes);
                    const uint32_t h = half_of_scales(*reinterpret_cast<const uint16_t *>(ks + f0 * 8 + 2 * c4 + (16 * kg + 8 * hf) * 8));
                    sc[kg][hf] = reinterpret_cast<const __half2 &>(h);
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // eight dims of each lane: two steps
                uint32_t a[kGroups][2][4];
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint4 &u = kr[kg][hf];
                        const uint32_t w = k == 0 ? u.x : (k == 1 ? u.y : (k == 2 ? u.z : u.w));
                        const __half2 two = k < 2 ? __low2half2(sc[kg][hf]) : __high2half2(sc[kg][hf]);
                        const uint32_t by = reinterpret_cast<const uint32_t &>(two);
                        a[kg][0][hf] = half2_mul(half_of_codes<0>(w), by);
                        a[kg][0][2 + hf] = half2_mul(half_of_codes<1>(w), by);
                        a[kg][1][hf] = half2_mul(half_of_codes<2>(w), by);
                        a[kg][1][2 + hf] = half2_mul(half_of_codes<3>(w), by);
                    }
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint4 f = qf[((t * NB + n) * 4 + k) * 32 + lane];
#pragma unroll
                        for (int kg = 0; kg < kGroups; ++kg) {
                            mma<F16>(s[kg][n], a[kg][0], f.x, f.y);
                            mma<F16>(s[kg][n], a[kg][1], f.z, f.w);
                        }
                    }
            }
        } else {
            constexpr int kBlocks = kD / (4 * S::kE), kWords = 4 / kBlocks;  // pairs of steps of a chunk
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                uint4 kr[kGroups][2];
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
                        kr[kg][hf] = *reinterpret_cast<const uint4 *>(sk + cell_off<C>(f0, 4 * b + c4) + (16 * kg + 8 * hf) * S::kRowBytes);
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                    uint32_t a[kGroups][2][4];
#pragma unroll
                    for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t w[4] = {kr[kg][hf].x, kr[kg][hf].y, kr[kg][hf].z, kr[kg][hf].w};
                            if constexpr (C == QSA_E4M3) {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    a[kg][i][hf] = half_of_e4m3<0>(w[2 * j + i]);
                                    a[kg][i][2 + hf] = half_of_e4m3<1>(w[2 * j + i]);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    a[kg][i][hf] = w[2 * i];
                                    a[kg][i][2 + hf] = w[2 * i + 1];
                                }
                            }
                        }
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint4 f = qf[((t * NB + n) * 4 + b * kWords + j) * 32 + lane];
#pragma unroll
                            for (int kg = 0; kg < kGroups; ++kg) {
                                mma<F16>(s[kg][n], a[kg][0], f.x, f.y);
                                mma<F16>(s[kg][n], a[kg][1], f.z, f.w);
                            }
                        }
                }
            }
        }
        // ---- log2 units (codes: with the exponent of the cell's values, x = logit + e), masked; the reference moves
        // where one is too far above it
        float inv_e[kGroups][2];  // 2^-e of this thread's cells
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float2 by = F16 ? *reinterpret_cast<const float2 *>(undo + 8 * n + 2 * c4) : make_float2(key_scale, key_scale);
#pragma unroll
            for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float2 y = mul2(make_float2(s[kg][n][2 * hf], s[kg][n][2 * hf + 1]), by);
                    s[kg][n][2 * hf] = y.x;
                    s[kg][n][2 * hf + 1] = y.y;
                }
        }
        if constexpr (F16) {
#pragma unroll
            for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float4 e4 = ex[16 * kg + 8 * hf + f0];
                    inv_e[kg][hf] = e4.z;
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const float2 y = fma2(make_float2(s[kg][n][2 * hf], s[kg][n][2 * hf + 1]), make_float2(e4.x, e4.x), make_float2(e4.y, e4.y));
                        s[kg][n][2 * hf] = y.x;
                        s[kg][n][2 * hf + 1] = y.y;
                    }
                }
        }
        if (edge) {
#pragma unroll
            for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int c = 16 * kg + 8 * hf + f0;
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (hide(c, n, e)) s[kg][n][2 * hf + e] = -INFINITY;
                }
        }
        bool move = false;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
                for (int kg = 1; kg < kGroups; ++kg) top[e] = fmaxf(top[e], fmaxf(s[kg][n][e], s[kg][n][2 + e]));
            }
            move |= fmaxf(top[0] - mx[n][0], top[1] - mx[n][1]) > S::kMove;
        }
        if constexpr (F16) {
            if (!wide && far) {
                wide = true;  // so far l is in units of mx
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) ms[n][e] = mx[n][e];
            }
            move |= wide;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float b = mx[n][e], a = ms[n][e];
#pragma unroll
                    for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const float v = s[kg][n][2 * hf + e];
                            b = fmaxf(b, v - S::kBelow);
                            if constexpr (F16) {
                                if (wide) a = fmaxf(a, v - ex[16 * kg + 8 * hf + f0].y);
                            }
                        }
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, k));
                    const float ao = ex2_approx(mx[n][e] - b);
                    mx[n][e] = b;
                    float al = ao;
                    if constexpr (F16) {
                        if (wide) {
#pragma unroll
                            for (int k = 4; k < 32; k <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, k));
                            al = ex2_approx(ms[n][e] - a);
                            ms[n][e] = a;
                        }
                    }
                    l[n][e] *= al;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        o[t][n][e] *= ao;
                        o[t][n][2 + e] *= ao;
                    }
                }
        }
        if constexpr (F16) {
            if (wide) {
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            l[n][i & 1] += ex2_approx(s[kg][n][i] - ex[16 * kg + 8 * (i >> 1) + f0].y - ms[n][i & 1]);
            }
        }
        // ---- weights and their product with the values, 16 cells at a time
#pragma unroll
        for (int kg = 0; kg < kGroups; ++kg) {
            uint32_t p[NB][NT][2];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                float w[2][2];  // [cell half][row]
                float2 l2 = make_float2(l[n][0], l[n][1]);
                const float2 m2 = make_float2(-mx[n][0], -mx[n][1]);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const float2 d = add2(make_float2(s[kg][n][2 * hf], s[kg][n][2 * hf + 1]), m2);
                    w[hf][0] = ex2_approx(d.x);
                    w[hf][1] = ex2_approx(d.y);
                    const float2 w2 = make_float2(w[hf][0], w[hf][1]);
                    if constexpr (F16) {
                        if (!wide) l2 = fma2(w2, make_float2(inv_e[kg][hf], inv_e[kg][hf]), l2);
                    } else {
                        l2 = add2(l2, w2);
                    }
                }
                l[n][0] = l2.x;
                l[n][1] = l2.y;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) p[n][t][hf] = transposed(pack16<F16>(w[hf][0], w[hf][1]));
            }
            if constexpr (C == QSA_E2M1) {
                // cells 2 c4, 2 c4 + 1 of the fragment (and + 8): eight bytes of their rows, the codes of two
                // cells interleaved so that a byte holds a pair
                const uint32_t at_a = cell_off<C>(va, g8 >> 1) + (g8 & 1) * 8, at_b = cell_off<C>(vb, g8 >> 1) + (g8 & 1) * 8;
                uint2 v[2][2];
                uint32_t by[2];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = 16 * kg + 8 * hf;
                    v[hf][0] = *reinterpret_cast<const uint2 *>(sv + at_a + r * S::kRowBytes);
                    v[hf][1] = *reinterpret_cast<const uint2 *>(sv + at_b + r * S::kRowBytes);
                    const unsigned char *const sc = vs + r * 8 + g8;
                    by[hf] = half_of_scales(__byte_perm((uint32_t)sc[va * 8], (uint32_t)sc[vb * 8], 0x5540));
                }
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {
                    uint32_t lo[2], hi[2];  // dims 0, 2, 4, 6 and 1, 3, 5, 7
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t a = hw ? v[hf][0].y : v[hf][0].x, b = hw ? v[hf][1].y : v[hf][1].x;
                        lo[hf] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
                        hi[hf] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
                    }
#define QSA_FOUR_STEP(i)                                                                                              \
    {                                                                                                                 \
const uint32_t a[4] = {half2_mul(half_of_codes<i>(lo[0]), by[0]), half2_mul(half_of_codes<i>(hi[0]), by[0]), \
                       half2_mul(half_of_codes<i>(lo[1]), by[1]), half2_mul(half_of_codes<i>(hi[1]), by[1])}; \
_Pragma("unroll") for (int n = 0; n < NB; ++n)                                                               \
    _Pragma("unroll") for (int t = 0; t < NT; ++t) mma<F16>(o[4 * hw + i][n], a, p[n][t][0], p[n][t][1]);    \
    }
                    QSA_FOUR_STEP(0)
                    QSA_FOUR_STEP(1)
                    QSA_FOUR_STEP(2)
                    QSA_FOUR_STEP(3)
#undef QSA_FOUR_STEP
                }
            } else if constexpr (C == QSA_E4M3) {
                uint4 v[2][2];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        v[hf][e] = *reinterpret_cast<const uint4 *>(sv + cell_off<C>(2 * c4 + e, g8) + (16 * kg + 8 * hf) * S::kRowBytes);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t pr[2][2];  // [half][dims 0, 1 / 2, 3]: codes of two cells side by side
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint4 &a4 = v[hf][0], &b4 = v[hf][1];
                        const uint32_t a = w == 0 ? a4.x : (w == 1 ? a4.y : (w == 2 ? a4.z : a4.w));
                        const uint32_t b = w == 0 ? b4.x : (w == 1 ? b4.y : (w == 2 ? b4.z : b4.w));
                        pr[hf][0] = __byte_perm(a, b, 0x5140);
                        pr[hf][1] = __byte_perm(a, b, 0x7362);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a[4] = {half_of_e4m3<0>(pr[0][i]), half_of_e4m3<1>(pr[0][i]), half_of_e4m3<0>(pr[1][i]),
                                               half_of_e4m3<1>(pr[1][i])};
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma<F16>(o[2 * w + i][n], a, p[n][t][0], p[n][t][1]);
                    }
                }
            } else {
                // lanes 8 m .. 8 m + 7 give the rows of matrix m: cells 0-7 and 8-15, dims 0-7 and 8-15 in turn
                const int r = (lane & 7) + 8 * (lane >> 4);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    uint32_t a[4];
                    ldsm_x4_t(a, sv + cell_off<C>(r, 2 * t + ((lane >> 3) & 1)));
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int u = 0; u < NT; ++u) mma<F16>(o[t][n], a, p[n][u][0], p[n][u][1]);
                }
            }
        }
    }

    // Behind the last stage: the sums over the warp's lanes, in units of ms; o stays in units of mx.
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (mx[n][e] == kUnset) mx[n][e] = -INFINITY;
                if (!F16 || !wide) ms[n][e] = mx[n][e];
                if (ms[n][e] == kUnset) ms[n][e] = -INFINITY;
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], k);
            }
    }
};

}  // namespace few
}  // namespace qsa
