// dense_decode.cu -- attention of a few new tokens per sequence over a paged (or packed) cache: fp32
// queries, and bf16 queries of up to 16 rows over short contexts (longer ones: dense_few_tc.cu).  Bound
// by latency (one sequence of 2,050 cells, 8 / 2 heads, bf16: 11.9 us with the join), by the
// instructions of the conversion on long e4m3 contexts.
//
// Mathematics: with s_j the logit of cell j in log2 units, a part of a row's cells gives
// (m, l, o) = (reference, sum 2^(s_j - m), sum 2^(s_j - m) v_j), and parts join by scaling to a
// common m.  m need not be the maximum: it moves only when a logit passes it by more than 8, so
// sums and weights stay within 2^8 of the largest and the common tile needs no reduction across
// lanes, one vote only.  On e4m3 cells v_j = c_j 2^e_j; the weight that multiplies the code is
// 2^(s_j + e_j - mx) with a reference of its own, so that the fp16 weights keep their bits on
// the cells that matter for o whatever the rows' exponents are; the sum l then adds 2^-e_j times it (and,
// where exponents lie more than 2^50 from one, exponentials of the logits alone).  fp16 weights end at
// 2^-25, so mx lies 13 below the maximum where it is set, and moves when a logit passes that by more than 2:
// the largest weight is 2^13 to 2^15, and a weight that the product loses is 2^-38 of it or less.
//
// Shape: a CTA of four warps takes a share of the flattened list of (sequence, KV head, row
// tile) items (dense.cuh), equal for every CTA, whatever the lengths: ragged batches stay
// balanced and a captured graph follows lengths that change in place.  The rows of an item (new
// tokens x the heads of its KV head) are one 16-row fragment of mma.m16n8k16; these
// tensor instructions suffice since 16 rows per 256 or 512 bytes of K and V leave them under a
// third busy.  Each warp runs its own ring of stages (cp.async, 8 KB each) over its own 16
// (bf16) or 32 (e4m3) cells of every tile and meets the others only at the end of a part.
// Fragments: a thread loads 16 contiguous bytes of a key row and uses them as the k indices it
// is due (the query's fragments are permuted alike), so e4m3 codes go from shared memory to
// registers to fp16 (exact) without a shuffle; values of two keys are interleaved by byte
// permutes.  An item's parts in several CTAs are joined by a second kernel (dense_join.cuh).
//
// fp32 queries are carried as three bf16 terms (24 significant bits) on a bf16 cache and as two
// fp16 terms (22 bits, scaled by the row's largest magnitude) on an e4m3 cache, and so are the
// weights: the products of memory-bound rows cost nothing.  bf16 queries are exact in one term;
// their weights are rounded to 16 bits as the bf16 output does not keep more.
#include <cuda_fp8.h>

#include "dense_join.cuh"
#include "mma_frag.cuh"
#include "umma.cuh"

namespace qsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kD = 128;
constexpr uint32_t kTile = 4096;                 // bytes of K (and of V) of a warp's stage
// A reference lies kBelow under the maximum where it is set, and moves once a logit is kMove above it.
template <bool E8>
constexpr float kBelow = E8 ? 13.0f : 0.0f;
template <bool E8>
constexpr float kMove = E8 ? 15.0f : 8.0f;
// Exponents of e4m3 rows within 2^+-50 of one: their sums are taken from the weights (2^(x - mx)
// times 2^-e stays far from fp32's ends); beyond it they get exponentials of their own.
constexpr float kFar = 50.0f;

// Stages of a warp's ring and CTAs per SM: a warp is a long chain of dependent instructions (a tile
// takes it over a thousand cycles whatever the memory does), so the more of them the better, as far
// as registers go: twelve warps with one term of a query, eight with several.
template <int NT>
struct Plan {
    static constexpr int kCtas = NT == 1 ? 3 : 2;
    static constexpr int kStages = NT == 1 ? 2 : 3;
};

template <bool E8>
struct Shape {
    static constexpr int kRowBytes = E8 ? kD : 2 * kD;
    static constexpr int kKeys = (int)kTile / kRowBytes;  // a warp's cells of a tile: 16 or 32
    static constexpr int kGroups = kKeys / 16;
};

template <int NT>
__host__ __device__ constexpr size_t q_bytes()
{
    return (size_t)NT * 8 * 32 * 16;  // fragments: 8 k steps x 32 lanes x 16 bytes
}
template <bool E8, int NT>
__host__ __device__ constexpr size_t decode_smem()
{
    return (size_t)kWarps * Plan<NT>::kStages * 2 * kTile + q_bytes<NT>() +
           (E8 ? (size_t)kWarps * Plan<NT>::kStages * 32 * 16 : 0);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// Two e4m3 codes (low byte first) as two fp16 values, exact.
__device__ __forceinline__ uint32_t half_pair(uint32_t codes)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(codes));
    return r;
}
__device__ __forceinline__ uint32_t half_pair_hi(uint32_t codes)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(codes));
    return r;
}

// Offset of 16-byte chunk c of row r in a tile of K: rows of two parities in different halves
// of the banks, for reads of two rows x four chunks.
template <bool E8>
__device__ __forceinline__ uint32_t k_off(int r, int c)
{
    return (uint32_t)r * Shape<E8>::kRowBytes + (uint32_t)((c ^ ((r & 1) << 2)) << 4);
}
// The same of V: bf16 rows are read by ldmatrix (eight rows of one chunk), e4m3 rows in 8-byte
// words (rows 2c of four lanes, two chunks).
template <bool E8>
__device__ __forceinline__ uint32_t v_off(int r, int c)
{
    const int x = E8 ? (((r >> 1) & 3) << 1) : (r & 7);
    return (uint32_t)r * Shape<E8>::kRowBytes + (uint32_t)((c ^ x) << 4);
}

// ------------------------------------------------------------------ the kernel
// E8: e4m3 cells (else bf16).  TQ: type of q and out;
// NT: 16-bit terms of a query or weight.
template <bool E8, typename TQ, int NT>
__global__ void __launch_bounds__(kThreads, (Plan<NT>::kCtas))
dense_decode_kernel(const KvView kv, const SeqView sv, const WorkShape ws, const TQ *__restrict__ q,
                    int64_t ld_q, int H_q, float scale_log2, float q_sign, TQ *__restrict__ out,
                    float *__restrict__ lse, float *__restrict__ partial, Split *__restrict__ splits,
                    int by_item)
{
    using S = Shape<E8>;
    constexpr int kRows = 16, kStages = Plan<NT>::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int bad_s, odd_s;
    __shared__ float red_m[kWarps][kRows], red_l[kWarps][kRows], top_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c4 = lane & 3;
    unsigned char *ring = smem + (size_t)warp * kStages * 2 * kTile;
    uint4 *qf = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * kStages * 2 * kTile);
    // per cell of a stage (E8): factor of the logit, exponent e of the value, 2^-e
    float4 *exps = reinterpret_cast<float4 *>(reinterpret_cast<unsigned char *>(qf) + q_bytes<NT>()) +
                   warp * kStages * 32;

    pdl_wait();
    const TQ *qp = q;
    QSA_AFTER_WAIT(qp);
    pdl_trigger();

    const float inv_scale = 1.0f / scale_log2;
    int64_t per, x, x1;
    WorkItem it;
    const int G = H_q / kv.H_kv;
    if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
    if (!work_share(sv, ws, blockIdx.x, gridDim.x, per, x, x1, it)) return;
    for (;;) {
        const int64_t item_end = it.start + it.tiles;
        const int tile0 = (int)(x - it.start);
        const int tile1 = (int)((item_end < x1 ? item_end : x1) - it.start);
        const bool starts = tile0 == 0, ends = tile1 == it.tiles;
        int64_t t0;
        int len;
        seq_tokens(sv, it.s, t0, len);
        const int cells = seq_cells(sv, it.s, len);
        const bool fits = cells_fit(kv, cells);
        const int n_see = fits ? item_cells(ws, len, cells, it.t) : 0;
        const int tok0 = it.t * ws.rt;
        const int rows = min(ws.rt, len - tok0) * G;
        // the first token's position: cells behind it are not seen by every row
        const int pos0 = ws.causal ? cells - len + tok0 : cells - 1;

        __syncthreads();  // the previous part's shared memory is free
        if (tid == 0) bad_s = odd_s = 0;
        // ---- the ring (its first copies are under way before the queries are looked at): a tile's cells are looked up two turns before its copies are issued (p_next,
        // entry_next: this lane's cell of the next tile to issue, and its page)
        const int my_key = lane < S::kKeys ? lane : 0;
        bool bad = false, odd = false;
        int32_t p_next = -1, entry_next = -1;
        auto look_up = [&](int tile) {
            const int p = tile * ws.kt + warp * S::kKeys + my_key;
            p_next = tile < tile1 && p < n_see ? p : -1;
            if (kv.table && p_next >= 0) {
                const int64_t j = p >> kv.page_shift;
                entry_next = j < kv.ld_table ? kv.table[(int64_t)it.s * kv.ld_table + j] : -1;
            }
        };
        auto row_next = [&]() -> int32_t {
            if (p_next < 0) return -1;  // not there: zeros
            if (!kv.table) return (int32_t)t0 + p_next;
            if ((uint32_t)entry_next >= (uint32_t)kv.n_pages) {
                bad = true;
                return -1;
            }
            return (entry_next << kv.page_shift) | (p_next & ((1 << kv.page_shift) - 1));
        };
        int pend_k[kStages - 1], pend_v[kStages - 1];  // exponents on their way
        auto load_exps = [&](int32_t row, int i) {
            pend_k[i] = row >= 0 ? kv.K_exp[(int64_t)row * kv.H_kv + it.g] : kExpBias;
            pend_v[i] = row >= 0 ? kv.V_exp[(int64_t)row * kv.H_kv + it.g] : kExpBias;
        };
        constexpr int kChunks = S::kRowBytes / 16, kAt = 32 / kChunks;
        const int cc = lane & (kChunks - 1), r0 = lane / kChunks;
        const unsigned char *Kl =
            static_cast<const unsigned char *>(kv.K) + (int64_t)it.g * S::kRowBytes + cc * 16;
        const unsigned char *Vl =
            static_cast<const unsigned char *>(kv.V) + (int64_t)it.g * S::kRowBytes + cc * 16;
        const int ldk_b = (int)kv.ld_k * (E8 ? 1 : 2), ldv_b = (int)kv.ld_v * (E8 ? 1 : 2);
        auto issue = [&](int stage, int32_t row) {
            const uint32_t st = smem_u32(ring + stage * 2 * kTile);
#pragma unroll
            for (int i = 0; i < S::kKeys / kAt; ++i) {
                const int r = r0 + kAt * i;
                const int32_t rr = __shfl_sync(0xffffffffu, row, r);
                const bool on = rr >= 0;
                const int64_t at = on ? rr : 0;
                cp16(st + k_off<E8>(r, cc), Kl + at * ldk_b, on);
                cp16(st + kTile + v_off<E8>(r, cc), Vl + at * ldv_b, on);
            }
        };
        look_up(tile0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            const int32_t row = row_next();
            look_up(tile0 + i + 1);
            if (tile0 + i < tile1) {
                issue(i, row);
                if constexpr (E8) load_exps(row, i);
            }
            cp_commit();
        }
        // ---- the query's fragments: lane's rows g8 and g8 + 8 of each fragment, k permuted as
        // the key rows are read (thread c4 holds 16 contiguous bytes of each block)
        float q_back = 1.0f;  // what undoes the queries' scaling
        {
            constexpr int E = E8 ? 16 : 8;       // dims of a thread in a block
            constexpr int kBlocks = kD / (4 * E);
            auto load_row = [&](int hf, float *xa) {
                const int r = g8 + 8 * hf;
                const TQ *src =
                    qp + (t0 + tok0 + r / G) * ld_q + (int64_t)(it.g * G + r % G) * kD + c4 * E;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int e = 0; e < E; e += 8) {
                        if (r < rows) {
                            load8(src + b * 4 * E + e, xa + b * E + e);
                        } else {
#pragma unroll
                            for (int k = 0; k < 8; ++k) xa[b * E + e + k] = 0.0f;
                        }
                    }
            };
            float mul = q_sign;
            if constexpr (E8) {
                // fp16 holds the queries once the tile's largest magnitude is below 2^8: one power
                // of two for all rows, as a row 2^20 times smaller than another keeps 2^-13 of its
                // own largest value and has logits that much smaller
                if (warp == 0) {
                    float top = 0.0f;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float xa[kBlocks * E];
                        load_row(hf, xa);
#pragma unroll
                        for (int e = 0; e < kBlocks * E; ++e)
                            if (isfinite(xa[e])) top = fmaxf(top, fabsf(xa[e]));
                    }
                    top = warp_max(top);
                    if (lane == 0) top_s = top;
                }
                __syncthreads();
                const float top = top_s;
                const int ex = (int)(__float_as_uint(top) >> 23) - 127;
                const int sh = top > 0.0f ? min(max(7 - ex, -120), 100) : 0;
                q_back = two_to(-sh);
                mul = q_sign * two_to(sh);
            }
            if (warp == 0) {
                float xa[2][kBlocks * E];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    load_row(hf, xa[hf]);
#pragma unroll
                    for (int e = 0; e < kBlocks * E; ++e) xa[hf][e] *= mul;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        uint4 f;
                        f.x = pack16<E8>(xa[0][4 * k], xa[0][4 * k + 1]);
                        f.y = pack16<E8>(xa[1][4 * k], xa[1][4 * k + 1]);
                        f.z = pack16<E8>(xa[0][4 * k + 2], xa[0][4 * k + 3]);
                        f.w = pack16<E8>(xa[1][4 * k + 2], xa[1][4 * k + 3]);
                        qf[(n * 8 + k) * 32 + lane] = f;
                    }
            }
        }
        __syncthreads();
        const float key_scale = scale_log2 * q_back;
        auto keep_exps = [&](int stage, int i) {
            const int ek = min(max(pend_k[i] - kExpBias, kExpMin), kExpMax);
            const int ev = min(max(pend_v[i] - kExpBias, kExpMin), kExpMax);
            exps[stage * 32 + lane] = make_float4(two_to(ek) * key_scale, (float)ev, two_to(-ev), 0.0f);
        };
        if constexpr (E8) {
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i)
                if (tile0 + i < tile1) keep_exps(i, i);
        }
        int last[2];  // the last cell each row sees
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int r = g8 + 8 * hf;
            last[hf] = r < rows ? (ws.causal ? pos0 + r / G : cells - 1) : -1;
        }

        // mx: the rows' reference; l: the sums in its units.  E8 with exponents far apart (wide):
        // l in units of ms, a reference of the logits alone.
        float o[16][4];
        float ms[2], mx[2], l[2];
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
        ms[0] = ms[1] = mx[0] = mx[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
        bool wide = false;

        int slot = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            cp_wait<kStages - 2>();
            __syncwarp();
            const unsigned char *sk = ring + slot * 2 * kTile, *sv_ = sk + kTile;
            const float4 *ex = exps + slot * 32;
            const int j0 = tile * ws.kt + warp * S::kKeys;
            // ---- issue the tile kStages - 1 ahead into the stage read in the last turn
            {
                const int nslot = slot == 0 ? kStages - 1 : slot - 1;
                const int32_t row = row_next();
                look_up(tile + kStages);
                if (tile + kStages - 1 < tile1) {
                    issue(nslot, row);
                    if constexpr (E8) load_exps(row, 0);
                }
                cp_commit();
            }
            if (j0 < n_see) {
                const bool edge = j0 + S::kKeys - 1 > pos0;  // some row may not see some cell
                // values that not every row sees: what is infinite or NaN among them becomes
                // zero here and is added to the rows that see it at the end
                if (edge) {
                    bool here = false;
                    for (int r = max(0, pos0 + 1 - j0); r < S::kKeys && j0 + r < n_see; ++r) {
                        unsigned char *row = const_cast<unsigned char *>(sv_);
                        if constexpr (E8) {
                            uint32_t *w = reinterpret_cast<uint32_t *>(
                                row + v_off<E8>(r, lane >> 2) + (lane & 3) * 4);
                            const uint32_t v = *w;
                            const uint32_t m = __vcmpeq4(v & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            here |= m != 0;
                            if (m) *w = v & ~m;
                        } else {
                            uint2 *w = reinterpret_cast<uint2 *>(row + v_off<E8>(r, lane >> 1) + (lane & 1) * 8);
                            uint2 v = *w;
                            const uint32_t m0 = __vcmpeq2(v.x & 0x7f807f80u, 0x7f807f80u);
                            const uint32_t m1 = __vcmpeq2(v.y & 0x7f807f80u, 0x7f807f80u);
                            here |= (m0 | m1) != 0;
                            if (m0 | m1) *w = make_uint2(v.x & ~m0, v.y & ~m1);
                        }
                    }
                    odd |= here;
                    __syncwarp();
                }
                // ---- logits: fragments of 16 rows x 8 cells
                float s[S::kGroups * 2][4];
#pragma unroll
                for (int n = 0; n < S::kGroups * 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
                constexpr int kBlocks = E8 ? 2 : 4, kStepsPer = 8 / kBlocks;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    uint4 kr[S::kGroups * 2];
#pragma unroll
                    for (int n = 0; n < S::kGroups * 2; ++n)
                        kr[n] = *reinterpret_cast<const uint4 *>(sk + k_off<E8>(8 * n + g8, 4 * b + c4));
#pragma unroll
                    for (int j = 0; j < kStepsPer; ++j) {
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint4 f = qf[(t * 8 + b * kStepsPer + j) * 32 + lane];
                            const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                            for (int n = 0; n < S::kGroups * 2; ++n) {
                                const uint32_t w[4] = {kr[n].x, kr[n].y, kr[n].z, kr[n].w};
                                if constexpr (E8)
                                    mma<true>(s[n], a, half_pair(w[j]), half_pair_hi(w[j]));
                                else
                                    mma<false>(s[n], a, w[2 * j], w[2 * j + 1]);
                            }
                        }
                    }
                }
                // ---- masked, and the references moved where they have to: on bf16 cells the raw
                // logit is compared, on e4m3 cells x = logit + e in log2 units takes its place
                bool far = false;
                if constexpr (E8) {
#pragma unroll
                    for (int n = 0; n < S::kGroups * 2; ++n) {
                        const float4 f0 = ex[8 * n + 2 * c4], f1 = ex[8 * n + 2 * c4 + 1];
                        far |= fabsf(f0.y) > kFar || fabsf(f1.y) > kFar;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            s[n][2 * hf] = fmaf(s[n][2 * hf], f0.x, f0.y);
                            s[n][2 * hf + 1] = fmaf(s[n][2 * hf + 1], f1.x, f1.y);
                        }
                    }
                }
                if (edge) {
#pragma unroll
                    for (int n = 0; n < S::kGroups * 2; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (j0 + 8 * n + 2 * c4 + (i & 1) > last[i >> 1]) s[n][i] = -INFINITY;
                }
                bool move = false;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    // (-inf before the first cell: any finite logit moves it)
                    const float over = E8 ? mx[hf] + kMove<E8> : (mx[hf] + kMove<E8>) * inv_scale;
#pragma unroll
                    for (int n = 0; n < S::kGroups * 2; ++n)
                        move |= fmaxf(s[n][2 * hf], s[n][2 * hf + 1]) > over;
                }
                if constexpr (E8) {
                    if (!wide && __any_sync(0xffffffffu, far)) {
                        wide = true;  // so far l is in units of mx
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) ms[hf] = mx[hf];
                    }
                    move |= wide;
                }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float b = mx[hf], a = ms[hf];
#pragma unroll
                        for (int n = 0; n < S::kGroups * 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float v = s[n][2 * hf + e];
                                b = fmaxf(b, E8 ? v - kBelow<E8> : v * scale_log2);
                                if constexpr (E8) {
                                    if (wide) a = fmaxf(a, v - ex[8 * n + 2 * c4 + e].y);
                                }
                            }
                        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 1));
                        b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 2));
                        const float ao = b == -INFINITY ? 1.0f : ex2_approx(mx[hf] - b);
                        mx[hf] = b;
                        float al = ao;
                        if constexpr (E8) {
                            if (wide) {
                                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
                                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
                                al = a == -INFINITY ? 1.0f : ex2_approx(ms[hf] - a);
                                ms[hf] = a;
                            }
                        }
                        l[hf] *= al;
#pragma unroll
                        for (int n = 0; n < 16; ++n) {
                            o[n][2 * hf] *= ao;
                            o[n][2 * hf + 1] *= ao;
                        }
                    }
                }
                // ---- weights and their product with the values, 16 cells at a time
#pragma unroll
                for (int kg = 0; kg < S::kGroups; ++kg) {
                    uint32_t a[NT][4];
                    float2 iv[2];  // 2^-e of this thread's cells
                    if constexpr (E8) {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float4 *f = ex + 8 * (2 * kg + n) + 2 * c4;
                            iv[n] = make_float2(f[0].z, f[1].z);
                        }
                    }
                    float w[2][2][2];  // [n tile][row half][cell]
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float ux = mx[hf] == -INFINITY ? 0.0f : mx[hf];
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float v = s[2 * kg + n][2 * hf + e];
                                const float p = ex2_approx(E8 ? v - ux : fmaf(v, scale_log2, -ux));
                                w[n][hf][e] = p;
                                if constexpr (E8) {
                                    const float g = e ? iv[n].y : iv[n].x;
                                    if (!wide) l[hf] = fmaf(p, g, l[hf]);
                                } else {
                                    l[hf] += p;
                                }
                            }
                    }
                    if constexpr (E8) {
                        if (wide) {
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const float us = ms[hf] == -INFINITY ? 0.0f : ms[hf];
#pragma unroll
                                for (int n = 0; n < 2; ++n)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        l[hf] += ex2_approx(s[2 * kg + n][2 * hf + e] -
                                                            ex[8 * (2 * kg + n) + 2 * c4 + e].y - us);
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        a[t][0] = pack16<E8>(w[0][0][0], w[0][0][1]);
                        a[t][1] = pack16<E8>(w[0][1][0], w[0][1][1]);
                        a[t][2] = pack16<E8>(w[1][0][0], w[1][0][1]);
                        a[t][3] = pack16<E8>(w[1][1][0], w[1][1][1]);
                    }
                    if constexpr (E8) {
                        // cells 2c4, 2c4 + 1 (and + 8): 8-byte words of their rows, interleaved
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint2 v[4];
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const int r = 16 * kg + 2 * c4 + (kk & 1) + 8 * (kk >> 1);
                                v[kk] = *reinterpret_cast<const uint2 *>(
                                    sv_ + v_off<E8>(r, 4 * i + (g8 >> 1)) + (g8 & 1) * 8);
                            }
#pragma unroll
                            for (int hw = 0; hw < 2; ++hw) {
                                const uint32_t v0 = hw ? v[0].y : v[0].x, v1 = hw ? v[1].y : v[1].x;
                                const uint32_t v2 = hw ? v[2].y : v[2].x, v3 = hw ? v[3].y : v[3].x;
#pragma unroll
                                for (int p = 0; p < 2; ++p) {
                                    const uint32_t sel = p ? 0x7362u : 0x5140u;
                                    const uint32_t lo = __byte_perm(v0, v1, sel);
                                    const uint32_t hi = __byte_perm(v2, v3, sel);
                                    const uint32_t b0 = half_pair(lo), b1 = half_pair(hi);
                                    const uint32_t d0 = half_pair_hi(lo), d1 = half_pair_hi(hi);
                                    const int n = 8 * i + 4 * hw + 2 * p;
#pragma unroll
                                    for (int t = 0; t < NT; ++t) {
                                        mma<true>(o[n], a[t], b0, b1);
                                        mma<true>(o[n + 1], a[t], d0, d1);
                                    }
                                }
                            }
                        }
                    } else {
                        const int r = 16 * kg + (lane & 7) + 8 * ((lane >> 3) & 1);
#pragma unroll
                        for (int np = 0; np < 8; ++np) {
                            uint32_t b[4];
                            ldsm_x4_t(b, sv_ + v_off<E8>(r, 2 * np + (lane >> 4)));
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                mma<false>(o[2 * np], a[t], b[0], b[1]);
                                mma<false>(o[2 * np + 1], a[t], b[2], b[3]);
                            }
                        }
                    }
                }
            }
            if constexpr (E8) {
                const int nslot = slot == 0 ? kStages - 1 : slot - 1;
                if (tile + kStages - 1 < tile1) keep_exps(nslot, 0);
            }
            __syncwarp();
            slot = slot == kStages - 1 ? 0 : slot + 1;
        }
        cp_wait<0>();
        if (__any_sync(0xffffffffu, bad) && lane == 0) bad_s = 1;
        if (__any_sync(0xffffffffu, odd) && lane == 0) odd_s = 1;

        // ---- join the four warps: o in units of the sums' reference
        if (!E8 || !wide) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) ms[hf] = mx[hf];
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float s = l[hf];
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            l[hf] = s;
            if (c4 == 0) {
                red_m[warp][g8 + 8 * hf] = ms[hf];
                red_l[warp][g8 + 8 * hf] = s;
            }
        }
        __syncthreads();  // every warp is done with its ring
        constexpr int kPitch = kD + 4;
        float *ob = reinterpret_cast<float *>(smem);  // [warp][row][kPitch]
        static_assert((size_t)kWarps * kRows * kPitch * 4 <= (size_t)kWarps * kStages * 2 * kTile,
                      "the warps' sums fit over the ring");
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int r = g8 + 8 * hf;
            const float m = fmaxf(fmaxf(red_m[0][r], red_m[1][r]), fmaxf(red_m[2][r], red_m[3][r]));
            const float u = m == -INFINITY ? 0.0f : m;
            const float f = mx[hf] == -INFINITY ? 0.0f : exp2f(mx[hf] - u);
            float *dst = ob + (size_t)(warp * kRows + r) * kPitch;
#pragma unroll
            for (int n = 0; n < 16; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // bf16: dims 8n + 2c4 + e; e4m3: dim 64 (n / 8) + 8 (2 c4 + e) + n % 8
                    const int dim = E8 ? 64 * (n >> 3) + 8 * (2 * c4 + e) + (n & 7) : 8 * n + 2 * c4 + e;
                    dst[dim] = o[n][2 * hf + e] * f;
                }
        }
        __syncthreads();
        const bool whole = starts && ends;
        const bool nan_out = bad_s != 0 || !fits;
        float *rec = partial + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * partial_floats(kRows, kD);
        for (int e = tid; e < rows * (kD / 4); e += kThreads) {
            const int r = e / (kD / 4), c = (e % (kD / 4)) * 4;
            float m = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red_m[w][r]);
            const float u = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                sum += red_m[w][r] == -INFINITY ? red_l[w][r] : red_l[w][r] * exp2f(red_m[w][r] - u);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 p = *reinterpret_cast<const float4 *>(&ob[(size_t)(w * kRows + r) * kPitch + c]);
                v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
            }
            const int tok = tok0 + r / G;
            const int h = it.g * G + r % G;
            if (odd_s) {
                const int to = min(n_see - 1, ws.causal ? pos0 + r / G : cells - 1);
                for (int j = max(pos0 + 1, tile0 * ws.kt); j <= to && j < tile1 * ws.kt; ++j) {
                    const int64_t row = cell_row(kv, it.s, t0, j);
                    if (row >= 0)
                        for (int k = 0; k < 4; ++k)
                            v[k] += odd_value_at<E8>(kv, row * kv.ld_v + (int64_t)it.g * kD + c + k);
                }
            }
            if (nan_out) sum = NAN;
            if (whole) {
                const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                TQ *dst = out + ((t0 + tok) * H_q + h) * (int64_t)kD + c;
                if constexpr (sizeof(TQ) == 2) {
                    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv),
                                                                 pack_bf16(v[2] * inv, v[3] * inv));
                } else {
                    *reinterpret_cast<float4 *>(dst) =
                        make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                }
                if (c == 0 && lse)
                    lse[(t0 + tok) * H_q + h] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
            } else {
                *reinterpret_cast<float4 *>(rec + 2 * kRows + (int64_t)r * kD + c) =
                    make_float4(v[0], v[1], v[2], v[3]);
                if (c == 0) {
                    rec[r] = m;
                    rec[kRows + r] = sum;
                }
            }
        }
        if (starts && tid == 0) note_split(splits, by_item, it, ends, div_pos(item_end - 1, per));
        x = it.start + tile1;
        if (x >= x1) break;
        if (!work_next(sv, ws, it)) break;
    }
}

constexpr int kMaxCtas = 3 * kTargetSMs;

int decode_ctas(int per_sm)
{
    const int n = per_sm * device_sm_count();
    return n < kMaxCtas ? n : kMaxCtas;
}

template <bool E8, typename TQ, int NT>
cudaError_t run(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv;
    const WorkShape ws = work_shape(a, 16 / G, kWarps * Shape<E8>::kKeys, 0);
    // the kernel takes a positive scale: a negative one turns the queries' signs, zero clears them
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr size_t smem = decode_smem<E8, NT>();
    cudaError_t e = ensure_kernel_attrs<dense_decode_kernel<E8, TQ, NT>>(smem);
    if (e != cudaSuccess) return e;
    const int ctas = decode_ctas(Plan<NT>::kCtas);
    Split *splits = static_cast<Split *>(workspace);
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + kMaxCtas * sizeof(Split));
    e = launch(dense_decode_kernel<E8, TQ, NT>, dim3((unsigned)ctas), dim3(kThreads), smem, st, 1, a.kv,
               a.sv, ws, static_cast<const TQ *>(a.q), a.ld_q, a.H_q, scale, q_sign,
               static_cast<TQ *>(a.out), a.lse, partial, splits, (int)join_by_item(a, ws.rt, ctas));
    if (e != cudaSuccess) return e;
    return launch_dense_join<TQ>(splits, partial, ctas, 16, ws.rt, a, st);
}

}  // namespace

bool dense_decode_ok(const DenseArgs &a, int64_t max_q)
{
    const int G = a.H_q / a.kv.H_kv;
    if (a.d != kD || (a.kv_dtype != QSA_BF16 && a.kv_dtype != QSA_E4M3)) return false;
    if (a.kv_dtype == QSA_E4M3 && (a.kv.ld_k % 16 || a.kv.ld_v % 16)) return false;
    if (a.kv.ld_k > (1 << 28) || a.kv.ld_v > (1 << 28)) return false;  // strides in 32 bits
    // a fragment holds all heads of a KV head; fp32 queries come in several terms of one, however many
    // tokens; bf16 queries beyond one fragment are the tcgen05 kernels'
    return G <= 16 && (a.q_dtype == QSA_F32 || max_q * G <= 16);
}

size_t dense_decode_workspace()
{
    return kMaxCtas * sizeof(Split) + (size_t)2 * kMaxCtas * partial_floats(16, kD) * sizeof(float);
}

cudaError_t launch_dense_decode(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    const bool e8 = a.kv_dtype == QSA_E4M3;
    if (a.q_dtype == QSA_F32) return e8 ? run<true, float, 2>(a, workspace, st) : run<false, float, 3>(a, workspace, st);
    return e8 ? run<true, __nv_bfloat16, 1>(a, workspace, st) : run<false, __nv_bfloat16, 1>(a, workspace, st);
}

}  // namespace qsa
