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
// A CTA of four warps; each warp runs a ring of stages of its own (cp.async) over its own 16 (bf16) or 32 (codes)
// cells of every tile, and meets the others only at the end of a part.
//   rows of codes and values lie swizzled in shared memory, and the cells of a fragment are numbered, such that
//   both the reads along a cell (keys) and across four cells (values) touch every bank once.
#pragma once

#include "dense_join.cuh"
#include "e2m1.cuh"
#include "mma_frag.cuh"
#include "umma.cuh"

namespace qsa {
namespace few {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
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

// Stages of a warp's ring and CTAs per SM.
template <int C, int NB, int NT>
struct Plan {
    static constexpr int kCtas = NB == 4 ? 2 : (NB * NT == 1 && C == QSA_E2M1 ? 4 : 3);
    static constexpr int kStages = C == QSA_E2M1 ? (kCtas == 4 ? 2 : 3) : 2;
};

template <int NB, int NT>
__host__ __device__ constexpr size_t q_bytes() { return (size_t)NT * NB * 4 * 32 * 16; }
template <int NB>
__host__ __device__ constexpr size_t fin_bytes() { return (size_t)8 * NB * (kPitch + 2) * 4; }
template <int C, int NB, int NT, bool LIST>
__host__ __device__ constexpr size_t few_cells_smem()
{
    constexpr int S = kWarps * Plan<C, NB, NT>::kStages;
    return (size_t)S * Cell<C>::kStage + q_bytes<NB, NT>() + (Cell<C>::kF16 ? (size_t)S * 32 * 16 : 0) +
           (LIST ? fin_bytes<NB>() : 0);
}

// `bytes` (0, 8, 16) of 16 from global memory, zeros behind.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes)
{
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
// The first of the dims (and the step to the second) that rows g8 and g8 + 8 of the fragment of dims number t hold.
template <int C>
__device__ __forceinline__ int frag_dim(int t, int g8, int half)
{
    return C == QSA_BF16 ? 16 * t + 8 * half + g8 : 16 * g8 + 2 * t + half;
}

// ------------------------------------------------------------------ the kernel
// NB: blocks of eight rows.  NT: 16-bit terms of a query and a weight.  LIST: a cluster takes one token and KV head,
// its CTAs equal shares of the token's listed cells; else shares of the flattened list (dense.cuh).
template <int C, typename TQ, int NB, int NT, bool LIST>
__global__ void __launch_bounds__(kThreads, (Plan<C, NB, NT>::kCtas))
few_cells_kernel(const KvView kv, const SeqView sv, const WorkShape ws, const ListView lv, const TQ *__restrict__ q,
                 int64_t ld_q, int H_q, float scale_log2, float q_sign, TQ *__restrict__ out, float *__restrict__ lse,
                 float *__restrict__ partial, Split *__restrict__ splits, int by_item)
{
    using S = Cell<C>;
    constexpr int kRows = 8 * NB, kStages = Plan<C, NB, NT>::kStages, kKeys = S::kKeys, kGroups = S::kGroups;
    constexpr bool F16 = S::kF16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int bad_s, odd_s;
    __shared__ float red_m[kWarps][kRows], red_l[kWarps][kRows], top_s[kWarps];
    __shared__ uint32_t there_s[kWarps][kStages];  // LIST: cells of a stage that are there

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c4 = lane & 3;
    unsigned char *const ring = smem + (size_t)warp * kStages * S::kStage;
    uint4 *const qf = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * kStages * S::kStage);
    unsigned char *after_q = reinterpret_cast<unsigned char *>(qf) + q_bytes<NB, NT>();
    // per cell of a stage (codes): factor of the logit, exponent e of the value, 2^-e
    float4 *const exps = reinterpret_cast<float4 *>(after_q) + warp * kStages * 32;
    float *const fin = reinterpret_cast<float *>(after_q + (F16 ? (size_t)kWarps * kStages * 32 * 16 : 0));

    pdl_wait();
    const TQ *qp = q;
    QSA_AFTER_WAIT(qp);
    pdl_trigger();

    const float inv_scale = 1.0f / scale_log2;
    const int G = H_q / kv.H_kv;
    int64_t per = 0, x = 0, x1 = 0;
    WorkItem it = {};
    uint32_t rank = 0, ranks = 1;
    int n_list = 0, pos = 0, cells = 0;
    const int32_t *list = nullptr;
    int64_t tok = 0;
    if constexpr (LIST) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
        const unsigned item = blockIdx.x / ranks;
        tok = item / (unsigned)kv.H_kv;
        it.g = (int)(item % (unsigned)kv.H_kv);
        if (!token_place(sv, tok, it.s, pos, cells)) return;  // (all CTAs of the cluster)
        n_list = (int)min((int64_t)max(lv.counts[tok], 0), lv.k_blk);
        list = lv.blocks + tok * lv.k_blk;
        it.tiles = n_list / (ws.kt / 4) + 1;  // of 4 n_list + 4 cells
    } else {
        if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
        if (!work_share(sv, ws, blockIdx.x, gridDim.x, per, x, x1, it)) return;
    }
    for (;;) {
        int tile0, tile1, len = 1, rows = G, tok0 = 0, n_see, pos0 = 0;
        int64_t t0 = tok, item_end = 0;
        if constexpr (LIST) {
            const int share = (it.tiles + (int)ranks - 1) / (int)ranks;
            tile0 = min((int)rank * share, it.tiles);
            tile1 = min(tile0 + share, it.tiles);
        } else {
            item_end = it.start + it.tiles;
            tile0 = (int)(x - it.start);
            tile1 = (int)((item_end < x1 ? item_end : x1) - it.start);
            seq_tokens(sv, it.s, t0, len);
            cells = seq_cells(sv, it.s, len);
            tok0 = it.t * ws.rt;
            rows = min(ws.rt, len - tok0) * G;
            // the first token's position: cells behind it are not seen by every row
            pos0 = ws.causal ? cells - len + tok0 : cells - 1;
        }
        const bool starts = tile0 == 0, ends = tile1 == it.tiles;
        const bool fits = cells_fit(kv, cells);
        n_see = !fits ? 0 : (LIST ? 4 * n_list + 4 : item_cells(ws, len, cells, it.t));

        __syncthreads();  // the previous part's shared memory is free
        if (tid == 0) bad_s = odd_s = 0;
        // ---- the ring: a tile's cells (LIST: its list entries, a turn before) are looked up ahead of its copies.
        // p_next, entry_next: this lane's cell of the next tile to issue, and its page; blk_next: the list entry of
        // its cell of the tile after that
        const int my_key = lane < kKeys ? lane : 0;
        bool bad = false, odd = false;
        int32_t p_next = -1, entry_next = -1, blk_next = -1;
        auto look_page = [&](int p) {
            p_next = p;
            if (p >= 0) {
                const int64_t j = p >> kv.page_shift;
                entry_next = j < kv.ld_table ? kv.table[(int64_t)it.s * kv.ld_table + j] : -1;
            }
        };
        auto look_list = [&](int tile) {
            const int i = tile * ws.kt + warp * kKeys + my_key;
            blk_next = tile < tile1 && (i >> 2) < n_list ? list[i >> 2] : -1;
        };
        // the cell of tile `tile`, whose entry is in blk_next; then the entry of the tile after it
        auto look_up = [&](int tile) {
            const int i = tile * ws.kt + warp * kKeys + my_key;
            if constexpr (LIST) {
                int p = -1;
                if (tile < tile1 && n_see > 0) {
                    if ((i >> 2) < n_list) p = blk_next >= 0 && blk_next <= ((pos - 3) >> 2) ? 4 * blk_next + (i & 3) : -1;
                    else if ((i >> 2) == n_list && ((pos + 1) & ~3) + (i & 3) <= pos) p = ((pos + 1) & ~3) + (i & 3);
                }
                look_page(p);
                look_list(tile + 1);
            } else {
                look_page(tile < tile1 && i < n_see ? i : -1);
            }
        };
        auto row_next = [&]() -> int32_t {
            if (p_next < 0) return -1;  // not there: zeros
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
        const unsigned char *const Kl = static_cast<const unsigned char *>(kv.K) + (int64_t)it.g * S::kRowBytes + cc * 16;
        const unsigned char *const Vl = static_cast<const unsigned char *>(kv.V) + (int64_t)it.g * S::kRowBytes + cc * 16;
        const int ldk_b = (int)(C == QSA_E2M1 ? kv.ld_k / 2 : kv.ld_k * (C == QSA_BF16 ? 2 : 1));
        const int ldv_b = (int)(C == QSA_E2M1 ? kv.ld_v / 2 : kv.ld_v * (C == QSA_BF16 ? 2 : 1));
        auto issue = [&](int stage, int32_t row) {
            const uint32_t st = smem_u32(ring + stage * S::kStage);
#pragma unroll
            for (int i = 0; i < kKeys / kAt; ++i) {
                const int r = r0 + kAt * i;
                const int32_t rr = __shfl_sync(0xffffffffu, row, r);
                const int on = rr >= 0 ? 16 : 0;
                const int64_t at = rr >= 0 ? rr : 0;
                cp16(st + cell_off<C>(r, cc), Kl + at * ldk_b, on);
                cp16(st + S::kTile + cell_off<C>(r, cc), Vl + at * ldv_b, on);
            }
            if constexpr (C == QSA_E2M1) {
                // scales of two cells (neighbours in a page): K's by the lower lanes, V's by the upper
                const int pair = lane & 15;
                const int32_t ra = __shfl_sync(0xffffffffu, row, 2 * pair), rb = __shfl_sync(0xffffffffu, row, 2 * pair + 1);
                const uint8_t *const from = lane < 16 ? kv.K_scale : kv.V_scale;
                cp16(st + 2 * S::kTile + (lane < 16 ? 0 : S::kScales) + pair * 16,
                     from + scale_row(kv, ra >= 0 ? ra : 0, it.g) * 8, ra >= 0 ? (rb >= 0 ? 16 : 8) : 0);
            }
        };
        if constexpr (LIST) look_list(tile0);
        look_up(tile0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if constexpr (LIST) {
                const uint32_t there = __ballot_sync(0xffffffffu, p_next >= 0);
                if (lane == 0) there_s[warp][i] = there;
            }
            const int32_t row = row_next();
            look_up(tile0 + i + 1);
            if (tile0 + i < tile1) {
                issue(i, row);
                if constexpr (F16) load_exps(row, i);
            }
            cp_commit();
        }
        // ---- the queries' fragments, k permuted as the key rows are read: lane (g8, c4) holds row g8 of a block, and
        // kE values of each 4 kE
        float q_back = 1.0f;  // what undoes the queries' scaling
        {
            constexpr int E = S::kE, kBlocks = kD / (4 * E);
            float xa[32];
            const int r = 8 * warp + g8;
            const bool mine = warp < NB;
            if (mine) {
                const TQ *src = qp + (t0 + tok0 + (LIST ? 0 : r / G)) * ld_q + (int64_t)(it.g * G + (LIST ? r : r % G)) * kD + c4 * E;
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
            }
            float mul = q_sign;
            if constexpr (F16) {
                // fp16 holds the queries once the rows' largest magnitude is below 2^8: one power of two for all
                float top = 0.0f;
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (isfinite(xa[e])) top = fmaxf(top, fabsf(xa[e]));
                    top = warp_max(top);
                }
                if (lane == 0) top_s[warp] = top;
                __syncthreads();
                top = fmaxf(fmaxf(top_s[0], top_s[1]), fmaxf(top_s[2], top_s[3]));
                const int ex = (int)(__float_as_uint(top) >> 23) - 127;
                const int sh = top > 0.0f ? min(max(7 - ex, -120), 100) : 0;
                q_back = two_to(-sh);
                mul = q_sign * two_to(sh);
            }
            if (mine) {
#pragma unroll
                for (int e = 0; e < 32; ++e) xa[e] *= mul;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {  // two steps of 16 dims
                        uint4 f;
                        f.x = pack16<F16>(xa[8 * k], xa[8 * k + 1]);
                        f.y = pack16<F16>(xa[8 * k + 2], xa[8 * k + 3]);
                        f.z = pack16<F16>(xa[8 * k + 4], xa[8 * k + 5]);
                        f.w = pack16<F16>(xa[8 * k + 6], xa[8 * k + 7]);
                        qf[((n * NB + warp) * 4 + k) * 32 + lane] = f;
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
        if constexpr (F16) {
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i)
                if (tile0 + i < tile1) keep_exps(i, i);
        }
        // rows 8 n + 2 c4 + e, e = 0, 1, are this thread's: the last cell each sees
        int last[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * c4 + e;
                last[n][e] = r < rows ? (ws.causal ? pos0 + r / G : cells - 1) : -1;
            }

        // mx: the rows' reference; l: the sums in its units.  Exponents far apart (wide): l in units of ms, a
        // reference of the logits alone.
        float o[8][NB][4], ms[NB][2], mx[NB][2], l[NB][2];
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
                ms[n][e] = mx[n][e] = -INFINITY;
                l[n][e] = 0.0f;
            }
        bool wide = false;

        int slot = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            cp_wait<kStages - 2>();
            __syncwarp();
            unsigned char *const sk = ring + slot * S::kStage, *const sv_ = sk + S::kTile;
            const float4 *const ex = exps + slot * 32;
            const int j0 = tile * ws.kt + warp * kKeys;
            const uint32_t there = LIST ? there_s[warp][slot] : 0u;
            // ---- issue the tile kStages - 1 ahead into the stage read in the last turn
            {
                const int nslot = slot == 0 ? kStages - 1 : slot - 1;
                if constexpr (LIST) {
                    const uint32_t t = __ballot_sync(0xffffffffu, p_next >= 0);
                    if (lane == 0) there_s[warp][nslot] = t;
                }
                const int32_t row = row_next();
                look_up(tile + kStages);
                if (tile + kStages - 1 < tile1) {
                    issue(nslot, row);
                    if constexpr (F16) load_exps(row, 0);
                }
                cp_commit();
            }
            if (j0 < n_see) {
                // some row may not see some cell
                const bool edge = LIST ? (uint32_t)(there << (32 - kKeys)) != 0xffffffffu << (32 - kKeys) : j0 + kKeys - 1 > pos0;
                // values that not every row sees: what is infinite or NaN among them becomes zero here and is added
                // to the rows that see it at the end (cells that are not there are zeros already)
                if (!LIST && edge) {
                    bool here = false;
                    if constexpr (C == QSA_E2M1) {
                        if (j0 + lane > pos0 && j0 + lane < n_see) {
                            uint2 *const w = reinterpret_cast<uint2 *>(sk + 2 * S::kTile + S::kScales + lane * 8);
                            const uint2 v = *w;
                            const uint32_t m0 = __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu), m1 = __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            here = (m0 | m1) != 0;
                            if (here) *w = make_uint2(v.x & ~m0, v.y & ~m1);
                        }
                    }
                    odd |= here;
                    __syncwarp();
                }
                // ---- logits: fragments of 16 cells x 8 rows
                float s[kGroups][NB][4];
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                    for (int n = 0; n < NB; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[kg][n][e] = 0.0f;
                const int f0 = frag_cell<C>(g8);
                if constexpr (C == QSA_E2M1) {
                    uint4 kr[kGroups][2];
                    uint32_t sc[kGroups][2][2];  // scales of the lane's two groups of a cell, twice each
#pragma unroll
                    for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const int r = 16 * kg + 8 * hf + f0;
                            kr[kg][hf] = *reinterpret_cast<const uint4 *>(sk + cell_off<C>(r, c4));
                            const uint32_t h = half_of_scales(*reinterpret_cast<const uint16_t *>(sk + 2 * S::kTile + r * 8 + 2 * c4));
                            sc[kg][hf][0] = __byte_perm(h, h, 0x1010);
                            sc[kg][hf][1] = __byte_perm(h, h, 0x3232);
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
                                const uint32_t by = sc[kg][hf][k >> 1];
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
                                kr[kg][hf] = *reinterpret_cast<const uint4 *>(sk + cell_off<C>(16 * kg + 8 * hf + f0, 4 * b + c4));
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
                // ---- masked, and the references moved where they have to: of bf16 cells the raw logit is compared,
                // of codes x = logit + e in log2 units takes its place
                bool far = false;
                float inv_e[kGroups][2];  // 2^-e of this thread's cells
                if constexpr (F16) {
#pragma unroll
                    for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const float4 f = ex[16 * kg + 8 * hf + f0];
                            inv_e[kg][hf] = f.z;
                            far |= fabsf(f.y) > kFar;
#pragma unroll
                            for (int n = 0; n < NB; ++n) {
                                s[kg][n][2 * hf] = fmaf(s[kg][n][2 * hf], f.x, f.y);
                                s[kg][n][2 * hf + 1] = fmaf(s[kg][n][2 * hf + 1], f.x, f.y);
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
                                    if (LIST ? !((there >> c) & 1u) : j0 + c > last[n][e]) s[kg][n][2 * hf + e] = -INFINITY;
                        }
                }
                bool move = false;
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // (-inf before the first cell: any finite logit moves it)
                        const float over = F16 ? mx[n][e] + S::kMove : (mx[n][e] + S::kMove) * inv_scale;
#pragma unroll
                        for (int kg = 0; kg < kGroups; ++kg) move |= fmaxf(s[kg][n][e], s[kg][n][2 + e]) > over;
                    }
                if constexpr (F16) {
                    if (!wide && __any_sync(0xffffffffu, far)) {
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
                                    b = fmaxf(b, F16 ? v - S::kBelow : v * scale_log2);
                                    if constexpr (F16) {
                                        if (wide) a = fmaxf(a, v - ex[16 * kg + 8 * hf + f0].y);
                                    }
                                }
#pragma unroll
                            for (int k = 4; k < 32; k <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, k));
                            const float ao = b == -INFINITY ? 1.0f : ex2_approx(mx[n][e] - b);
                            mx[n][e] = b;
                            float al = ao;
                            if constexpr (F16) {
                                if (wide) {
#pragma unroll
                                    for (int k = 4; k < 32; k <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, k));
                                    al = a == -INFINITY ? 1.0f : ex2_approx(ms[n][e] - a);
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
                // ---- weights and their product with the values, 16 cells at a time
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg) {
                    uint32_t p[NB][NT][2];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        float w[2][2];  // [cell half][row]
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float ux = mx[n][e] == -INFINITY ? 0.0f : mx[n][e];
                                const float v = s[kg][n][2 * hf + e];
                                const float y = ex2_approx(F16 ? v - ux : fmaf(v, scale_log2, -ux));
                                w[hf][e] = y;
                                if constexpr (F16) {
                                    if (!wide) l[n][e] = fmaf(y, inv_e[kg][hf], l[n][e]);
                                    else l[n][e] += ex2_approx(v - ex[16 * kg + 8 * hf + f0].y - (ms[n][e] == -INFINITY ? 0.0f : ms[n][e]));
                                } else {
                                    l[n][e] += y;
                                }
                            }
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) p[n][t][hf] = transposed(pack16<F16>(w[hf][0], w[hf][1]));
                    }
                    if constexpr (C == QSA_E2M1) {
                        // cells 2 c4, 2 c4 + 1 of the fragment (and + 8): eight bytes of their rows, the codes of two
                        // cells interleaved so that a byte holds a pair
                        const int ra = 16 * kg + frag_cell<C>(2 * c4), rb = 16 * kg + frag_cell<C>(2 * c4 + 1);
                        uint2 v[2][2];
                        uint32_t by[2];
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            v[hf][0] = *reinterpret_cast<const uint2 *>(sv_ + cell_off<C>(ra + 8 * hf, g8 >> 1) + (g8 & 1) * 8);
                            v[hf][1] = *reinterpret_cast<const uint2 *>(sv_ + cell_off<C>(rb + 8 * hf, g8 >> 1) + (g8 & 1) * 8);
                            const unsigned char *const sc = sk + 2 * S::kTile + S::kScales;
                            by[hf] = half_of_scales((uint32_t)sc[(ra + 8 * hf) * 8 + g8] | (uint32_t)sc[(rb + 8 * hf) * 8 + g8] << 8);
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
                                v[hf][e] = *reinterpret_cast<const uint4 *>(sv_ + cell_off<C>(16 * kg + 8 * hf + 2 * c4 + e, g8));
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
                            ldsm_x4_t(a, sv_ + cell_off<C>(r, 2 * t + ((lane >> 3) & 1)));
#pragma unroll
                            for (int n = 0; n < NB; ++n)
#pragma unroll
                                for (int u = 0; u < NT; ++u) mma<F16>(o[t][n], a, p[n][u][0], p[n][u][1]);
                        }
                    }
                }
            }
            if constexpr (F16) {
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
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!F16 || !wide) ms[n][e] = mx[n][e];
                float sum = l[n][e];
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
                if (g8 == 0) {
                    red_m[warp][8 * n + 2 * c4 + e] = ms[n][e];
                    red_l[warp][8 * n + 2 * c4 + e] = sum;
                }
            }
        __syncthreads();  // every warp is done with its ring
        const bool whole = starts && ends;
        const bool nan_out = bad_s != 0 || !fits;
        float *const rec = LIST ? nullptr : partial + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * partial_floats(kRows, kD);
        constexpr int kTurn = NB > 2 ? 2 : NB;  // blocks that are joined at a time
        float *const ob = reinterpret_cast<float *>(smem);  // [warp][row][kPitch]
        static_assert((size_t)kWarps * 8 * kTurn * kPitch * 4 <= (size_t)kWarps * kStages * S::kStage, "the warps' sums fit over the ring");
#pragma unroll
        for (int n0 = 0; n0 < NB; n0 += kTurn) {
            if (n0 > 0) __syncthreads();
#pragma unroll
            for (int n = n0; n < n0 + kTurn; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * n + 2 * c4 + e;
                    const float m = fmaxf(fmaxf(red_m[0][r], red_m[1][r]), fmaxf(red_m[2][r], red_m[3][r]));
                    const float u = m == -INFINITY ? 0.0f : m;
                    const float f = mx[n][e] == -INFINITY ? 0.0f : exp2f(mx[n][e] - u);
                    float *const dst = ob + (size_t)(warp * 8 * kTurn + r - 8 * n0) * kPitch;
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) dst[frag_dim<C>(t, g8, hf)] = o[t][n][2 * hf + e] * f;
                }
            __syncthreads();
            for (int i = tid; i < 8 * kTurn * (kD / 4); i += kThreads) {
                const int rl = i / (kD / 4), r = 8 * n0 + rl, c = (i % (kD / 4)) * 4;
                if (r >= rows) break;
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
                    const float4 y = *reinterpret_cast<const float4 *>(&ob[(size_t)(w * 8 * kTurn + rl) * kPitch + c]);
                    v[0] += y.x; v[1] += y.y; v[2] += y.z; v[3] += y.w;
                }
                if (!LIST && odd_s) {
                    const int to = min(n_see - 1, ws.causal ? pos0 + r / G : cells - 1);
                    for (int j = max(pos0 + 1, tile0 * ws.kt); j <= to && j < tile1 * ws.kt; ++j) {
                        const int64_t row = cell_row(kv, it.s, t0, j);
                        if (C == QSA_E2M1 && row >= 0 && scale_is_nan(kv.V_scale[scale_row(kv, row, it.g) * 8 + (c >> 4)]))
                            v[0] = v[1] = v[2] = v[3] = NAN;
                    }
                }
                if (nan_out) sum = NAN;
                const int64_t at = (t0 + tok0 + (LIST ? 0 : r / G)) * H_q + it.g * G + (LIST ? r : r % G);
                if (LIST ? ranks == 1 : whole) {
                    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                    TQ *const dst = out + at * kD + c;
                    if constexpr (sizeof(TQ) == 2)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
                    else
                        *reinterpret_cast<float4 *>(dst) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                    if (c == 0 && lse) lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
                } else if constexpr (LIST) {
                    *reinterpret_cast<float4 *>(fin + r * kPitch + c) = make_float4(v[0], v[1], v[2], v[3]);
                    if (c == 0) {
                        fin[kRows * kPitch + r] = m;
                        fin[kRows * kPitch + kRows + r] = sum;
                    }
                } else {
                    *reinterpret_cast<float4 *>(rec + 2 * kRows + (int64_t)r * kD + c) = make_float4(v[0], v[1], v[2], v[3]);
                    if (c == 0) {
                        rec[r] = m;
                        rec[kRows + r] = sum;
                    }
                }
            }
        }
        if constexpr (LIST) {
            if (ranks > 1) {
                // ---- join the cluster's CTAs: each takes a share of the rows' values
                asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
                const uint32_t mine = smem_u32(fin);
                auto there = [&](uint32_t of, int word) {
                    uint32_t a;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(mine + 4 * (uint32_t)word), "r"(of));
                    return a;
                };
                auto load1 = [&](uint32_t a) {
                    float f;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
                    return f;
                };
                for (int i = (int)rank * kThreads + tid; i < rows * (kD / 4); i += (int)ranks * kThreads) {
                    const int r = i / (kD / 4), c = (i % (kD / 4)) * 4;
                    float m = -INFINITY, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (uint32_t k = 0; k < ranks; ++k) m = fmaxf(m, load1(there(k, kRows * kPitch + r)));
                    const float u = m == -INFINITY ? 0.0f : m;
                    for (uint32_t k = 0; k < ranks; ++k) {
                        const float km = load1(there(k, kRows * kPitch + r)), kl = load1(there(k, kRows * kPitch + kRows + r));
                        const float f = km == -INFINITY ? 1.0f : exp2f(km - u);  // an unset side is zero or NaN
                        float4 y;
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                                     : "r"(there(k, r * kPitch + c))
                                     : "memory");
                        sum += kl * f;
                        v[0] += y.x * f; v[1] += y.y * f; v[2] += y.z * f; v[3] += y.w * f;
                    }
                    const int64_t at = tok * H_q + it.g * G + r;
                    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                    TQ *const dst = out + at * kD + c;
                    if constexpr (sizeof(TQ) == 2)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
                    else
                        *reinterpret_cast<float4 *>(dst) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                    if (c == 0 && lse) lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
                }
                // no CTA leaves while another reads its part
                asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
            }
            return;
        }
        if (starts && tid == 0) note_split(splits, by_item, it, ends, div_pos(item_end - 1, per));
        x = it.start + tile1;
        if (x >= x1) break;
        if (!work_next(sv, ws, it)) break;
    }
}

}  // namespace few
}  // namespace qsa
