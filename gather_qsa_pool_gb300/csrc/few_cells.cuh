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
// A CTA of four warps; each warp runs a ring of stages of its own (cp.async) over 16 (bf16) or 32 (codes) cells of
// every tile and meets the others only at the end of a part.  The warps take one, two or four KV heads of the same
// cells (`hpc` heads of a CTA), so that the heads of a row are read together: L2 fetches more than a head's 64
// bytes of 4-bit codes, and with the heads in different CTAs 306 MB of cells took 510 MB of reads.
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
    static constexpr int kCtas = NB == 4 || NB * NT == 4 ? 2 : 3;
    static constexpr int kStages = C == QSA_E2M1 ? 3 : 2;
};

// Of one head.
template <int NB, int NT>
__host__ __device__ constexpr size_t q_bytes() { return (size_t)NT * NB * 4 * 32 * 16; }
template <int NB>
__host__ __device__ constexpr size_t fin_bytes() { return (size_t)8 * NB * (kPitch + 2) * 4; }
template <int C, int NB, int NT, bool LIST>
__host__ __device__ constexpr size_t few_cells_smem(int hpc)
{
    constexpr int S = kWarps * Plan<C, NB, NT>::kStages;
    return (size_t)S * Cell<C>::kStage + (Cell<C>::kF16 ? (size_t)S * 32 * 16 : 0) +
           hpc * (q_bytes<NB, NT>() + (LIST ? fin_bytes<NB>() : 0));
}

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

// ------------------------------------------------------------------ shares of the work
// As dense.cuh's flattened list, made short: every row tile of a sequence counts the tiles of its whole context (the
// earlier ones of a few tokens see hardly less; turns behind what they see read nothing), so that a share is found
// with shifts and a few 32-bit divisions.  (The exact list took 11,000 to 24,000 cycles at 64 sequences, most of
// them fetching code that runs once.)
struct Item {
    int32_t s, g, t;     // sequence, group of heads, row tile
    int32_t tiles;
    int32_t len, cells;  // of the sequence
    int32_t nt;          // its row tiles
    int64_t t0;          // its first token
    int64_t start;       // the item's first place in the list
    int64_t index;       // its number
};

// A sequence's tokens, cells, tiles of an item and row tiles.
__device__ __forceinline__ void look_at(const SeqView &sv, const WorkShape &w, int kt_log2, Item &it)
{
    seq_tokens(sv, it.s, it.t0, it.len);
    it.cells = seq_cells(sv, it.s, it.len);
    it.nt = it.len <= w.rt ? (it.len > 0) : (int)((uint32_t)(it.len + w.rt - 1) / (uint32_t)w.rt);
    it.tiles = it.cells > 0 && it.cells <= w.most ? ((it.cells - 1) >> kt_log2) + 1 : 1;
}

// The share of CTA `cta` of `ctas`: places [x0, x1) and the item at x0; false when there is none.  One warp calls it.
__device__ __forceinline__ bool share_of(const SeqView &sv, const WorkShape &w, int kt_log2, int cta, int ctas, int64_t &per,
                                         int64_t &x0, int64_t &x1, Item &it)
{
    const int lane = threadIdx.x & 31;
    int64_t total = 0;
#pragma unroll 1
    for (int s = lane; s < sv.n_seq; s += 32) {
        Item i;
        i.s = s;
        look_at(sv, w, kt_log2, i);
        total += (int64_t)i.tiles * ((int64_t)i.nt * w.H_kv);
    }
    total = warp_sum_i64(total);
    per = div_pos(total + ctas - 1, ctas);
    x0 = cta * per;
    x1 = x0 + per < total ? x0 + per : total;
    if (x0 >= x1) return false;
    int64_t base = 0, before = 0;  // places and items of the sequences so far
#pragma unroll 1
    for (int s0 = 0;; s0 += 32) {
        it.s = s0 + lane;
        it.nt = it.tiles = 0;
        if (it.s < sv.n_seq) look_at(sv, w, kt_log2, it);
        const int64_t items = (int64_t)it.nt * w.H_kv, mine = items * it.tiles;
        int64_t upto = mine, items_upto = items;
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o), u = __shfl_up_sync(0xffffffffu, items_upto, o);
            if (lane >= o) {
                upto += v;
                items_upto += u;
            }
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, x0 < base + upto);
        if (hit) {
            // the first lane whose sum passes x0 has it
            const int j = __ffs(hit) - 1;
            const int64_t first = base + upto - mine, n = div_pos(lane == j ? x0 - first : 0, max(it.tiles, 1));
            it.g = (int)div_pos(n, max(it.nt, 1));
            it.t = (int)(n - (int64_t)it.g * it.nt);
            it.start = first + n * it.tiles;
            it.index = before + items_upto - items + n;
            uint32_t *const words = reinterpret_cast<uint32_t *>(&it);
#pragma unroll
            for (int i = 0; i < (int)sizeof(Item) / 4; ++i) words[i] = __shfl_sync(0xffffffffu, words[i], j);
            return true;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
        before += __shfl_sync(0xffffffffu, items_upto, 31);
    }
}

// The item after `it`; false past the end.  Any thread, by itself.
__device__ __forceinline__ bool item_after(const SeqView &sv, const WorkShape &w, int kt_log2, Item &it)
{
    it.start += it.tiles;
    ++it.index;
    if (++it.t < it.nt) return true;
    it.t = 0;
    if (++it.g < w.H_kv) return true;
    it.g = 0;
    do {
        if (++it.s >= sv.n_seq) return false;
        look_at(sv, w, kt_log2, it);
    } while (it.nt == 0);
    return true;
}

// ------------------------------------------------------------------ the kernel
// NB: blocks of eight rows.  NT: 16-bit terms of a query and a weight.  LIST: a cluster takes one token and hpc KV
// heads, its CTAs equal shares of the token's listed cells; else shares of the flattened list (dense.cuh), in which
// hpc heads are one.  Warp w: head w mod hpc, cells w / hpc of a tile's 4 / hpc parts.
template <int C, typename TQ, int NB, int NT, bool LIST>
__global__ void __launch_bounds__(kThreads, (Plan<C, NB, NT>::kCtas))
few_cells_kernel(const KvView kv, const SeqView sv, const WorkShape ws, const ListView lv, const TQ *__restrict__ q,
                 int64_t ld_q, int H_q, float scale_log2, float q_sign, TQ *__restrict__ out, float *__restrict__ lse,
                 float *__restrict__ partial, Split *__restrict__ splits, int by_item, int hpc_log2, int kt_log2)
{
    using S = Cell<C>;
    constexpr int kRows = 8 * NB, kStages = Plan<C, NB, NT>::kStages, kKeys = S::kKeys, kGroups = S::kGroups;
    constexpr bool F16 = S::kF16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int bad_s, odd_s;
    __shared__ float red_m[kWarps][kRows], red_l[kWarps][kRows];
    __shared__ uint32_t top_s[kWarps];
    __shared__ uint32_t there_s[kWarps][kStages];  // LIST: cells of a stage that are there
    __shared__ Item item_s;
    __shared__ int64_t share_s[3];  // a share's places: of each CTA, the first, behind the last

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c4 = lane & 3;
    unsigned char *const ring = smem + (size_t)warp * kStages * S::kStage;
    const int hpc = 1 << hpc_log2, head = warp & (hpc - 1), part = warp >> hpc_log2;
    // per cell of a stage (codes): factor of the logit, exponent e of the value, 2^-e
    float4 *const exps = reinterpret_cast<float4 *>(smem + (size_t)kWarps * kStages * S::kStage) + warp * kStages * 32;
    uint4 *const q_all = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * kStages * (S::kStage + (F16 ? 512 : 0)));  // by head
    const uint4 *const qf = q_all + head * (int)(q_bytes<NB, NT>() / 16);
    float *const fin = reinterpret_cast<float *>(q_all + hpc * (int)(q_bytes<NB, NT>() / 16));  // LIST, rows head by head

    pdl_wait();
    const TQ *qp = q;
    QSA_AFTER_WAIT(qp);
    pdl_trigger();

    const int G = H_q / kv.H_kv;
    int64_t x = 0, x1 = 0;
    Item it;
    uint32_t rank = 0, ranks = 1;
    int n_list = 0, pos = 0, cells = 0;
    const int32_t *list = nullptr;
    int64_t tok = 0;
    if constexpr (LIST) {
        asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
        const unsigned item = blockIdx.x / ranks;
        tok = item / (unsigned)ws.H_kv;
        it.g = (int)(item % (unsigned)ws.H_kv);
        if (!token_place(sv, tok, it.s, pos, cells)) return;  // (all CTAs of the cluster)
        n_list = (int)min((int64_t)max(lv.counts[tok], 0), lv.k_blk);
        list = lv.blocks + tok * lv.k_blk;
        it.tiles = (n_list >> (kt_log2 - 2)) + 1;  // of 4 n_list + 4 cells
    } else {
        if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
        if (warp == 0) {
            int64_t per;
            if (!share_of(sv, ws, kt_log2, blockIdx.x, gridDim.x, per, x, x1, it)) it.s = -1;
            if (lane == 0) {
                item_s = it;
                share_s[0] = per;
                share_s[1] = x;
                share_s[2] = x1;
            }
        }
        __syncthreads();
        it = item_s;
        if (it.s < 0) return;
        x = share_s[1];
        x1 = share_s[2];
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
            t0 = it.t0;
            len = it.len;
            cells = it.cells;
            tok0 = it.t * ws.rt;
            rows = min(ws.rt, len - tok0) * G;
            // the first token's position: cells behind it are not seen by every row
            pos0 = ws.causal ? cells - len + tok0 : cells - 1;
        }
        const bool starts = tile0 == 0, ends = tile1 == it.tiles;
        const bool fits = cells_fit(kv, cells);
        n_see = !fits ? 0 : (LIST ? 4 * n_list + 4 : item_cells(ws, len, cells, it.t));
        const int kv_head = (it.g << hpc_log2) + head;

        __syncthreads();  // the previous part's shared memory is free
        if (tid == 0) bad_s = odd_s = 0;
        // ---- the ring: a tile's cells (LIST: its list entries, a turn before) are looked up ahead of its copies.
        // p_next, entry_next: this lane's cell of the next tile to issue, and its page; blk_next: the list entry of
        // its cell of the tile after that
        const int my_key = lane < kKeys ? lane : 0;
        bool bad = false, odd = false, far = false;
        int32_t p_next = -1, entry_next = -1, blk_next = -1;
        auto look_page = [&](int p) {
            p_next = p;
            if (p >= 0) {
                const int64_t j = p >> kv.page_shift;
                entry_next = j < kv.ld_table ? kv.table[(int64_t)it.s * kv.ld_table + j] : -1;
            }
        };
        auto look_list = [&](int tile) {
            const int i = (tile << kt_log2) + part * kKeys + my_key;
            blk_next = tile < tile1 && (i >> 2) < n_list ? list[i >> 2] : -1;
        };
        // the cell of tile `tile`, whose entry is in blk_next; then the entry of the tile after it
        auto look_up = [&](int tile) {
            const int i = (tile << kt_log2) + part * kKeys + my_key;
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
        const uint8_t *const Ke = F16 ? kv.K_exp + kv_head : nullptr, *const Ve = F16 ? kv.V_exp + kv_head : nullptr;
        auto load_exps = [&](int32_t row, int i) {
            const uint64_t at = (uint64_t)(uint32_t)row * (uint32_t)kv.H_kv;
            pend_k[i] = row >= 0 ? Ke[at] : kExpBias;
            pend_v[i] = row >= 0 ? Ve[at] : kExpBias;
        };
        constexpr int kChunks = S::kRowBytes / 16, kAt = 32 / kChunks;
        const int cc = lane & (kChunks - 1), r0 = lane / kChunks;
        const unsigned char *const Kl = static_cast<const unsigned char *>(kv.K) + (int64_t)kv_head * S::kRowBytes + cc * 16;
        const unsigned char *const Vl = static_cast<const unsigned char *>(kv.V) + (int64_t)kv_head * S::kRowBytes + cc * 16;
        const uint32_t ldk_b = (uint32_t)(C == QSA_E2M1 ? kv.ld_k / 2 : kv.ld_k * (C == QSA_BF16 ? 2 : 1));
        const uint32_t ldv_b = (uint32_t)(C == QSA_E2M1 ? kv.ld_v / 2 : kv.ld_v * (C == QSA_BF16 ? 2 : 1));
        // (rows kAt apart, a multiple of eight but for bf16's two, lie on the same places of the swizzle)
        const uint32_t ring_u = smem_u32(ring), to_k = cell_off<C>(r0, cc);
        // scales of two cells (neighbours in a page): K's by the lower lanes, V's by the upper
        const int pair = lane & 15;
        const uint32_t to_s = 2 * S::kTile + (lane < 16 ? 0 : S::kScales) + pair * 16;
        const uint8_t *const Sl = C == QSA_E2M1 ? (lane < 16 ? kv.K_scale : kv.V_scale) + ((int64_t)kv_head << (kv.page_shift + 3)) : nullptr;
        auto issue = [&](int stage, int32_t row) {
            const uint32_t st = ring_u + stage * S::kStage;
#pragma unroll
            for (int i = 0; i < kKeys / kAt; ++i) {
                const int32_t rr = __shfl_sync(0xffffffffu, row, r0 + kAt * i);
                const int on = rr >= 0 ? 16 : 0;
                const uint32_t at = max(rr, 0), to = st + (kAt % 8 == 0 ? to_k + kAt * i * S::kRowBytes : cell_off<C>(r0 + kAt * i, cc));
                cp16<C>(to, Kl + (uint64_t)at * ldk_b, on);
                cp16<C>(to + S::kTile, Vl + (uint64_t)at * ldv_b, on);
            }
            if constexpr (C == QSA_E2M1) {
                const int32_t ra = __shfl_sync(0xffffffffu, row, 2 * pair), rb = __shfl_sync(0xffffffffu, row, 2 * pair + 1);
                const uint32_t at = max(ra, 0), off = at & ((1u << kv.page_shift) - 1);
                // scale_row's place: rows of a page head by head
                cp16<C>(st + to_s, Sl + (uint64_t)(at - off) * (8u * (uint32_t)kv.H_kv) + 8u * off, ra >= 0 ? (rb >= 0 ? 16 : 8) : 0);
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
            constexpr int E = S::kE;
            // unit u: block u mod NB of head u / NB; warp w takes units w, w + 4, ...: up to NB of them
            constexpr int kWords = sizeof(TQ) == 2 ? 16 : 32;
            const int units = hpc * NB;
            uint32_t raw[NB][kWords];
            uint32_t top = 0;  // the largest finite magnitude, by its bits
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int u = warp + kWarps * i, r = 8 * (u % NB) + g8, h = ((it.g << hpc_log2) + u / NB) * G;
                const int tk = LIST || r < G ? 0 : (int)((uint32_t)r / (uint32_t)G);
                const uint4 *const src = reinterpret_cast<const uint4 *>(
                    qp + (t0 + tok0 + tk) * ld_q + (int64_t)(h + r - tk * G) * kD + c4 * E);
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
            float mul = q_sign;
            if constexpr (F16) {
                // fp16 holds the queries once the rows' largest magnitude is below 2^8: one power of two for all
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int k = 0; k < kWords; ++k) {
                        const uint32_t a = (sizeof(TQ) == 2 ? raw[i][k] << 16 : raw[i][k]) & 0x7fffffffu;
                        const uint32_t b = sizeof(TQ) == 2 ? raw[i][k] & 0x7fff0000u : 0u;
                        top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
                    }
                top = __reduce_max_sync(0xffffffffu, top);
                if (lane == 0) top_s[warp] = top;
                __syncthreads();
                top = max(max(top_s[0], top_s[1]), max(top_s[2], top_s[3]));
                const int sh = top > 0u ? min(max(134 - (int)(top >> 23), -120), 100) : 0;
                q_back = two_to(-sh);
                mul = q_sign * two_to(sh);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int u = warp + kWarps * i;
                if (u >= units) break;
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
        __syncthreads();
        const float key_scale = scale_log2 * q_back;
        auto keep_exps = [&](int stage, int i) {
            const int ek = min(max(pend_k[i] - kExpBias, kExpMin), kExpMax);
            const int ev = min(max(pend_v[i] - kExpBias, kExpMin), kExpMax);
            far |= abs(ev) > (int)kFar;
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
                ms[n][e] = mx[n][e] = kUnset;
                l[n][e] = 0.0f;
            }
        bool wide = false;
        // where this thread's parts of a fragment lie: key rows f0 (+ 8, + 16 kg), values of cells va, vb (likewise)
        const int f0 = frag_cell<C>(g8), va = frag_cell<C>(2 * c4), vb = frag_cell<C>(2 * c4 + 1);
        const uint32_t at_k = cell_off<C>(f0, c4);

        int slot = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            cp_wait<kStages - 2>();
            __syncwarp();
            unsigned char *const sk = ring + slot * S::kStage, *const sv_ = sk + S::kTile;
            const float4 *const ex = exps + slot * 32;
            const int j0 = (tile << kt_log2) + part * kKeys;
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
                if constexpr (C == QSA_E2M1) {
                    uint4 kr[kGroups][2];
                    __half2 sc[kGroups][2];  // scales of the lane's two groups of a cell
#pragma unroll
                    for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            kr[kg][hf] = *reinterpret_cast<const uint4 *>(sk + at_k + (16 * kg + 8 * hf) * S::kRowBytes);
                            const uint32_t h = half_of_scales(*reinterpret_cast<const uint16_t *>(sk + 2 * S::kTile + f0 * 8 + 2 * c4 + (16 * kg + 8 * hf) * 8));
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
                // ---- log2 units (codes: with the exponent of the cell's values, x = logit + e), masked; d: above the
                // reference, which moves where it has to
                float inv_e[kGroups][2];  // 2^-e of this thread's cells
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        float2 f = make_float2(scale_log2, 0.0f);
                        if constexpr (F16) {
                            const float4 e4 = ex[16 * kg + 8 * hf + f0];
                            inv_e[kg][hf] = e4.z;
                            f = make_float2(e4.x, e4.y);
                        }
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            float2 y = make_float2(s[kg][n][2 * hf], s[kg][n][2 * hf + 1]);
                            y = F16 ? fma2(y, make_float2(f.x, f.x), make_float2(f.y, f.y)) : mul2(y, make_float2(f.x, f.x));
                            s[kg][n][2 * hf] = y.x;
                            s[kg][n][2 * hf + 1] = y.y;
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
                float d[kGroups][NB][4];
                bool move = false;
                auto above = [&]() {
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const float2 m2 = make_float2(-mx[n][0], -mx[n][1]);
                        float top = -INFINITY;
#pragma unroll
                        for (int kg = 0; kg < kGroups; ++kg)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const float2 y = add2(make_float2(s[kg][n][2 * hf], s[kg][n][2 * hf + 1]), m2);
                                d[kg][n][2 * hf] = y.x;
                                d[kg][n][2 * hf + 1] = y.y;
                                top = fmaxf(top, fmaxf(y.x, y.y));
                            }
                        move |= top > S::kMove;
                    }
                };
                above();
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
                    above();
                }
                // ---- weights and their product with the values, 16 cells at a time
#pragma unroll
                for (int kg = 0; kg < kGroups; ++kg) {
                    uint32_t p[NB][NT][2];
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        float w[2][2];  // [cell half][row]
                        float2 l2 = make_float2(l[n][0], l[n][1]);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            w[hf][0] = ex2_approx(d[kg][n][2 * hf]);
                            w[hf][1] = ex2_approx(d[kg][n][2 * hf + 1]);
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
                    if constexpr (F16) {
                        if (wide) {
#pragma unroll
                            for (int n = 0; n < NB; ++n)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    l[n][i & 1] += ex2_approx(s[kg][n][i] - ex[16 * kg + 8 * (i >> 1) + f0].y - ms[n][i & 1]);
                        }
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
                            v[hf][0] = *reinterpret_cast<const uint2 *>(sv_ + at_a + r * S::kRowBytes);
                            v[hf][1] = *reinterpret_cast<const uint2 *>(sv_ + at_b + r * S::kRowBytes);
                            const unsigned char *const sc = sk + 2 * S::kTile + S::kScales + r * 8 + g8;
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
                                v[hf][e] = *reinterpret_cast<const uint4 *>(sv_ + cell_off<C>(2 * c4 + e, g8) + (16 * kg + 8 * hf) * S::kRowBytes);
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
                if (mx[n][e] == kUnset) mx[n][e] = -INFINITY;
                if (!F16 || !wide) ms[n][e] = mx[n][e];
                if (ms[n][e] == kUnset) ms[n][e] = -INFINITY;
                float sum = l[n][e];
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
                if (g8 == 0) {
                    red_m[warp][8 * n + 2 * c4 + e] = ms[n][e];
                    red_l[warp][8 * n + 2 * c4 + e] = sum;
                }
            }
        __syncthreads();  // every warp is done with its ring
        if constexpr (!LIST) {
            if (starts && tid == 0) {
                // (as dense_join.cuh's note_split)
                const bool uncut = ends;
                if (!uncut || by_item) {
                    const int64_t last_cta = div_pos(item_end - 1, share_s[0]);
                    splits[by_item ? it.index : (int64_t)blockIdx.x] = {uncut ? -1 : it.s, it.g, it.t, (int32_t)blockIdx.x,
                                                                        (int32_t)(last_cta - blockIdx.x) + 1, {0, 0, 0}};
                }
            }
        }
        const bool whole = starts && ends;
        const bool nan_out = bad_s != 0 || !fits;
        const int rec_rows = kRows << hpc_log2, heads = G << hpc_log2;  // of a record: rows token by token
        float *const rec = LIST ? nullptr : partial + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * partial_floats(rec_rows, kD);
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
                    float m = -INFINITY;
                    for (int w = head; w < kWarps; w += hpc) m = fmaxf(m, red_m[w][r]);
                    const float u = m == -INFINITY ? 0.0f : m;
                    const float f = mx[n][e] == -INFINITY ? 0.0f : ex2_approx(mx[n][e] - u);
                    float *const dst = ob + (size_t)(warp * 8 * kTurn + r - 8 * n0) * kPitch;
#pragma unroll
                    for (int t = 0; t < 8; ++t)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) dst[frag_dim<C>(t, g8, hf)] = o[t][n][2 * hf + e] * f;
                }
            __syncthreads();
            for (int i = tid; i < (8 * kTurn * (kD / 4)) << hpc_log2; i += kThreads) {
                const int rl = (i / (kD / 4)) % (8 * kTurn), h = i / (kD / 4 * 8 * kTurn), r = 8 * n0 + rl, c = (i % (kD / 4)) * 4;
                if (r >= rows) continue;
                float m = -INFINITY, sum = 0.0f;
                for (int w = h; w < kWarps; w += hpc) m = fmaxf(m, red_m[w][r]);
                const float u = m == -INFINITY ? 0.0f : m;
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int w = h; w < kWarps; w += hpc) {
                    sum += red_m[w][r] == -INFINITY ? red_l[w][r] : red_l[w][r] * ex2_approx(red_m[w][r] - u);
                    const float4 y = *reinterpret_cast<const float4 *>(&ob[(size_t)(w * 8 * kTurn + rl) * kPitch + c]);
                    v[0] += y.x; v[1] += y.y; v[2] += y.z; v[3] += y.w;
                }
                if (!LIST && odd_s) {
                    const int to = min(n_see - 1, ws.causal ? pos0 + r / G : cells - 1);
                    for (int j = max(pos0 + 1, tile0 << kt_log2); j <= to && j < tile1 << kt_log2; ++j) {
                        const int64_t row = cell_row(kv, it.s, t0, j);
                        if (C == QSA_E2M1 && row >= 0 &&
                            scale_is_nan(kv.V_scale[scale_row(kv, row, (it.g << hpc_log2) + h) * 8 + (c >> 4)]))
                            v[0] = v[1] = v[2] = v[3] = NAN;
                    }
                }
                if (nan_out) sum = NAN;
                const int q_head = h * G + (LIST ? r : r % G);  // of the record's
                const int64_t at = (t0 + tok0 + (LIST ? 0 : r / G)) * H_q + it.g * heads + q_head;
                if (LIST ? ranks == 1 : whole) {
                    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                    TQ *const dst = out + at * kD + c;
                    if constexpr (sizeof(TQ) == 2)
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
                    else
                        *reinterpret_cast<float4 *>(dst) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                    if (c == 0 && lse) lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
                } else if constexpr (LIST) {
                    *reinterpret_cast<float4 *>(fin + q_head * kPitch + c) = make_float4(v[0], v[1], v[2], v[3]);
                    if (c == 0) {
                        fin[rec_rows * kPitch + q_head] = m;
                        fin[rec_rows * kPitch + rec_rows + q_head] = sum;
                    }
                } else {
                    const int rr = (r / G) * heads + q_head;
                    *reinterpret_cast<float4 *>(rec + 2 * rec_rows + (int64_t)rr * kD + c) = make_float4(v[0], v[1], v[2], v[3]);
                    if (c == 0) {
                        rec[rr] = m;
                        rec[rec_rows + rr] = sum;
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
                for (int i = (int)rank * kThreads + tid; i < heads * (kD / 4); i += (int)ranks * kThreads) {
                    const int r = i / (kD / 4), c = (i % (kD / 4)) * 4;
                    float m = -INFINITY, sum = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (uint32_t k = 0; k < ranks; ++k) m = fmaxf(m, load1(there(k, rec_rows * kPitch + r)));
                    const float u = m == -INFINITY ? 0.0f : m;
                    for (uint32_t k = 0; k < ranks; ++k) {
                        const float km = load1(there(k, rec_rows * kPitch + r)), kl = load1(there(k, rec_rows * kPitch + rec_rows + r));
                        const float f = km == -INFINITY ? 1.0f : exp2f(km - u);  // an unset side is zero or NaN
                        float4 y;
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                                     : "r"(there(k, r * kPitch + c))
                                     : "memory");
                        sum += kl * f;
                        v[0] += y.x * f; v[1] += y.y * f; v[2] += y.z * f; v[3] += y.w * f;
                    }
                    const int64_t at = tok * H_q + it.g * heads + r;
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
        x = it.start + tile1;
        if (x >= x1 || !item_after(sv, ws, kt_log2, it)) break;
    }
}

}  // namespace few
}  // namespace qsa
