// paged_four.cu -- attention of a few new tokens per sequence over a 4-bit paged cache.
//
// Mathematics and a warp's products: few_cells.cuh.
// Shape: persistent CTAs of four warps take equal shares of the list of (sequence, group of hpc KV heads, row tile)
// items.  Warp w takes head w mod hpc and part w / hpc of every tile's 4 / hpc parts of 32 cells, and runs a ring of
// stages of its own (cp.async, 4.6 KB each); with four heads (or a multiple) the warps of a CTA meet only where the
// queries are laid out.  A warp's 32 cells follow one another in a page of 32 cells or more, so their addresses are one
// product and additions.  An item's parts in several CTAs are joined by dense_join.cuh.
// TMA copies by one warp or four beside the computing ones were tried and were not faster: a tile is small, and a
// copying warp's instructions wait their turn behind those of the warps that compute.
#include "few_cells.cuh"

namespace qsa {
namespace few {

using Q4 = Cell<QSA_E2M1>;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = Q4::kKeys;

template <int NB, int NT>
struct Four {
    static constexpr int kCtas = NB == 4 || NB * NT == 4 ? 2 : 3;  // of an SM
    static constexpr int kStages = NB * NT == 2 ? 2 : 3;
};

// As dense.cuh's flattened list, made short: every row tile of a sequence counts the tiles of its whole context (turns
// behind what a row tile sees read nothing), so that a share is found with shifts and a few 32-bit divisions.  (The exact
// list took 11,000 to 24,000 cycles at 64 sequences, most of them fetching code that runs once.)  The row tiles of a few
// tokens see hardly less.  Those of fp32 prompts, which come here too, do: shares are uneven then, and 8,192 tokens over
// themselves (32 / 4 heads) take 5.5 ms where even ones would take 3.6 at the pace of 1,024 tokens over 8,192 cells (0.84).
struct Item {
    int32_t s, g, t;     // sequence, group of heads, row tile
    int32_t tiles;
    int32_t len, cells;  // of the sequence
    int32_t nt;          // its row tiles
    int32_t pad;
    int64_t t0;          // its first token
    int64_t start;       // the item's first place in the list
    int64_t index;       // its number
};

// A sequence's tokens, cells, tiles of an item and row tiles.
__device__ __forceinline__ void look_at(const SeqView &sv, const WorkShape &w, Item &it)
{
    seq_tokens(sv, it.s, it.t0, it.len);
    it.cells = seq_cells(sv, it.s, it.len);
    it.nt = it.len <= w.rt ? (it.len > 0) : (int)((uint32_t)(it.len + w.rt - 1) / (uint32_t)w.rt);
    it.tiles = it.cells > 0 && it.cells <= w.most ? (int)((uint32_t)(it.cells - 1) / (uint32_t)w.kt) + 1 : 1;
}

// The share of CTA `cta` of `ctas`: places [x0, x1) and the item at x0; false when there is none.  One warp calls it.
__device__ __forceinline__ bool share_of(const SeqView &sv, const WorkShape &w, int cta, int ctas, int64_t &per, int64_t &x0,
                                         int64_t &x1, Item &it)
{
    const int lane = threadIdx.x & 31;
    int64_t total = 0;
#pragma unroll 1
    for (int s = lane; s < sv.n_seq; s += 32) {
        Item i;
        i.s = s;
        look_at(sv, w, i);
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
        if (it.s < sv.n_seq) look_at(sv, w, it);
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
__device__ __forceinline__ bool item_after(const SeqView &sv, const WorkShape &w, Item &it)
{
    it.start += it.tiles;
    ++it.index;
    if (++it.t < it.nt) return true;
    it.t = 0;
    if (++it.g < w.H_kv) return true;
    it.g = 0;
    do {
        if (++it.s >= sv.n_seq) return false;
        look_at(sv, w, it);
    } while (it.nt == 0);
    return true;
}

// A CTA's share, part by part: an item and its tiles [tile0, tile1).
struct Walk {
    Item it;
    int64_t x1;
    int32_t tile0, tile1, n_see, n;  // n: number of the part
    __device__ __forceinline__ void set(const KvView &kv, const WorkShape &w, int64_t x)
    {
        tile0 = (int)(x - it.start);
        tile1 = (int)(min(it.start + it.tiles, x1) - it.start);
        n_see = cells_fit(kv, it.cells) ? item_cells(w, it.len, it.cells, it.t) : 0;
    }
    __device__ __forceinline__ bool next(const KvView &kv, const SeqView &sv, const WorkShape &w)
    {
        ++n;
        const int64_t x = it.start + tile1;
        if (x >= x1 || !item_after(sv, w, it)) return false;
        set(kv, w, x);
        return true;
    }
};

// The ring, then by head the queries; a head's results lie over the ring while the warps that share it are joined.
template <int NB, int NT>
__host__ __device__ constexpr size_t four_smem(int hpc)
{
    return (size_t)kWarps * Four<NB, NT>::kStages * (Q4::kStage + 512) + hpc * q_bytes<NB, NT>();
}

template <typename TQ, int NB, int NT>
__global__ void __launch_bounds__(kThreads, (Four<NB, NT>::kCtas))
paged_four_kernel(const KvView kv, const SeqView sv, const WorkShape ws, const TQ *__restrict__ q, int64_t ld_q, int H_q,
                  float scale_log2, float q_sign, TQ *__restrict__ out, float *__restrict__ lse, float *__restrict__ partial,
                  Split *__restrict__ splits, int by_item, int hpc_log2)
{
    constexpr int kRows = 8 * NB, kStages = Four<NB, NT>::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Walk walk_s, walks_s[kWarps];  // the first part; each warp's own
    __shared__ int64_t per_s;
    __shared__ int none_s, bad_s, odd_s[kWarps];  // number + 1 of the part that set it; odd_s: by head
    __shared__ __align__(16) float undo_s[kWarps][kRows];  // by head
    __shared__ float red_m[kWarps][kRows], red_l[kWarps][kRows];

    const int tid = threadIdx.x, lane = tid & 31, g8 = lane >> 2, c4 = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, as the compiler sees it
    const int hpc = 1 << hpc_log2, head = warp & (hpc - 1), part = warp >> hpc_log2, P = kWarps >> hpc_log2;
    unsigned char *const ring = smem + (size_t)warp * kStages * Q4::kStage;
    float4 *const exps = reinterpret_cast<float4 *>(smem + (size_t)kWarps * kStages * Q4::kStage) + warp * kStages * 32;
    uint4 *const q_all = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * kStages * (Q4::kStage + 512));
    const uint4 *const qf = q_all + head * (int)(q_bytes<NB, NT>() / 16);
    float *const fin = reinterpret_cast<float *>(smem);  // [head][row][kPitch]
    static_assert((size_t)2 * kRows * kPitch * 4 <= (size_t)kWarps * kStages * Q4::kStage, "two heads' results fit over the ring");

    pdl_wait();
    const TQ *qp = q;
    QSA_AFTER_WAIT(qp);
    pdl_trigger();
    if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
    if (warp == 0) {
        Walk w;
        int64_t per, x;
        w.n = 0;
        const bool some = share_of(sv, ws, blockIdx.x, gridDim.x, per, x, w.x1, w.it);
        if (some) w.set(kv, ws, x);
        if (lane == 0) {
            walk_s = w;
            per_s = per;
            none_s = !some;
            bad_s = 0;
        }
        if (lane < kWarps) odd_s[lane] = 0;
    }
    __syncthreads();
    if (none_s) return;
    // (the part is read where it lies: its fields would take the registers that the rows need)
    Walk &p = walks_s[warp];
    if (lane == 0) p = walk_s;
    __syncwarp();
    const int G = H_q / kv.H_kv, heads = G << hpc_log2, rec_rows = kRows << hpc_log2;
    const bool wide_pages = kv.page_shift >= 5;

    // ---- what a lane copies of a row: chunk cc of rows r0, r0 + 8, ...; scales of two cells, K's by the lower lanes
    const int cc = lane & 3, r0 = lane >> 2, pair = lane & 15;
    const uint32_t ldk_b = (uint32_t)(kv.ld_k / 2), ldv_b = (uint32_t)(kv.ld_v / 2);
    const uint32_t ring_u = smem_u32(ring), to_k = cell_off<QSA_E2M1>(r0, cc);
    const uint32_t to_s = 2 * Q4::kTile + (lane < 16 ? 0 : Q4::kScales) + pair * 16;
    for (;;) {
        const bool starts = p.tile0 == 0, ends = p.tile1 == p.it.tiles;
        const int tok0 = p.it.t * ws.rt, rows = min(ws.rt, p.it.len - tok0) * G, n_see = p.n_see, tile0 = p.tile0, tile1 = p.tile1;
        // the first token's position: cells behind it are not seen by every row
        const int pos0 = ws.causal ? p.it.cells - p.it.len + tok0 : p.it.cells - 1;
        const int kv_head = (p.it.g << hpc_log2) + head;
        const int32_t *const table = kv.table + (int64_t)p.it.s * kv.ld_table;
        const unsigned char *const Kl = static_cast<const unsigned char *>(kv.K) + (int64_t)kv_head * Q4::kRowBytes + cc * 16;
        const unsigned char *const Vl = static_cast<const unsigned char *>(kv.V) + (int64_t)kv_head * Q4::kRowBytes + cc * 16;
        const unsigned char *const Sl = (lane < 16 ? kv.K_scale : kv.V_scale) + ((int64_t)kv_head << (kv.page_shift + 3));
        const uint8_t *const Ke = kv.K_exp + kv_head, *const Ve = kv.V_exp + kv_head;
        if (p.n > 0) __syncthreads();  // the last part's queries and results are no longer read
        bool bad = false, far = false;
        uint8_t pend_k[kStages - 1], pend_v[kStages - 1];  // exponents of the next tiles, on their way
        // the next tile to issue: this lane's cell (wide pages: the warp's first), below 0: none, and its page; the cells
        // that are there
        int32_t c_next = -1, page_next = 0;
        int n_next = 0;
        auto look_up = [&](int tile) {
            const int c0 = tile * ws.kt + part * kKeys, c = wide_pages ? c0 : c0 + lane;
            n_next = tile < tile1 ? min(max(n_see - c0, 0), kKeys) : 0;
            c_next = tile < tile1 && c < n_see ? c : -1;
            if (c_next >= 0) {
                const int64_t j = c >> kv.page_shift;
                page_next = j < kv.ld_table ? table[j] : -1;
            }
        };
        auto issue = [&](int stage, int i) {
            const uint32_t st = ring_u + stage * Q4::kStage;
            int32_t row = -1;
            if (c_next >= 0) {
                if ((uint32_t)page_next >= (uint32_t)kv.n_pages) bad = true;
                else row = (page_next << kv.page_shift) | (c_next & ((1 << kv.page_shift) - 1));
            }
            const uint32_t page = 1u << kv.page_shift;
            int32_t mine;  // row of this lane's cell
            if (wide_pages) {
                const int n = row >= 0 ? n_next : 0;
                const uint32_t at = max(row, 0), off = at & (page - 1);
                const unsigned char *ks = Kl + (uint64_t)(at + r0) * ldk_b, *vs = Vl + (uint64_t)(at + r0) * ldv_b;
#pragma unroll
                for (int k = 0; k < kKeys / 8; ++k) {
                    const int on = r0 + 8 * k < n ? 16 : 0;
                    cp16<QSA_E2M1>(st + to_k + 8 * k * Q4::kRowBytes, ks, on);
                    cp16<QSA_E2M1>(st + Q4::kTile + to_k + 8 * k * Q4::kRowBytes, vs, on);
                    ks += 8 * ldk_b;
                    vs += 8 * ldv_b;
                }
                // scale_row's place: rows of a page head by head
                cp16<QSA_E2M1>(st + to_s, Sl + (uint64_t)(at - off) * (8u * (uint32_t)kv.H_kv) + 8u * off + pair * 16,
                               8 * min(max(n - 2 * pair, 0), 2));
                mine = lane < n ? row + lane : -1;
            } else {
#pragma unroll
                for (int k = 0; k < kKeys / 8; ++k) {
                    const int32_t rr = __shfl_sync(0xffffffffu, row, r0 + 8 * k);
                    const int on = rr >= 0 ? 16 : 0;
                    const uint32_t at = max(rr, 0);
                    cp16<QSA_E2M1>(st + to_k + 8 * k * Q4::kRowBytes, Kl + (uint64_t)at * ldk_b, on);
                    cp16<QSA_E2M1>(st + Q4::kTile + to_k + 8 * k * Q4::kRowBytes, Vl + (uint64_t)at * ldv_b, on);
                }
                const int32_t ra = __shfl_sync(0xffffffffu, row, 2 * pair), rb = __shfl_sync(0xffffffffu, row, 2 * pair + 1);
                const uint32_t at = max(ra, 0), off = at & (page - 1);
                cp16<QSA_E2M1>(st + to_s, Sl + (uint64_t)(at - off) * (8u * (uint32_t)kv.H_kv) + 8u * off, ra >= 0 ? (rb >= 0 ? 16 : 8) : 0);
                mine = row;
            }
            pend_k[i] = pend_v[i] = kExpBias;
            if (mine >= 0) {
                const uint64_t at = (uint64_t)(uint32_t)mine * (uint32_t)kv.H_kv;
                pend_k[i] = Ke[at];
                pend_v[i] = Ve[at];
            }
        };
        auto keep_exps = [&](int stage) {  // the next tile's
            const int ke = min(max((int)pend_k[0], kExpBias + kExpMin), kExpBias + kExpMax);
            const int ve = min(max((int)pend_v[0], kExpBias + kExpMin), kExpBias + kExpMax);
            far = far || __any_sync(0xffffffffu, abs(ve - kExpBias) > (int)kFar);
            exps[stage * 32 + lane] = make_float4(__int_as_float(ke << 23), (float)(ve - kExpBias), __int_as_float((254 - ve) << 23), 0.0f);
#pragma unroll
            for (int i = 0; i + 1 < kStages - 1; ++i) {
                pend_k[i] = pend_k[i + 1];
                pend_v[i] = pend_v[i + 1];
            }
        };
        look_up(tile0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (tile0 + i < tile1) issue(i, i);
            look_up(tile0 + i + 1);
            cp_commit();
        }
        stage_queries<QSA_E2M1, TQ, NB, NT, kWarps>(tid, qp + (p.it.t0 + tok0) * ld_q + (int64_t)p.it.g * heads * kD, ld_q, G, rows, hpc,
                                                    q_sign, scale_log2, q_all, undo_s[0]);
        __syncthreads();
        int last[NB][2];  // the last cell each row sees
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c4 + e;
                last[i][e] = r >= rows ? -1 : (ws.causal ? pos0 + (r < G ? 0 : (int)((uint32_t)r / (uint32_t)G)) : p.it.cells - 1);
            }
        Rows<QSA_E2M1, NB, NT> w;
        w.clear();
        int slot = 0;
        for (int tile = tile0; tile < tile1; ++tile) {
            cp_wait<kStages - 2>();
            keep_exps(slot);
            __syncwarp();
            unsigned char *const sk = ring + slot * Q4::kStage;
            const int j0 = tile * ws.kt + part * kKeys, nslot = slot == 0 ? kStages - 1 : slot - 1;
            const bool more = tile + kStages - 1 < tile1;
            // ---- issue the tile kStages - 1 ahead into the stage read in the last turn
            if (more) issue(nslot, kStages - 2);
            look_up(tile + kStages);
            cp_commit();
            if (j0 < n_see) {
                const bool edge = j0 + kKeys - 1 > pos0;  // some row may not see some cell
                if (edge) {
                    // values that not every row sees: NaN scales become zero here, and the values NaN at the end for the
                    // rows that see them (cells that are not there are zeros already)
                    if (j0 + lane > pos0) {
                        uint2 *const v = reinterpret_cast<uint2 *>(sk + 2 * Q4::kTile + Q4::kScales + lane * 8);
                        const uint2 x = *v;
                        const uint32_t m0 = __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu), m1 = __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        if (m0 | m1) {
                            *v = make_uint2(x.x & ~m0, x.y & ~m1);
                            *reinterpret_cast<volatile int *>(&odd_s[head]) = p.n + 1;
                        }
                    }
                    __syncwarp();
                }
                w.tile(sk, exps + slot * 32, qf, undo_s[head], scale_log2, far, edge, [&](int c, int i, int e) { return j0 + c > last[i][e]; });
            }
            __syncwarp();
            slot = slot == kStages - 1 ? 0 : slot + 1;
        }
        cp_wait<0>();
        if (__any_sync(0xffffffffu, bad) && lane == 0) *reinterpret_cast<volatile int *>(&bad_s) = p.n + 1;
        w.finish();
        if (g8 == 0) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    red_m[warp][8 * i + 2 * c4 + e] = w.ms[i][e];
                    red_l[warp][8 * i + 2 * c4 + e] = w.l[i][e];
                }
        }
        __syncthreads();  // every warp is done with its ring
        // ---- the warps of a head: to a common reference, then added up in turn; the last has the result
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * i + 2 * c4 + e;
                if (P > 1) {
                    float m = -INFINITY, sum = 0.0f;
                    for (int k = 0; k < P; ++k) m = fmaxf(m, red_m[(k << hpc_log2) + head][r]);
                    for (int k = 0; k < P; ++k) {
                        const float km = red_m[(k << hpc_log2) + head][r], kl = red_l[(k << hpc_log2) + head][r];
                        sum += km == -INFINITY ? kl : kl * ex2_approx(km - m);
                    }
                    w.l[i][e] = sum;
                    w.ms[i][e] = m;
                }
                const float f = w.mx[i][e] == -INFINITY ? 0.0f : ex2_approx(w.mx[i][e] - w.ms[i][e]);
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    w.o[t][i][e] *= f;
                    w.o[t][i][2 + e] *= f;
                }
            }
#pragma unroll 1
        for (int k = 0; k < P - 1; ++k) {
            if (part == k) {
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float4 *const to = reinterpret_cast<float4 *>(fin + (head * kRows + 8 * i + 2 * c4 + e) * kPitch + 16 * g8);
#pragma unroll
                        for (int t = 0; t < 8; t += 2) {
                            float4 y = make_float4(w.o[t][i][e], w.o[t][i][2 + e], w.o[t + 1][i][e], w.o[t + 1][i][2 + e]);
                            if (k > 0) {
                                const float4 z = to[t / 2];
                                y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
                            }
                            to[t / 2] = y;
                        }
                    }
            }
            __syncthreads();
        }
        if (starts && tid == 0 && (!ends || by_item)) {
            // (as dense_join.cuh's note_split)
            const int64_t last_cta = div_pos(p.it.start + p.it.tiles - 1, per_s);
            splits[by_item ? p.it.index : (int64_t)blockIdx.x] = {ends ? -1 : p.it.s, p.it.g, p.it.t, (int32_t)blockIdx.x,
                                                                  (int32_t)(last_cta - blockIdx.x) + 1, {0, 0, 0}};
        }
        if (part == P - 1) {
            const bool whole = starts && ends;
            const bool nan_out = !cells_fit(kv, p.it.cells) || *reinterpret_cast<volatile int *>(&bad_s) == p.n + 1;
            const bool odd = *reinterpret_cast<volatile int *>(&odd_s[head]) == p.n + 1;
            float *const rec = partial + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * partial_floats(rec_rows, kD);
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * i + 2 * c4 + e;
                    if (r >= rows) continue;
                    float v[16];
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        v[2 * t] = w.o[t][i][e];
                        v[2 * t + 1] = w.o[t][i][2 + e];
                    }
                    if (P > 1) {
                        const float4 *const from = reinterpret_cast<const float4 *>(fin + (head * kRows + r) * kPitch + 16 * g8);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float4 z = from[k];
                            v[4 * k] += z.x; v[4 * k + 1] += z.y; v[4 * k + 2] += z.z; v[4 * k + 3] += z.w;
                        }
                    }
                    if (odd) {
                        const int to = min(n_see - 1, last[i][e]);
                        bool nan = false;
                        for (int j = max(pos0 + 1, tile0 * ws.kt); j <= to && j < tile1 * ws.kt; ++j) {
                            const int64_t row = cell_row(kv, p.it.s, 0, j);
                            nan |= row >= 0 && scale_is_nan(kv.V_scale[scale_row(kv, row, kv_head) * 8 + g8]);
                        }
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = nan ? NAN : v[k];
                    }
                    const float m = w.ms[i][e], sum = nan_out ? NAN : w.l[i][e];
                    const int tk = r < G ? 0 : (int)((uint32_t)r / (uint32_t)G), q_head = head * G + r - tk * G;
                    if (whole) {
                        const int64_t at = (p.it.t0 + tok0 + tk) * H_q + (int64_t)p.it.g * heads + q_head;
                        const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                        TQ *const dst = out + at * kD + 16 * g8;
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] *= inv;
                        if constexpr (sizeof(TQ) == 2) {
                            uint4 *const d4 = reinterpret_cast<uint4 *>(dst);
                            d4[0] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                            d4[1] = make_uint4(pack_bf16(v[8], v[9]), pack_bf16(v[10], v[11]), pack_bf16(v[12], v[13]), pack_bf16(v[14], v[15]));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                reinterpret_cast<float4 *>(dst)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        }
                        if (g8 == 0 && lse) lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
                    } else {
                        const int rr = tk * heads + q_head;
                        float4 *const dst = reinterpret_cast<float4 *>(rec + 2 * rec_rows + (int64_t)rr * kD + 16 * g8);
#pragma unroll
                        for (int k = 0; k < 4; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        if (g8 == 0) {
                            rec[rr] = m;
                            rec[rec_rows + rr] = sum;
                        }
                    }
                }
        }
        Walk next = p;
        const bool more = next.next(kv, sv, ws);
        __syncwarp();
        if (lane == 0) p = next;
        __syncwarp();
        if (!more) break;
    }
}

// The join of items in many parts (few items, listed by number): a CTA for 32 values of a row.  A thread takes the
// reference and sum of one part, and eight lanes a part's values, eight parts in turn; all that is read at once, before
// the weights are known, so that what remains is a chain of four loads.  (One pass with a running maximum, a CTA a row, 456
// parts of one sequence: 33 us behind the attention's 37; weights first, then values by turns of eight: 15.)
constexpr int kJoinWarps = 16, kJoinSlices = 4;
constexpr int kJoinTurns = 8;  // parts of eight lanes
static_assert(3 * kTargetSMs <= 32 * kJoinWarps && 4 * kJoinWarps * kJoinTurns >= 3 * kTargetSMs, "every part has its thread");
template <typename TQ>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_many_kernel(const Split *__restrict__ splits, const float *__restrict__ partial, int rec_rows, const SeqView sv, int rt, int groups,
                 int heads, TQ *__restrict__ out, float *__restrict__ lse)
{
    __shared__ float weight[32 * kJoinWarps], red[2][kJoinWarps];
    __shared__ float4 red_o[kJoinWarps][8];
    pdl_wait();
    QSA_AFTER_WAIT(splits);
    QSA_AFTER_WAIT(partial);
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Split sp = splits[blockIdx.x];
    // fewer items than the host could tell have no entry
    int64_t items = 0;
    for (int s = lane; s < sv.n_seq; s += 32) {
        int64_t t0;
        int len;
        seq_tokens(sv, s, t0, len);
        items += (len + rt - 1) / rt;
    }
    if ((int64_t)blockIdx.x >= warp_sum_i64(items) * groups) return;
    if (sp.s < 0) return;
    int64_t t0;
    int len;
    seq_tokens(sv, sp.s, t0, len);
    const int r = blockIdx.y, tok = sp.t * rt + r / heads;
    if (r >= rt * heads || tok >= len) return;
    const int64_t rec = partial_floats(rec_rows, kD);
    auto part_of = [&](int k) { return partial + (2 * (int64_t)(sp.cta + k) + (k == 0 ? 1 : 0)) * rec; };
    const int n = min(sp.parts, 3 * kTargetSMs), first = tid >> 3, dim = 32 * blockIdx.z + 4 * (lane & 7);
    float4 y[kJoinTurns];
#pragma unroll
    for (int i = 0; i < kJoinTurns; ++i) {
        const int k = first + 4 * kJoinWarps * i;
        y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k < n) y[i] = *reinterpret_cast<const float4 *>(part_of(k) + 2 * rec_rows + (int64_t)r * kD + dim);
    }
    const float pm = tid < n ? part_of(tid)[r] : -INFINITY, pl = tid < n ? part_of(tid)[rec_rows + r] : 0.0f;
    float m = warp_max(pm);
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, red[0][w]);
    const float f = pm == -INFINITY ? 1.0f : exp2f(pm - (m == -INFINITY ? 0.0f : m));  // an unset side is zero or NaN
    weight[tid] = f;
    float l = pl * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kJoinTurns; ++i) {
        const float w = weight[first + 4 * kJoinWarps * i];
        o.x = fmaf(y[i].x, w, o.x);
        o.y = fmaf(y[i].y, w, o.y);
        o.z = fmaf(y[i].z, w, o.z);
        o.w = fmaf(y[i].w, w, o.w);
    }
#pragma unroll
    for (int k = 8; k < 32; k <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, k);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, k);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, k);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, k);
    }
    if (lane < 8) red_o[warp][lane] = o;
    __syncthreads();
    if (tid >= 8) return;
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += red[1][w];
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
        const float4 z = red_o[w][lane];
        o.x += z.x; o.y += z.y; o.z += z.z; o.w += z.w;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // a NaN sum stays NaN
    const int64_t at = (t0 + tok) * groups * heads + sp.g * heads + r % heads;
    TQ *const dst = out + at * kD + dim;
    if constexpr (sizeof(TQ) == 2)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    else
        *reinterpret_cast<float4 *>(dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (dim == 0 && lse) lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace few

namespace {

// KV heads of a CTA, as a power of two.
int heads_log2(int H_kv) { return H_kv % 4 == 0 ? 2 : (H_kv % 2 == 0 ? 1 : 0); }

template <typename TQ, int NB, int NT>
cudaError_t run(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    using F = few::Four<NB, NT>;
    const int G = a.H_q / a.kv.H_kv, hl = heads_log2(a.kv.H_kv), hpc = 1 << hl;
    DenseArgs b = a;  // as the work list and the join see it: hpc KV heads are one
    b.kv.H_kv >>= hl;
    const WorkShape ws = work_shape(b, 8 * NB / G, few::kKeys * (few::kWarps >> hl), 0);
    // the kernel takes a positive scale: a negative one turns the queries' signs, zero clears them
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr auto kernel = few::paged_four_kernel<TQ, NB, NT>;
    static_assert(F::kCtas * (few::four_smem<NB, NT>(4) + 2048) <= 228 * 1024, "shared memory of an SM");
    cudaError_t e = ensure_kernel_attrs<few::paged_four_kernel<TQ, NB, NT>>(few::four_smem<NB, NT>(4));
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count(), ctas = F::kCtas * (sms < kTargetSMs ? sms : kTargetSMs);
    Split *splits = static_cast<Split *>(workspace);
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + 3 * kTargetSMs * sizeof(Split));
    e = launch(kernel, dim3((unsigned)ctas), dim3(few::kThreads), few::four_smem<NB, NT>(hpc), st, 1, a.kv, a.sv, ws,
               static_cast<const TQ *>(a.q), a.ld_q, a.H_q, scale, q_sign, static_cast<TQ *>(a.out), a.lse, partial, splits,
               (int)join_by_item(b, ws.rt, ctas), hl);
    if (e != cudaSuccess) return e;
    // Few rows in many parts each: 200,000 cells in all, 32 / 4 heads, us here / by dense_join: a token of 1 sequence 50 / 73,
    // of 4 46 / 49, of 8 48 / 42, of 16 60 / 40; four tokens of 1 88 / 101, of 2 95 / 94, of 4 99 / 83.
    const int64_t items = ((a.sv.n_tok + ws.rt - 1) / ws.rt + a.sv.n_seq) * b.kv.H_kv;
    if (items * (8 * NB * hpc) <= 256)
        return launch(few::join_many_kernel<TQ>, dim3((unsigned)items, (unsigned)(8 * NB * hpc), few::kJoinSlices), dim3(32 * few::kJoinWarps), 0, st, 1, splits,
                      partial, 8 * NB * hpc, a.sv, ws.rt, b.kv.H_kv, G << hl, static_cast<TQ *>(a.out), a.lse);
    return launch_dense_join<TQ>(splits, partial, ctas, 8 * NB * hpc, ws.rt, b, st);
}

}  // namespace

bool few_four_ok(const DenseArgs &a, int64_t max_q)
{
    const int G = a.H_q / a.kv.H_kv;
    if (a.kv_dtype != QSA_E2M1 || a.d != few::kD || !a.kv.table || a.kv.ld_k % 32 || a.kv.ld_v % 32) return false;
    if (a.kv.ld_k > (1 << 28) || a.kv.ld_v > (1 << 28)) return false;  // strides in 32 bits
    // fp32 queries come here however many tokens they are; bf16 queries of more than 64 rows (tokens x heads of a KV
    // head) are the tcgen05 kernel's.  Here / there, us, groups of 8: 48 sequences of up to 16,384 cells with 4 tokens
    // 158 / 281, 8 tokens 260 / 286, 12 tokens 361 / 287; one of 61,789 with 4 tokens 50 / 68, 8 tokens 68 / 68, 16 tokens
    // 104 / 70; one of 4,000 32 / 37, 36 / 36, 48 / 38.  Groups of 4 cross at the same rows.
    return G <= (a.q_dtype == QSA_F32 ? 16 : 32) && (a.q_dtype == QSA_F32 || max_q * G <= 64);
}

size_t few_four_workspace()
{
    // records of 128 rows (four heads) at two CTAs per SM; of fewer rows three are no more
    return 3 * kTargetSMs * sizeof(Split) + (size_t)4 * kTargetSMs * partial_floats(128, few::kD) * sizeof(float);
}

cudaError_t launch_few_four(const DenseArgs &a, int64_t max_q, void *workspace, cudaStream_t st)
{
    const int64_t rows = max_q * (a.H_q / a.kv.H_kv);
    const int G = a.H_q / a.kv.H_kv;
    if (a.q_dtype == QSA_F32)
        return rows <= 8 ? run<float, 1, 2>(a, workspace, st) : run<float, 2, 2>(a, workspace, st);
    if (rows <= 8) return run<__nv_bfloat16, 1, 1>(a, workspace, st);
    if (rows <= 16 && G <= 16) return run<__nv_bfloat16, 2, 1>(a, workspace, st);
    return run<__nv_bfloat16, 4, 1>(a, workspace, st);
}

}  // namespace qsa
