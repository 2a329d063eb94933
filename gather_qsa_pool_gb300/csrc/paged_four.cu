// paged_four.cu -- attention of a few new tokens per sequence over a 4-bit paged cache.
//
// Mathematics and a warp's products: few_cells.cuh.
// Shape: persistent CTAs take equal shares of the list of (sequence, group of KV heads, row tile) items.  W warps
// compute, a head and 32 cells of a tile each (warp w: head w mod hpc, part w / hpc); four more copy: K's rows, V's
// rows (TMA boxes of two heads, PAIR; an odd number of heads: of one, x the cells of a page or tile), the scales (boxes
// of all heads where a page holds the tile), and the exponents (loads that run a tile ahead and leave as factors).
// They are bound by latency, some 200 cycles a TMA instruction: one warp for all took 2,400 cycles a tile with nothing
// computed beside it, as long as memory takes for three CTAs' tiles.  With the copies among the computing warps' own
// instructions (cp.async, look-ups, exponents) these were a quarter of all.  The list goes on across items: the next
// item's tiles are under way while an item's results are written.  An item's parts in several CTAs are joined by
// dense_join.cuh.
//
// Every mbarrier wait is bounded: after one gives up nothing new is issued, what was issued is waited for, and the
// rows not finished become NaN.
#include <algorithm>

#include "dense_tc.cuh"
#include "few_cells.cuh"

namespace qsa {
namespace few {

using Q4 = Cell<QSA_E2M1>;
constexpr int kKeys = Q4::kKeys;

// W: computing warps of a CTA.  kRegs, kCopyRegs: registers of the computing warpgroups' threads and of the copying
// one's, which share what the CTA was launched with.
template <int NB, int NT>
struct Four {
    static constexpr int W = NB == 4 ? 8 : 4;
    static constexpr int kCtas = NB == 4 ? 1 : (NB * NT == 1 ? 3 : 2);
    static constexpr int kStages = NB * NT == 2 ? 4 : 3;
    static constexpr int kThreads = 32 * (W + 4);
    static constexpr int kLaunchRegs = NB == 4 ? 168 : (kCtas == 3 ? 80 : 128);
    static constexpr int kCopyRegs = NB == 4 ? 56 : (kCtas == 3 ? 40 : 56);
    static constexpr int kRegs = ((W + 4) * kLaunchRegs - 4 * kCopyRegs) / W;
    static_assert(kRegs % 8 == 0 && kRegs * W + kCopyRegs * 4 <= kLaunchRegs * (W + 4), "the launch's registers");
    static constexpr uint32_t kStage = W * Q4::kStage;
};

// As dense.cuh's flattened list, made short: every row tile of a sequence counts the tiles of its whole context (the
// earlier ones of a few tokens see hardly less; turns behind what they see read nothing), so that a share is found
// with shifts and a few 32-bit divisions.  (The exact list took 11,000 to 24,000 cycles at 64 sequences, most of
// them fetching code that runs once.)
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
    __device__ __forceinline__ bool next(const KvView &kv, const SeqView &sv, const WorkShape &w, int kt_log2)
    {
        ++n;
        const int64_t x = it.start + tile1;
        if (x >= x1 || !item_after(sv, w, kt_log2, it)) return false;
        set(kv, w, x);
        return true;
    }
};

template <int NB, int NT>
struct FourBars {
    using F = Four<NB, NT>;
    uint64_t full[F::kStages], empty[F::kStages];
    int64_t per;
    Walk walk, walks[F::W + 4];        // the first part; each warp's own
    int32_t none;
    int32_t far[F::kStages];           // a stage has exponents beyond kFar
    int32_t bad[kSlots], odd[F::W];    // number + 1 of the part that set it; odd: by head
    uint32_t top[F::W];
    float red_m[F::W][8 * NB], red_l[F::W][8 * NB];
};

// hpc heads; a head's results pass through shared memory where it has several warps.
template <int NB, int NT>
__host__ __device__ constexpr size_t four_smem(int hpc)
{
    using F = Four<NB, NT>;
    return 1024 + (size_t)F::kStages * (F::kStage + F::W * 512) + hpc * q_bytes<NB, NT>() +
           (hpc < F::W ? (size_t)hpc * 8 * NB * kPitch * 4 : 0) + sizeof(FourBars<NB, NT>);
}
// Rows of K and V, and their scales.
struct FourMaps {
    CUtensorMap rows[2], scales[2];
};

template <typename TQ, int NB, int NT, bool PAIR>
__global__ void __launch_bounds__(Four<NB, NT>::kThreads, (Four<NB, NT>::kCtas))
paged_four_kernel(const __grid_constant__ FourMaps maps, const KvView kv, const SeqView sv,
                  const WorkShape ws, int box_log2, const TQ *__restrict__ q, int64_t ld_q, int H_q, float scale_log2, float q_sign,
                  TQ *__restrict__ out, float *__restrict__ lse, float *__restrict__ partial, Split *__restrict__ splits, int by_item,
                  int hpc_log2, int kt_log2, const WaitCtl wc)
{
    using F = Four<NB, NT>;
    constexpr int W = F::W, kStages = F::kStages, kRows = 8 * NB;
    constexpr uint32_t kV = W * Q4::kTile, kKs = 2 * kV, kVs = kKs + W * Q4::kScales;  // of a stage: K, V, scales by head
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char *const ring = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float4 *const exps_all = reinterpret_cast<float4 *>(ring + (size_t)kStages * F::kStage);  // [stage][warp][cell]
    uint4 *const q_all = reinterpret_cast<uint4 *>(exps_all + kStages * W * 32);
    const int hpc = 1 << hpc_log2;
    float *const fin = reinterpret_cast<float *>(q_all + hpc * (int)(q_bytes<NB, NT>() / 16));
    FourBars<NB, NT> &bars = *reinterpret_cast<FourBars<NB, NT> *>(fin + (hpc < W ? hpc * kRows * kPitch : 0));

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, as the compiler sees it
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.full[s], 4);
            mbar_init(&bars.empty[s], W);
        }
        for (int i = 0; i < kSlots; ++i) bars.bad[i] = 0;
        for (int i = 0; i < W; ++i) bars.odd[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    const TQ *qp = q;
    QSA_AFTER_WAIT(qp);
    pdl_trigger();
    if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
    if (warp == 0) {
        Walk w;
        int64_t per, x;
        w.n = 0;
        const bool some = share_of(sv, ws, kt_log2, blockIdx.x, gridDim.x, per, x, w.x1, w.it);
        if (some) w.set(kv, ws, x);
        if (lane == 0) {
            bars.walk = w;
            bars.per = per;
            bars.none = !some;
        }
    }
    __syncthreads();
    if (bars.none) return;
    bool ok = true;
    // (the part is read where it lies: its fields would take the registers that the rows need)
    Walk &p = bars.walks[warp];
    if (lane == 0) p = bars.walk;
    __syncwarp();
    auto next_part = [&]() -> bool {
        Walk next = p;
        const bool more = next.next(kv, sv, ws, kt_log2);
        __syncwarp();
        if (lane == 0) p = next;
        __syncwarp();
        return more;
    };
    if (warp >= W) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(F::kCopyRegs));
        const int P = W >> hpc_log2;                   // parts of a tile
        const int pieces = 1 << (kt_log2 - box_log2);  // boxes of a tile's cells
        const int role = warp - W;
        bool more = true;
        int tile = p.tile0;
        uint32_t n = 0;
        auto step = [&] {
            if (++tile >= p.tile1) {
                more = next_part();
                tile = p.tile0;
            }
        };
        auto page_of = [&](int c) -> int32_t {
            const int64_t j = c >> kv.page_shift;
            return j < kv.ld_table ? kv.table[(int64_t)p.it.s * kv.ld_table + j] : -1;
        };
        auto row_of = [&](int32_t page, int c) -> int32_t { return (page << kv.page_shift) | (c & ((1 << kv.page_shift) - 1)); };
        auto stage_free = [&](int st) -> bool {
            return n < (uint32_t)kStages || bar_wait_warp(&bars.empty[st], ((n / kStages) - 1) & 1u, wc.limit_ns);
        };
        if (role < 3) {
            // ---- K's rows, V's rows, scales: lane j has piece j's page, looked up a tile ahead
            const int wide = PAIR ? hpc / 2 : 1;         // row boxes of a piece
            const int s_heads = pieces == 1 ? hpc : 1;   // heads of a scale box
            const uint32_t piece_bytes = (uint32_t)((role == 2 ? 16 : 64) << hpc_log2) << box_log2;
            int32_t page[2], g[2], cell[2];  // of the next two tiles (g below 0: none; cell below 0: not there)
            auto look_up = [&](int i) {
                const int c = (tile << kt_log2) + (lane << box_log2);
                g[i] = more ? p.it.g : -1;
                cell[i] = more && lane < pieces && c < p.n_see ? c : -1;
                page[i] = cell[i] >= 0 ? page_of(c) : -1;
                if (more) step();
            };
            look_up(0);
            while (g[0] >= 0) {
                look_up(1);
                const int st = (int)(n % kStages);
                if (!stage_free(st)) {
                    ok = false;
                    break;
                }
                const int32_t mine = cell[0] >= 0 && (uint32_t)page[0] < (uint32_t)kv.n_pages ? row_of(page[0], cell[0]) : -1;
                const uint32_t here = __ballot_sync(0xffffffffu, mine >= 0);
                if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], (uint32_t)__popc(here) * piece_bytes);
                const uint32_t to = smem_u32(ring) + (uint32_t)st * F::kStage;
                const int first = g[0] << hpc_log2;
                __syncwarp();
#pragma unroll 1
                for (uint32_t todo = here; todo; todo &= todo - 1) {
                    const int j = __ffs(todo) - 1;
                    const int32_t r = __shfl_sync(0xffffffffu, mine, j);
                    // (one lane issues them all: with a box to a lane each takes its turn of a loop)
                    if (lane == 0) {
                        if (role < 2) {
                            constexpr uint32_t kPitchB = PAIR ? 128 : 64;
                            const uint32_t dst = to + (role ? kV : 0) + ((uint32_t)j << box_log2) * kPitchB;
                            for (int k = 0; k < wide; ++k)
                                tma_box(dst + ((uint32_t)k << kt_log2) * kPitchB, &maps.rows[role], first * 64 + k * (int)kPitchB, r, &bars.full[st]);
                        } else {
                            const int off = (r & ((1 << kv.page_shift) - 1)) * 8;
                            for (int h = 0; h < hpc; h += s_heads) {
                                const uint32_t dst = kKs + (((uint32_t)h << kt_log2) + ((uint32_t)j << box_log2)) * 8;
                                // (a tensor copy lands on 128 bytes: the 64 of a page of eight cells come by a plain one)
                                if (box_log2 == 3) {
                                    unsigned char *const sm = ring + (size_t)st * F::kStage + dst;
                                    const int64_t at = scale_row(kv, r, first + h) * 8;
                                    bulk_g2s(sm, kv.K_scale + at, 64u, &bars.full[st]);
                                    bulk_g2s(sm + (kVs - kKs), kv.V_scale + at, 64u, &bars.full[st]);
                                } else {
                                    tma_box3(to + dst, &maps.scales[0], off, first + h, r >> kv.page_shift, &bars.full[st]);
                                    tma_box3(to + dst + (kVs - kKs), &maps.scales[1], off, first + h, r >> kv.page_shift, &bars.full[st]);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
                page[0] = page[1];
                g[0] = g[1];
                cell[0] = cell[1];
                ++n;
            }
        } else {
            // ---- exponents: a lane's cell of each part.  A cell's exponents of all heads come by one load where they are
            // aligned.
            const bool words = ((reinterpret_cast<uintptr_t>(kv.K_exp) | reinterpret_cast<uintptr_t>(kv.V_exp)) & (uintptr_t)(hpc - 1)) == 0;
            for (; more; ++n) {
                const int st = (int)(n % kStages);
                const int c0 = (tile << kt_log2) + lane, n_see = p.n_see, g = p.it.g, part_n = p.n;
                uint32_t kx[W], vx[W];
                bool bad = false, far = false;
                int32_t row[W];
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (i >= P) break;
                    const int c = c0 + kKeys * i;
                    row[i] = c < n_see ? page_of(c) : -1;
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (i >= P) break;
                    const int c = c0 + kKeys * i;
                    const bool there = c < n_see && (uint32_t)row[i] < (uint32_t)kv.n_pages;
                    bad |= c < n_see && !there;
                    kx[i] = vx[i] = kExpBias * 0x01010101u;
                    if (there) {
                        const uint64_t at = (uint64_t)(uint32_t)row_of(row[i], c) * (uint32_t)kv.H_kv + (uint32_t)(g << hpc_log2);
                        const uint8_t *const ke = kv.K_exp + at, *const ve = kv.V_exp + at;
                        if (words && hpc == 4) {
                            kx[i] = *reinterpret_cast<const uint32_t *>(ke);
                            vx[i] = *reinterpret_cast<const uint32_t *>(ve);
                        } else if (words && hpc == 2) {
                            kx[i] = *reinterpret_cast<const uint16_t *>(ke);
                            vx[i] = *reinterpret_cast<const uint16_t *>(ve);
                        } else {
                            kx[i] = vx[i] = 0;
#pragma unroll 1
                            for (int h = hpc - 1; h >= 0; --h) {
                                kx[i] = kx[i] << 8 | ke[h];
                                vx[i] = vx[i] << 8 | ve[h];
                            }
                        }
                    }
                }
                step();
                if (!stage_free(st)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int i = 0; i < W; ++i) {
                    if (i >= P) break;
#pragma unroll 1
                    for (int h = 0; h < hpc; ++h) {
                        const uint32_t ke = min(max((kx[i] >> (8 * h)) & 255u, (uint32_t)(kExpBias + kExpMin)), (uint32_t)(kExpBias + kExpMax));
                        const uint32_t ve = min(max((vx[i] >> (8 * h)) & 255u, (uint32_t)(kExpBias + kExpMin)), (uint32_t)(kExpBias + kExpMax));
                        const float e = (float)((int)ve - kExpBias);
                        far |= fabsf(e) > kFar;
                        exps_all[(st * W + (i << hpc_log2) + h) * 32 + lane] =
                            make_float4(__uint_as_float(ke << 23), e, __uint_as_float((254u - ve) << 23), 0.0f);
                    }
                }
                far = __any_sync(0xffffffffu, far);
                bad = __any_sync(0xffffffffu, bad);
                if (lane == 0) {
                    *reinterpret_cast<volatile int32_t *>(&bars.far[st]) = far;
                    if (bad) *reinterpret_cast<volatile int32_t *>(&bars.bad[part_n % kSlots]) = part_n + 1;
                    mbar_arrive(&bars.full[st]);
                }
            }
        }
        // every copy issued has landed before the CTA may leave (a stage's earlier copies landed before it was used
        // again)
        for (uint32_t k = n > (uint32_t)kStages ? n - kStages : 0; k < n; ++k)
            if (!mbar_wait(&bars.full[k % kStages], (k / kStages) & 1u)) ok = false;
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(F::kRegs));
        // ---- a head's rows over a part's cells
        const int head = warp & (hpc - 1), part = warp >> hpc_log2, P = W >> hpc_log2, g8 = lane >> 2, c4 = lane & 3;
        const uint4 *const qf = q_all + head * (int)(q_bytes<NB, NT>() / 16);
        const int G = H_q / kv.H_kv, heads = G << hpc_log2, rec_rows = kRows << hpc_log2;
        uint32_t n = 0;
        for (;;) {
            const bool starts = p.tile0 == 0, ends = p.tile1 == p.it.tiles;
            const int tok0 = p.it.t * ws.rt, rows = min(ws.rt, p.it.len - tok0) * G, n_see = p.n_see, tile1 = p.tile1;
            // the first token's position: cells behind it are not seen by every row
            const int pos0 = ws.causal ? p.it.cells - p.it.len + tok0 : p.it.cells - 1;
            if (p.n > 0) named_sync<32 * W>(1);  // the last part's queries are no longer read
            const float q_back = stage_queries<QSA_E2M1, TQ, NB, NT, W>(
                tid, qp + (p.it.t0 + tok0) * ld_q + (int64_t)p.it.g * heads * kD, ld_q, G, rows, hpc, q_sign, q_all, bars.top,
                [] { named_sync<32 * W>(1); });
            named_sync<32 * W>(1);
            const float key_scale = scale_log2 * q_back;
            int last[NB][2];  // the last cell each row sees
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * i + 2 * c4 + e;
                    last[i][e] = r >= rows ? -1 : (ws.causal ? pos0 + (r < G ? 0 : (int)((uint32_t)r / (uint32_t)G)) : p.it.cells - 1);
                }
            Rows<QSA_E2M1, NB, NT, PAIR> w;
            w.clear();
            for (int tile = p.tile0; ok && tile < tile1; ++tile, ++n) {
                const int st = (int)(n % kStages);
                if (!bar_wait_warp(&bars.full[st], (n / kStages) & 1u, wc.limit_ns)) {
                    ok = false;
                    break;
                }
                unsigned char *const stage = ring + (size_t)st * F::kStage;
                unsigned char *const vs = stage + kVs + (head << kt_log2) * 8 + part * kKeys * 8;
                const int j0 = (tile << kt_log2) + part * kKeys;
                if (j0 < n_see) {
                    const bool edge = j0 + kKeys - 1 > pos0 || j0 + kKeys > n_see;  // some row may not see some cell
                    if (edge) {
                        // values that not every row sees: NaN scales become zero here and their values are NaN at the
                        // end for the rows that see them; what lies in the place of cells that are not there is zero
                        if (j0 + lane > pos0 || j0 + lane >= n_see) {
                            uint2 *const v = reinterpret_cast<uint2 *>(vs + lane * 8);
                            if (j0 + lane >= n_see) {
                                *v = make_uint2(0u, 0u);
                            } else {
                                const uint2 x = *v;
                                const uint32_t m0 = __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu), m1 = __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                if (m0 | m1) {
                                    *v = make_uint2(x.x & ~m0, x.y & ~m1);
                                    *reinterpret_cast<volatile int32_t *>(&bars.odd[head]) = p.n + 1;
                                }
                            }
                            // written by this thread (generic proxy), before copies (async proxy) come here again
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        }
                        __syncwarp();
                    }
                    // (PAIR: the heads of a pair share their rows)
                    const unsigned char *const sk = stage + (PAIR ? ((head >> 1) << kt_log2) * 128 + part * kKeys * 128 : ((head << kt_log2) + part * kKeys) * 64);
                    w.tile(sk, sk + kV, vs - W * Q4::kScales, vs, PAIR ? (head & 1) * 4 : 0, exps_all + (st * W + warp) * 32, qf, key_scale, *reinterpret_cast<volatile int32_t *>(&bars.far[st]) != 0, edge,
                           [&](int c, int i, int e) { return j0 + c > last[i][e] || j0 + c >= n_see; });
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.empty[st]);
            }
            w.finish();
            // ---- the warps of a head: to a common reference, then added up in turn; the last has the result
            if (P > 1) {
                if (g8 == 0) {
#pragma unroll
                    for (int i = 0; i < NB; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            bars.red_m[warp][8 * i + 2 * c4 + e] = w.ms[i][e];
                            bars.red_l[warp][8 * i + 2 * c4 + e] = w.l[i][e];
                        }
                }
                ok = !named_or<32 * W>(1, !ok);
            } else {
                ok = !named_or<32 * W>(1, !ok);
            }
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * i + 2 * c4 + e;
                    float m = w.ms[i][e];
                    for (int k = 0; P > 1 && k < P; ++k) m = fmaxf(m, bars.red_m[(k << hpc_log2) + head][r]);
                    if (P > 1) {
                        float sum = 0.0f;
                        for (int k = 0; k < P; ++k) {
                            const float km = bars.red_m[(k << hpc_log2) + head][r], kl = bars.red_l[(k << hpc_log2) + head][r];
                            sum += km == -INFINITY ? kl : kl * ex2_approx(km - m);
                        }
                        w.l[i][e] = sum;
                        w.ms[i][e] = m;
                    }
                    const float f = w.mx[i][e] == -INFINITY ? 0.0f : ex2_approx(w.mx[i][e] - m);
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
                named_sync<32 * W>(1);
            }
            const int64_t item_end = p.it.start + p.it.tiles;
            if (starts && tid == 0 && (!ends || by_item)) {
                // (as dense_join.cuh's note_split)
                const int64_t last_cta = div_pos(item_end - 1, bars.per);
                splits[by_item ? p.it.index : (int64_t)blockIdx.x] = {ends ? -1 : p.it.s, p.it.g, p.it.t, (int32_t)blockIdx.x,
                                                                      (int32_t)(last_cta - blockIdx.x) + 1, {0, 0, 0}};
            }
            if (part == P - 1) {
                const bool whole = starts && ends;
                const bool nan_out = !ok || !cells_fit(kv, p.it.cells) || *reinterpret_cast<volatile int32_t *>(&bars.bad[p.n % kSlots]) == p.n + 1;
                const bool odd = *reinterpret_cast<volatile int32_t *>(&bars.odd[head]) == p.n + 1;
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
                            for (int j = max(pos0 + 1, p.tile0 << kt_log2); j <= to && j < p.tile1 << kt_log2; ++j) {
                                const int64_t row = cell_row(kv, p.it.s, 0, j);
                                nan |= row >= 0 && scale_is_nan(kv.V_scale[scale_row(kv, row, (p.it.g << hpc_log2) + head) * 8 + g8]);
                            }
                            if (nan) v[0] = NAN;
#pragma unroll
                            for (int k = 1; k < 16; ++k) v[k] = nan ? NAN : v[k];
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
            if (!next_part()) break;
        }
    }
    if (!ok) report_timeout(wc);
}

}  // namespace few

namespace {

// KV heads of a CTA, as a power of two.
int heads_log2(int H_kv) { return H_kv % 4 == 0 ? 2 : (H_kv % 2 == 0 ? 1 : 0); }

template <int NB, int NT>
constexpr size_t most_smem()
{
    return std::max({few::four_smem<NB, NT>(1), few::four_smem<NB, NT>(2), few::four_smem<NB, NT>(4)});
}
static_assert(most_smem<4, 1>() <= 227 * 1024 && 2 * (most_smem<2, 2>() + 1024) <= 228 * 1024 &&
                  2 * (most_smem<2, 1>() + 1024) <= 228 * 1024 && 3 * (most_smem<1, 1>() + 1024) <= 228 * 1024,
              "shared memory of an SM");

// Rows of H_kv heads in boxes of one head's or a pair's bytes x box_rows rows, and scales in boxes of s_heads heads x
// box_rows cells of a page.
bool make_maps(few::FourMaps &m, const KvView &kv, int64_t pool_rows, bool pair, int box_rows, int s_heads)
{
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t page = (cuuint64_t)1 << kv.page_shift;
    for (int v = 0; v < 2; ++v) {
        const cuuint64_t dims[2] = {(cuuint64_t)kv.H_kv * 64, (cuuint64_t)pool_rows};
        const cuuint64_t strides[1] = {(cuuint64_t)(v ? kv.ld_v : kv.ld_k) / 2};
        const cuuint32_t box[2] = {pair ? 128u : 64u, (cuuint32_t)box_rows}, ones[3] = {1, 1, 1};
        if (fn(&m.rows[v], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(v ? kv.V : kv.K), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, pair ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
        const cuuint64_t s_dims[3] = {page * 8, (cuuint64_t)kv.H_kv, (cuuint64_t)kv.n_pages};
        const cuuint64_t s_strides[2] = {page * 8, page * 8 * (cuuint64_t)kv.H_kv};
        const cuuint32_t s_box[3] = {(cuuint32_t)box_rows * 8, (cuuint32_t)s_heads, 1};
        if (fn(&m.scales[v], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(v ? kv.V_scale : kv.K_scale), s_dims, s_strides, s_box,
               ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

template <typename TQ, int NB, int NT, bool PAIR>
qsa_status run(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    using F = few::Four<NB, NT>;
    const int G = a.H_q / a.kv.H_kv, hl = heads_log2(a.kv.H_kv), hpc = 1 << hl;
    DenseArgs b = a;  // as the work list and the join see it: hpc KV heads are one
    b.kv.H_kv >>= hl;
    const int kt_log2 = (F::W == 8 ? 8 : 7) - hl;
    const WorkShape ws = work_shape(b, 8 * NB / G, 1 << kt_log2, 0);
    // (a box of scales is 256 bytes wide at most)
    const int box_log2 = std::min({kt_log2, (int)a.kv.page_shift, 5});
    few::FourMaps maps;
    if (!make_maps(maps, a.kv, a.pool_rows, PAIR, 1 << box_log2, box_log2 == kt_log2 ? hpc : 1)) return QSA_ERR_CUDA;
    // the kernel takes a positive scale: a negative one turns the queries' signs, zero clears them
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr auto kernel = few::paged_four_kernel<TQ, NB, NT, PAIR>;
    if (ensure_kernel_attrs<few::paged_four_kernel<TQ, NB, NT, PAIR>>(most_smem<NB, NT>()) != cudaSuccess) return QSA_ERR_CUDA;
    const int sms = device_sm_count(), ctas = F::kCtas * (sms < kTargetSMs ? sms : kTargetSMs);
    Split *splits = static_cast<Split *>(workspace);
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + 3 * kTargetSMs * sizeof(Split));
    cudaError_t e = launch(kernel, dim3((unsigned)ctas), dim3(F::kThreads), few::four_smem<NB, NT>(hpc), st, 1, maps, a.kv, a.sv, ws, box_log2,
                           static_cast<const TQ *>(a.q), a.ld_q, a.H_q, scale, q_sign, static_cast<TQ *>(a.out), a.lse, partial, splits,
                           (int)join_by_item(b, ws.rt, ctas), hl, kt_log2, current_wait_ctl());
    if (e == cudaSuccess) e = launch_dense_join<TQ>(splits, partial, ctas, 8 * NB * hpc, ws.rt, b, st);
    return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

template <typename TQ, int NB, int NT>
qsa_status run_pair(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    return a.kv.H_kv % 2 == 0 ? run<TQ, NB, NT, true>(a, workspace, st) : run<TQ, NB, NT, false>(a, workspace, st);
}

}  // namespace

bool few_four_ok(const DenseArgs &a, int64_t max_q)
{
    const int G = a.H_q / a.kv.H_kv;
    if (a.kv_dtype != QSA_E2M1 || a.d != few::kD || !a.kv.table || a.kv.ld_k % 32 || a.kv.ld_v % 32) return false;
    // (a TMA map's strides are multiples of 16 bytes, and below 2^40)
    if (a.kv.ld_k > kMaxStride || a.kv.ld_v > kMaxStride || a.pool_rows <= 0 || a.pool_rows > 0x7fffffffLL) return false;
    // fp32 queries come here however many tokens they are; bf16 queries of more rows are the tcgen05 kernel's
    return G <= (a.q_dtype == QSA_F32 ? 16 : 32) && (a.q_dtype == QSA_F32 || max_q * G <= 64);
}

size_t few_four_workspace()
{
    // records of 32 rows (four heads) at three CTAs per SM, 64 at two, 128 at one
    return 3 * kTargetSMs * sizeof(Split) + (size_t)2 * kTargetSMs * 128 * (few::kD + 2) * sizeof(float);
}

qsa_status launch_few_four(const DenseArgs &a, int64_t max_q, void *workspace, cudaStream_t st)
{
    const int64_t rows = max_q * (a.H_q / a.kv.H_kv);
    const int G = a.H_q / a.kv.H_kv;
    if (a.q_dtype == QSA_F32)
        return rows <= 8 ? run_pair<float, 1, 2>(a, workspace, st) : run_pair<float, 2, 2>(a, workspace, st);
    if (rows <= 8) return run_pair<__nv_bfloat16, 1, 1>(a, workspace, st);
    if (rows <= 16 && G <= 16) return run_pair<__nv_bfloat16, 2, 1>(a, workspace, st);
    return run_pair<__nv_bfloat16, 4, 1>(a, workspace, st);
}

}  // namespace qsa
