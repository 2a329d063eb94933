// dense_attn_tc.cu -- attention of many query rows over every visible cell on the tcgen05 tensor
// cores: whole packed prompts, and chunks of new tokens over a paged cache.
//
// Mathematics: as dense_attn.cu; one pass over the cells with a running reference m and sum l
// per row, o += P V in tensor memory.  m moves (and o is rescaled) only when a tile's maximum
// passes it by more than 2^8, so almost no tile rescales.
//
// Shape: one persistent CTA per SM takes an equal share of the flattened list of (sequence, KV
// head, row tile) items in tiles of 128 cells (dense.cuh).  A row tile is two groups of 128 rows
// (query tokens x heads of one KV head, so the heads of a group read each K and V tile once).
// Warps 0-15 are the softmax: eight per group, each row shared by two threads that take 64 cells
// each (four warps per scheduler: with one thread per row, 128 logits in registers and half the
// warps, the chain logits -> maximum -> exponentials -> weights left the tensor cores idle for
// half the time).  Warp 16 issues the MMAs; warp 17 stages queries, K and V tiles by TMA (one box
// per page, 128-byte swizzle), K and V into a ring of 32 KB stages; warps 18 and 19 see to the
// tiles where some row does not see some cell (e4m3 and e2m1 cells: six warps that also turn codes
// into bf16).
//   tensor memory (512 columns): S of group A, S of group B (128 fp32 columns each; a row's
//   weights P overwrite its own S as bf16, each thread's 64 over its own logits), O of A and of B
//   (128 each).
// Per tile the tensor cores run O_A += P_A V, S_A = Q_A K', O_B += P_B V, S_B = Q_B K' (K' the
// next tile's keys): while one group's weights are computed the other group's products run.
// One thread issues them all, in the order in which they use S and P.
//
// Parts of an item in several CTAs are joined by dense_join (dense_join.cuh).  Every mbarrier
// wait is bounded: after one gives up, nothing new is issued, what was issued is waited for, the
// rows not finished become NaN and the tensor memory is returned.
#include "dense_join.cuh"
#include "dense_tc.cuh"

namespace qsa {
namespace {

constexpr int kM = 128;                  // rows of a group
constexpr int kSoftWarps = 16, kMmaWarp = 16, kLoadWarp = 17, kAuxWarp = 18;
constexpr int kOver = 4;                 // an item's fixed cost in tiles
constexpr uint32_t kTmemCols = 512;

__host__ __device__ constexpr uint32_t col_s(int g) { return g ? 128u : 0u; }
__host__ __device__ constexpr uint32_t col_o(int g) { return g ? 384u : 256u; }

// What differs between caches.  bf16: five stages, two warps for the tiles with a causal edge.
// e4m3: four stages of bf16 filled by six warps from two raw 16 KB tiles.
// Registers: 640 x 96 at launch = 512 x 104 + 128 x 64; 768 x 80 = 512 x 88 + 256 x 64 (a chunk of
// 1,024 tokens over 61,789 e4m3 cells 1,253 us, bound by the conversion; 1,355 with 96 and 48).
template <bool E8>
struct Cfg {
    static constexpr int kStages = E8 ? 4 : 5;
    static constexpr int kAuxWarps = E8 ? 6 : 2;
    static constexpr int kThreads = 32 * (kAuxWarp + kAuxWarps);
};
constexpr int kAuxBar = 9;                // their named barriers: 9, 10
constexpr int kSoftBar = 11;              // the softmax warps'

template <bool E8>
struct Bars {
    uint64_t full[Cfg<E8>::kStages], empty[Cfg<E8>::kStages];
    uint64_t raw[E8 ? 1 : Cfg<E8>::kStages];         // bf16: copies of a stage with an edge
    uint64_t raw_full[2], raw_empty[2];              // e4m3: raw tiles
    uint64_t s_full[2], p_full[2], o_full[2], q_full[2], q_free[2], drain;
    uint32_t tmem, pad;
    int32_t odd[kSlots], bad[kSlots];  // number + 1 of the part that set it
    uint8_t exps[2][2][E8 ? kN : 1];   // e4m3: exponents of the cells of K and V tiles, two turns
    float row[2][kM];                  // exchanged by the two threads of a row
    Parts part[2];                     // the softmax warps' part, and the next
    int64_t per;                       // places of a CTA
};

template <bool E8>
__host__ __device__ constexpr size_t tc_smem()
{
    return 1024 + 2 * kTileB + (size_t)Cfg<E8>::kStages * kTileB + (E8 ? 2 * kRawTile : 0) + sizeof(Bars<E8>);
}
static_assert(tc_smem<false>() <= 227 * 1024 && tc_smem<true>() <= 227 * 1024, "shared memory of one CTA");

// E8: cells of codes; E4: of 4-bit codes.
template <bool E8, bool E4 = false>
__global__ void __launch_bounds__(Cfg<E8>::kThreads, 1)
dense_tc_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                const __grid_constant__ CUtensorMap mapV, const KvView kv, const SeqView sv,
                const WorkShape ws, int box_rows, int H_q, float scale_log2,
                __nv_bfloat16 *__restrict__ out, float *__restrict__ lse, float *__restrict__ partial, Split *__restrict__ splits,
                int by_item, int whole_items, const WaitCtl wc)
{
    constexpr int kStages = Cfg<E8>::kStages, kAuxWarps = Cfg<E8>::kAuxWarps;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char *sQ = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);  // [group][dim half]
    unsigned char *ring = sQ + 2 * kTileB;
    unsigned char *raw_tiles = ring + (size_t)kStages * kTileB;  // e4m3: two
    Bars<E8> &bars = *reinterpret_cast<Bars<E8> *>(raw_tiles + (E8 ? 2 * kRawTile : 0));

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, as the compiler sees it
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.full[s], E8 ? kTeamWarps : kAuxWarps);
            mbar_init(&bars.empty[s], 1);
            if (!E8) mbar_init(&bars.raw[s], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bars.s_full[g], 1);
            mbar_init(&bars.p_full[g], kSoftWarps / 2);
            mbar_init(&bars.o_full[g], 1);
            mbar_init(&bars.q_full[g], 1);
            mbar_init(&bars.q_free[g], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bars.raw_full[s], 1);
            mbar_init(&bars.raw_empty[s], kTeamWarps);
        }
        mbar_init(&bars.drain, 1);
        for (int i = 0; i < kSlots; ++i) bars.odd[i] = bars.bad[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();

    Parts p;
    int64_t per;
    p.n = 0;
    if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
    if (whole_items) {
        if (!work_item(sv, ws, blockIdx.x, gridDim.x, per, p.x, p.x1, p.it)) return;
    } else if (!work_share(sv, ws, blockIdx.x, gridDim.x, per, p.x, p.x1, p.it)) {
        return;
    }
    p.set(kv, sv, ws);
    if (p.tile1 <= p.tile0) {  // only places without a tile
        --p.n;
        if (!p.next(kv, sv, ws)) return;
    }

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        bars.part[0] = p;
        bars.per = per;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = bars.tmem;
    const int G = H_q / kv.H_kv;
    const int rt2 = ws.rt / 2;  // tokens of a group
    bool ok = true;
    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == kMmaWarp) {
            // ---- MMA issue (all lanes walk, one issues)
            const uint32_t lead = elect_leader();
            constexpr uint32_t id_s = idesc_m128(kN, false), id_o = idesc_m128(kD, true);
            const uint64_t dk0 = desc_kmajor_sw128(smem_u32(ring));
            const uint64_t dv0 = desc_mnmajor_sw128(smem_u32(ring), kHalf);
            const uint64_t dq0 = desc_kmajor_sw128(smem_u32(sQ));
            // a stage, dim half or k step moves only the descriptors' start address (16-byte
            // units, below 2^14: the add does not carry out of the field)
            auto mma_s = [&](int g, int st) {
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint32_t off = ((uint32_t)(k >> 2) * kHalf + (uint32_t)(k & 3) * 32) >> 4;
                    umma_m128_ss_lead(tmem + col_s(g), dq0 + (((uint32_t)g * kTileB) >> 4) + off,
                                 dk0 + (((uint32_t)st * kTileB) >> 4) + off, id_s, k ? 1u : 0u, lead);
                }
            };
            auto mma_o = [&](int g, int st, bool first) {
#pragma unroll
                for (int k = 0; k < kN / 16; ++k)
                    umma_m128_ta_lead(tmem + col_o(g), tmem + col_s(g) + (uint32_t)(k >> 2) * 64 + (uint32_t)(k & 3) * 8,
                                 dv0 + (((uint32_t)st * kTileB + (uint32_t)k * 2048) >> 4), id_o,
                                 (!first || k) ? 1u : 0u, lead);
            };
            uint32_t n = 0, np[2] = {0, 0}, nq[2] = {0, 0};  // stages, weights, queries so far
            auto stage_ready = [&](uint32_t i) {
                return bar_wait(&bars.full[i % kStages], (i / kStages) & 1u, wc.limit_ns);
            };
            do {
                const int tiles = p.tile1 - p.tile0;
                const bool two = p.toks > rt2;  // group B has rows
                ok = stage_ready(n) && bar_wait(&bars.q_full[0], nq[0]++ & 1u, wc.limit_ns);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                mma_s(0, (int)(n % kStages));
                umma_commit_lead(&bars.s_full[0], lead);
                if (tiles == 1) umma_commit_lead(&bars.q_free[0], lead);
                if (two) {
                    ok = bar_wait(&bars.q_full[1], nq[1]++ & 1u, wc.limit_ns);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    mma_s(1, (int)(n % kStages));
                    umma_commit_lead(&bars.s_full[1], lead);
                    if (tiles == 1) umma_commit_lead(&bars.q_free[1], lead);
                }
                umma_commit_lead(&bars.empty[n % kStages], lead);
                for (int t = 0; t < tiles; ++t) {
                    const uint32_t iv = n + 2 * (uint32_t)t + 1, ik = iv + 1;
                    const bool more = t + 1 < tiles, last_s = t + 2 == tiles;
                    ok = stage_ready(iv) && bar_wait(&bars.p_full[0], np[0]++ & 1u, wc.limit_ns);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    mma_o(0, (int)(iv % kStages), t == 0);
                    if (more) {
                        ok = stage_ready(ik);
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        mma_s(0, (int)(ik % kStages));
                        umma_commit_lead(&bars.s_full[0], lead);
                        if (last_s) umma_commit_lead(&bars.q_free[0], lead);
                    } else {
                        umma_commit_lead(&bars.o_full[0], lead);
                    }
                    if (two) {
                        ok = bar_wait(&bars.p_full[1], np[1]++ & 1u, wc.limit_ns);
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        mma_o(1, (int)(iv % kStages), t == 0);
                    }
                    umma_commit_lead(&bars.empty[iv % kStages], lead);
                    if (two && more) {
                        mma_s(1, (int)(ik % kStages));
                        umma_commit_lead(&bars.s_full[1], lead);
                        if (last_s) umma_commit_lead(&bars.q_free[1], lead);
                    } else if (two) {
                        umma_commit_lead(&bars.o_full[1], lead);
                    }
                    if (more) umma_commit_lead(&bars.empty[ik % kStages], lead);
                }
                n += 2 * (uint32_t)tiles;
            } while (ok && p.next(kv, sv, ws));
            // every MMA issued has completed before the tensor memory is freed
            umma_commit_lead(&bars.drain, lead);
            if (!mbar_wait(&bars.drain, 0)) ok = false;
        } else if (warp == kLoadWarp) {
            // ---- queries, K and V tiles: box b of a tile is box_rows cells, by lane b
            const int boxes = kN / box_rows;
            uint32_t n = 0, nq[2] = {0, 0};
            uint32_t edge_last = 0, raw_phase = 0, used = 0;  // bits by stage
            do {
                // (a tile's pages are looked up two tiles ahead: nothing waits for them)
                PageAhead ahead[2];
                auto look = [&](int t) {
                    PageAhead a;
                    a.load(kv, p, t < p.tile1 && lane < boxes, (int64_t)t * kN + lane * box_rows);
                    return a;
                };
                ahead[0] = look(p.tile0);
                ahead[1] = look(p.tile0 + 1);
                for (int t = p.tile0; ok && t < p.tile1; ++t) {
                    const int row = ahead[0].row(kv, p);
                    ahead[0] = ahead[1];
                    ahead[1] = look(t + 2);
                    const uint32_t go = __ballot_sync(0xffffffffu, row >= 0);
                    if (__any_sync(0xffffffffu, row == -1) && lane == 0)
                        *reinterpret_cast<volatile int32_t *>(&bars.bad[p.n % kSlots]) = p.n + 1;
                    for (int half = 0; ok && half < 2; ++half) {  // K, then V
                        const CUtensorMap *map = half ? &mapV : &mapK;
                        if constexpr (E8) {
                            const int s = (int)(n & 1u);
                            if (n >= 2 &&
                                !bar_wait_warp(&bars.raw_empty[s], ((n >> 1) - 1) & 1u, wc.limit_ns)) {
                                ok = false;
                                break;
                            }
                            if (lane == 0)
                                mbar_arrive_expect_tx(&bars.raw_full[s],
                                                      (uint32_t)__popc(go) * (uint32_t)box_rows * (E4 ? 72u : 128u));
                            ++n;
                            __syncwarp();
                            if (E4 && row >= 0) {
                                // codes, and behind the tile's the scales
                                unsigned char *const to = raw_tiles + (size_t)s * kRawTile;
                                tma_box(smem_u32(to) + (uint32_t)(lane * box_rows) * 64, map, p.it.g * (kD / 2), row,
                                        &bars.raw_full[s]);
                                bulk_g2s(to + kN * 64 + lane * box_rows * 8,
                                         (half ? kv.V_scale : kv.K_scale) + scale_row(kv, row, p.it.g) * 8,
                                         (uint32_t)box_rows * 8u, &bars.raw_full[s]);
                            } else if (row >= 0) {
                                tma_box(smem_u32(raw_tiles) + (uint32_t)s * kRawTile +
                                            (uint32_t)(lane * box_rows) * 128,
                                        map, p.it.g * kD, row, &bars.raw_full[s]);
                            }
                        } else {
                            const int s = (int)(n % kStages);
                            if (n >= kStages &&
                                !bar_wait_warp(&bars.empty[s], ((n / kStages) - 1) & 1u, wc.limit_ns)) {
                                ok = false;
                                break;
                            }
                            const bool edge = half == 1 && p.edge(t);
                            uint64_t *bar = edge ? &bars.raw[s] : &bars.full[s];
                            if (lane == 0) {
                                mbar_arrive_expect_tx(bar, (uint32_t)__popc(go) * (uint32_t)box_rows * 256u);
                                if (!edge) mbar_arrive_n(bar, kAuxWarps - 1);
                            }
                            used |= 1u << s;
                            edge_last = edge ? edge_last | (1u << s) : edge_last & ~(1u << s);
                            if (edge) raw_phase ^= 1u << s;
                            ++n;
                            __syncwarp();
                            if (row >= 0) {
                                const uint32_t dst =
                                    smem_u32(ring) + (uint32_t)s * kTileB + (uint32_t)(lane * box_rows) * 128;
                                tma_box(dst, map, p.it.g * kD, row, bar);
                                tma_box(dst + kHalf, map, p.it.g * kD + 64, row, bar);
                            }
                        }
                        if (half == 0 && t == p.tile0) {
                            // this part's queries, once the last part's logits are done with theirs
                            for (int g = 0; g < (p.toks > rt2 ? 2 : 1); ++g) {
                                if (nq[g] > 0 && !bar_wait_warp(&bars.q_free[g], (nq[g] - 1) & 1u, wc.limit_ns)) {
                                    ok = false;
                                    break;
                                }
                                ++nq[g];
                                if (lane == 0) {
                                    mbar_arrive_expect_tx(&bars.q_full[g], (uint32_t)(rt2 * G) * 256u);
                                    const uint32_t dst = smem_u32(sQ) + (uint32_t)g * kTileB;
                                    const int tok = (int)p.t0 + p.tok0 + g * rt2;
                                    tma_box3(dst, &mapQ, 0, p.it.g * G, tok, &bars.q_full[g]);
                                    tma_box3(dst + kHalf, &mapQ, 64, p.it.g * G, tok, &bars.q_full[g]);
                                }
                                __syncwarp();
                            }
                        }
                    }
                }
            } while (ok && p.next(kv, sv, ws));
            // every copy issued has landed before the CTA may leave (a stage's earlier copies
            // landed before it was used again)
            if (lane == 0) {
                for (int s = 0; E8 && s < 2; ++s) {
                    const uint32_t uses = (n + 1 - (uint32_t)s) >> 1;
                    if (uses > 0 && !mbar_wait(&bars.raw_full[s], (uses - 1) & 1u)) ok = false;
                }
                for (int s = 0; !E8 && s < kStages; ++s) {
                    if (!((used >> s) & 1u)) continue;
                    // the last use of stage s: the largest i < n with i % kStages == s
                    const uint32_t i = n - 1 - ((n - 1 - (uint32_t)s) % kStages);
                    const bool done = (edge_last >> s) & 1u
                                          ? mbar_wait(&bars.raw[s], ((raw_phase >> s) & 1u) ^ 1u)
                                          : mbar_wait(&bars.full[s], (i / kStages) & 1u);
                    if (!done) ok = false;
                }
                for (int g = 0; g < 2; ++g)
                    if (nq[g] > 0 && !mbar_wait(&bars.q_full[g], (nq[g] - 1) & 1u)) ok = false;
            }
        } else if (E8 && warp >= kAuxWarp) {
            // ---- e4m3 cells to bf16: value = code * 2^e, exact.  Three warps take the K tiles, three
            // the V tiles; the exponents of a team's next tile are on their way meanwhile.  In V tiles
            // with an edge, what not every row sees is treated as below.
            const int team = (warp - kAuxWarp) / kTeamWarps;  // K tiles, V tiles
            const int at = (warp - kAuxWarp - team * kTeamWarps) * 32 + lane;
            const uint8_t *const exp_of = team ? kv.V_exp : kv.K_exp;
            uint32_t turn = 0;
            uint32_t ex[2];  // exponents of cells at and at + 96 of the next tile
            auto load_exps = [&](int tile) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = at + 32 * kTeamWarps * i, j = tile * kN + c;
                    ex[i] = kExpBias;
                    if (c < kN && tile < p.tile1 && j < p.n_see) {
                        const int64_t row = cell_row(kv, p.it.s, p.t0, j);
                        if (row >= 0) ex[i] = exp_of[row * kv.H_kv + p.it.g];
                    }
                }
            };
            do {
                load_exps(p.tile0);
                for (int t = p.tile0; t < p.tile1; ++t, ++turn) {
                    const uint32_t n = 2 * turn + (uint32_t)team;  // raw tile `team`, stage n
                    const int st = (int)(n % kStages);
                    uint8_t *const exps = bars.exps[team][turn & 1u];
                    unsigned char *const raw = raw_tiles + (size_t)team * kRawTile;
                    // (4 bits: as factors, behind the scales)
                    float *const factors = reinterpret_cast<float *>(raw + kN * 72) + (turn & 1u) * kN;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = at + 32 * kTeamWarps * i;
                        if (c >= kN) continue;
                        if constexpr (E4) factors[c] = two_to(min(max((int)ex[i] - kExpBias, kExpMin), kExpMax));
                        else exps[c] = (uint8_t)ex[i];
                    }
                    bool here = bar_wait_warp(&bars.raw_full[team], turn & 1u, wc.limit_ns);
                    if (here && n >= kStages)
                        here = bar_wait_warp(&bars.empty[st], ((n / kStages) - 1) & 1u, wc.limit_ns);
                    // the exponents are there (the other buffer is free: every warp of the team is past
                    // the last turn); a wait that gave up ends the whole team's work
                    if (named_or<32 * kTeamWarps>(kAuxBar + team, !here)) {
                        ok = false;
                        break;
                    }
                    load_exps(t + 1);
                    const bool edge = team && p.edge(t);
                    const int e0 = edge ? max(0, p.pos0 + 1 - t * kN) : kN, e1 = p.n_see - t * kN;
                    const bool odd = E4 ? convert_tile4<32 * kTeamWarps>(raw, ring + (size_t)st * kTileB, factors, at, e0, e1)
                                        : convert_tile<32 * kTeamWarps>(raw, ring + (size_t)st * kTileB, exps, at, e0, e1);
                    if (odd) *reinterpret_cast<volatile int32_t *>(&bars.odd[p.n % kSlots]) = p.n + 1;
                    // written by this warp (generic proxy), read by the tensor cores (async proxy)
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars.raw_empty[team]);
                        mbar_arrive(&bars.full[st]);
                    }
                }
            } while (ok && p.next(kv, sv, ws));
        } else if (!E8 && warp >= kAuxWarp) {
            // ---- V tiles in which some row does not see some cell: values of cells that no row
            // sees become zero (their weight is zero, but zero times an infinity is not), and so
            // do infinities and NaN of cells that only some rows see; the epilogue adds those
            const int aux = warp - kAuxWarp;
            uint32_t n = 0, raw_phase = 0;
            do {
                for (int t = p.tile0; ok && t < p.tile1; ++t, n += 2) {
                    if (!p.edge(t)) continue;
                    const int s = (int)((n + 1) % kStages);
                    if (!bar_wait_warp(&bars.raw[s], (raw_phase >> s) & 1u, wc.limit_ns)) {
                        ok = false;
                        break;
                    }
                    raw_phase ^= 1u << s;
                    const bool here = scrub_tile(ring + (size_t)s * kTileB, max(0, p.pos0 + 1 - t * kN),
                                                 p.n_see - t * kN, 2 * aux, 2 * kAuxWarps);
                    if (here) *reinterpret_cast<volatile int32_t *>(&bars.odd[p.n % kSlots]) = p.n + 1;
                    // written by this warp (generic proxy), read by the tensor cores (async proxy)
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.full[s]);
                }
            } while (ok && p.next(kv, sv, ws));
        }
        __syncwarp();
    } else {
        if constexpr (E8) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        // ---- softmax of group gi: row r by two threads, cells 64 hf .. 64 hf + 63 of each tile.
        // The two warps of a row stay in step (pair barriers): what one of them cannot wait for
        // any more, both give up.
        const int gi = warp >> 3, hf = (warp >> 2) & 1, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const int pair = 1 + gi * 4 + quarter;
        const uint32_t lrow = (uint32_t)(quarter * 32) << 16;
        const uint32_t colS = tmem + lrow + col_s(gi), colO = tmem + lrow + col_o(gi) + 64 * hf;
        float *const swap = &bars.row[gi][r];
        uint32_t cs = 0, co = 0;  // waits on s_full, o_full so far
        // (the part is read where it lies: its fields would take the registers of logits)
        int n = 0;
        bool more;
        do {
            const Parts &p = bars.part[n & 1];
            const int tok = gi * rt2 + r / G;  // of the item
            const bool group = gi == 0 || p.toks > rt2;
            const bool live = r < rt2 * G && tok < p.toks;
            float m = -INFINITY, l = 0.0f;
            {
                const int last = live ? (ws.causal ? p.pos0 + tok : p.cells - 1) : -1;
                const int first_pos = p.pos0 + (ws.causal ? gi * rt2 : 0);  // all rows see up to here
                for (int t = p.tile0; ok && group && t < p.tile1; ++t) {
                    bool here = bar_wait_warp(&bars.s_full[gi], cs & 1u, wc.limit_ns);
                    ++cs;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    float x[64];
                    tmem_ld32_async(colS + 64u * hf, x);
                    tmem_ld32_async(colS + 64u * hf + 32u, x + 32);
                    tmem_wait_ld<64>(x);
                    if (t * kN + kN - 1 > first_pos) {
                        const int lim = last - t * kN - 64 * hf;  // cells up to lim are seen
#pragma unroll
                        for (int e = 0; e < 64; ++e) x[e] = e <= lim ? x[e] : -INFINITY;
                    }
                    // the weights relative to the reference as it stands, over this thread's own
                    // logits; the maximum, meanwhile, says whether they may stay
                    float2 ls[2];
                    const float2 sc = make_float2(scale_log2, scale_log2);
                    auto weights = [&]() {
                        const float mu = m == -INFINITY ? 0.0f : m;
                        const float2 mm = make_float2(-mu, -mu);
                        ls[0] = ls[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float2 v = fma2(make_float2(x[16 * h + e], x[16 * h + e + 1]), sc, mm);
                                v.x = ex2_approx(v.x);
                                v.y = ex2_approx(v.y);
                                ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], v);
                                w[e / 2] = pack_bf16(v.x, v.y);
                            }
                            tmem_st8(colS + (uint32_t)(64 * hf + 8 * h), w);
                        }
                    };
                    weights();
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; e += 8) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], fmaxf(x[e + 2 * k], x[e + 2 * k + 1]));
                    }
                    float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
                    if (named_or<64>(pair, !here || mt > m + kMove)) {
                        // the row's maximum from both; NaN says that a wait gave up
                        if (hf) *swap = here ? mt : NAN;
                        named_sync<64>(pair);
                        if (!hf) {
                            const float other = *swap;
                            here = here && other == other;
                            mt = fmaxf(mt, other);
                            *swap = here ? mt : NAN;
                        }
                        named_sync<64>(pair);
                        if (hf) mt = *swap;
                        if (hf) here = mt == mt;
                        // a maximum over logits is no NaN (fmaxf leaves them out); a quarter of a
                        // row block gives up as a whole
                        if (!__all_sync(0xffffffffu, here)) {
                            ok = false;
                            break;
                        }
                        // the weights stored so far land before those that replace them: two stores
                        // of a thread to one place are ordered by a wait alone
                        tmem_wait_st();
                        const bool move = mt > m + kMove;  // also the first finite maximum
                        const float alpha = move ? ex2_approx(m - mt) : 1.0f;
                        if (move) {
                            l *= alpha;
                            m = mt;
                        }
                        // s_full follows this group's last product with V: o may be rescaled
                        if (t > p.tile0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
                            for (int c = 0; c < 64; c += 16) {
                                float o[16];
                                tmem_ld16(colO + (uint32_t)c, o);
                                uint32_t ou[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) ou[e] = __float_as_uint(o[e] * alpha);
                                tmem_st16(colO + (uint32_t)c, ou);
                            }
                        }
                        weights();
                    }
                    l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                    tmem_wait_st();
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.p_full[gi]);
                }
            }
            if (ok && group) {
                bool here = bar_wait_warp(&bars.o_full[gi], co & 1u, wc.limit_ns);
                ++co;
                here = !named_or<64>(pair, !here);
                if (hf) *swap = l;
                named_sync<64>(pair);
                if (!hf) {
                    l += *swap;
                    *swap = l;
                }
                named_sync<64>(pair);
                if (hf) l = *swap;
                if (!here) ok = false;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            // ---- the part's result: finished rows, or a record to be joined
            const bool starts = p.tile0 == 0, ends = p.tile1 == p.it.tiles;
            const bool odd = *reinterpret_cast<volatile int32_t *>(&bars.odd[n % kSlots]) == n + 1;
            const bool bad = !ok || !p.fits ||
                             *reinterpret_cast<volatile int32_t *>(&bars.bad[n % kSlots]) == n + 1;
            if (group) {
                if (bad) l = NAN;
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                const bool whole = starts && ends;
                float *rec = partial + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * partial_floats(2 * kM, kD);
                const int rr = gi * kM + r;
                const int64_t at = ((p.t0 + p.tok0 + tok) * H_q + p.it.g * G + r % G);
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                    float o[32];
                    if (ok) {
                        tmem_ld32(colO + (uint32_t)c, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.0f;
                    }
                    if (!live) continue;
                    if (odd && ok) {
                        const int see = ws.causal ? p.pos0 + tok : p.cells - 1;
                        const int to = min(min(see, p.n_see - 1), p.tile1 * kN - 1);
                        for (int j = max(p.pos0 + 1, p.tile0 * kN); j <= to; ++j) {
                            const int64_t row = cell_row(kv, p.it.s, p.t0, j);
                            if (row < 0) continue;
                            const int64_t v0 = row * kv.ld_v + (int64_t)p.it.g * kD + 64 * hf + c;
                            if constexpr (E4) {
                                const uint8_t *const sc = kv.V_scale + scale_row(kv, row, p.it.g) * 8 + 4 * hf + c / 16;
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (scale_is_nan(sc[e / 16])) o[e] = NAN;
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] += odd_value_at<E8>(kv, v0 + e);
                            }
                        }
                    }
                    if (whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(out + at * kD + 64 * hf + c);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            dst[e / 8] = make_uint4(pack_bf16(o[e] * inv, o[e + 1] * inv),
                                                    pack_bf16(o[e + 2] * inv, o[e + 3] * inv),
                                                    pack_bf16(o[e + 4] * inv, o[e + 5] * inv),
                                                    pack_bf16(o[e + 6] * inv, o[e + 7] * inv));
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(rec + 4 * kM + (int64_t)rr * kD + 64 * hf + c);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            dst[e / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (live && hf == 0) {
                    if (whole) {
                        if (lse) lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
                    } else {
                        rec[rr] = m;
                        rec[2 * kM + rr] = l;
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            }
            if (starts && tid == 0 && !whole_items)
                note_split(splits, by_item, p.it, ends,
                           div_pos(p.it.start + ws.over + p.it.tiles - 1, bars.per));
            Parts next = p;
            more = next.next(kv, sv, ws);
            if (tid == 0) bars.part[(n + 1) & 1] = next;
            named_sync<32 * kSoftWarps>(kSoftBar);
            ++n;
        } while (more);
    }

    if (!ok) report_timeout(wc);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
}

// The queries [n_tok][H_q][128]: boxes of 64 values x G heads x as many tokens as fill a group.
bool make_query_map(CUtensorMap *m, const void *q, int64_t n_tok, int H_q, int64_t ld_q, int G)
{
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)H_q, (cuuint64_t)n_tok};
    const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)ld_q * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kM / G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxCtas = kTargetSMs;

}  // namespace

bool dense_tc_ok(const DenseArgs &a)
{
    const int G = a.H_q / a.kv.H_kv;
    if (a.kv.ld_k > kMaxStride || a.kv.ld_v > kMaxStride || a.ld_q > kMaxStride) return false;
    // (a TMA map's strides are multiples of 16 bytes; the softmax takes its maximum over unscaled
    // logits: a positive scale)
    const bool cells = a.kv_dtype == QSA_BF16 ||
                       (a.kv_dtype == QSA_E4M3 && a.kv.ld_k % 16 == 0 && a.kv.ld_v % 16 == 0) ||
                       (a.kv_dtype == QSA_E2M1 && a.kv.ld_k % 32 == 0 && a.kv.ld_v % 32 == 0);
    return a.d == kD && a.q_dtype == QSA_BF16 && cells && G <= kM && a.scale > 0.0f && a.pool_rows > 0 &&
           a.pool_rows <= 0x7fffffffLL;
}

size_t dense_tc_workspace()
{
    return kMaxCtas * sizeof(Split) + (size_t)2 * kMaxCtas * partial_floats(2 * kM, kD) * sizeof(float);
}

// Items that are not too long are not cut: a CTA an item (in turns, where there are more than run at once),
// and nothing to join.  What either way costs, in us, fitted to measurements (with nothing in L2, less the
// 8.5 us of an empty call; off by a tenth at most, a few by a quarter): `longest` tiles of the longest item,
// `share` tiles a CTA, `turns` items a CTA.  Long work on bf16 cells runs at the power cap when calls follow one
// another, and more SMs at work win less there: the chunk of 1,024 tokens below takes 745 whole and 777 cut
// in a row of calls, after a pause 730 and 693.
//
// The host does not know the lengths.  A sequence alone is taken to be as long as it may be.  Of several, both
// ends of what they may be are looked at: much alike (chunks as long as the table allows, prompts half as
// long again as their mean), and all but one short.  Whole must be faster in the first, and lose no more in
// the second than cutting loses in the first, nor more than three tenths.
//
// Measured whole and cut, bf16 cells, 32 / 4 heads: a chunk of 1,024 tokens over 61,789 cells 730 and 693, over
// 8,000 115 and 137, of 400 over 2,000 46 and 59, of 64 over 3,000 59 and 48; on e4m3 cells the first 1,482
// and 1,224, over 4,000 118 and 128 (4-bit cells take as long as these and go by their costs).  Four chunks of 256 tokens over 60,000 cells each 712 and 730, over
// 60,000, 500, 500 and 500 704 and 218; over 8,000 each 117 and 145, over 8,000 and three times 500 115 and 81;
// over 2,000 each 48 and 81, over 2,000 and three times 300 46 and 63; sixteen of 512 over 4,000 each 400 and
// 407, over 4,000 and fifteen times 600 145 and 153.  Prompts: 777 tokens, 8 / 2 heads, 30 and 45, of 8,000
// 168 and 149, and beside fifteen of one token 168 and 144; three of 900, 32 / 4 heads, 62 and 77.
template <bool E8>
static bool whole_items(const DenseArgs &a, int rt, int64_t items, int ctas)
{
    if (items > 16 * (int64_t)ctas) return false;
    const double n_tok = (double)a.sv.n_tok, n_seq = (double)a.sv.n_seq;
    const double turns = fmax(n_tok / rt, n_seq) * a.kv.H_kv / ctas;
    struct Cost {
        double whole, cut;
    };
    const auto cost = [&](double longest, double share) -> Cost {
        const double held = 1.6 * share + (items <= ctas ? 0.2 : 0.1) * fmax(0.0, share - 100.0);
        if (items <= ctas)
            return E8 ? Cost{12.0 + 3.0 * longest, 36.0 + 2.9 * share + 15.0 * turns}
                      : Cost{14.0 + 1.46 * longest, 35.0 + held + 16.0 * turns};
        return E8 ? Cost{15.0 + 1.6 * longest + 3.0 * share + 4.6 * turns, 37.0 + 2.75 * share + 10.0 * turns}
                  : Cost{14.0 + 0.9 * longest + 1.5 * share + 8.0 * turns, 41.0 + held + 7.0 * turns};
    };
    Cost alike, one_long;
    if (a.kv.table) {
        const double cells = fmax((double)(a.kv.ld_table << a.kv.page_shift), 1.0), longest = cells / kN;
        // (a row tile in the midst of the new tokens does not see those behind it)
        const double share = longest * turns * (1.0 - 0.5 * fmin(1.0, n_tok / n_seq / cells));
        alike = cost(longest, share);
        one_long = cost(longest, share / n_seq + turns);
    } else {
        const double longest = (a.sv.n_seq > 1 ? fmin(n_tok, 1.5 * n_tok / n_seq) : n_tok) / kN;
        const double most = fmax(n_tok - n_seq + 1.0, 1.0) / kN;
        alike = cost(longest, 0.5 * longest * turns);
        one_long = cost(most, 0.5 * most * turns);
    }
    return alike.whole < alike.cut &&
           (a.sv.n_seq == 1 || (one_long.whole - one_long.cut < alike.cut - alike.whole &&
                                one_long.whole < 1.3 * one_long.cut));
}

// 4-bit rows in boxes of one head's 64 bytes x box_rows rows, row after row.
static bool make_map4(CUtensorMap *m, const void *base, int64_t rows, int H_kv, int64_t ld, int box_rows)
{
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)H_kv * (kD / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld / 2};
    const cuuint32_t box[2] = {kD / 2, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool E8, bool E4 = false>
static qsa_status run_tc(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv;
    const int page = 1 << a.kv.page_shift;
    const int box_rows = a.kv.table && page < kN ? page : kN;
    CUtensorMap mq, mk, mv;
    const int64_t width = (int64_t)a.kv.H_kv * kD;
    if (!make_query_map(&mq, a.q, a.sv.n_tok, a.H_q, a.ld_q, G)) return QSA_ERR_CUDA;
    if (E4 ? !make_map4(&mk, a.kv.K, a.pool_rows, a.kv.H_kv, a.kv.ld_k, box_rows) ||
                 !make_map4(&mv, a.kv.V, a.pool_rows, a.kv.H_kv, a.kv.ld_v, box_rows)
           : !make_map(&mk, a.kv.K, a.pool_rows, width, a.kv.ld_k, box_rows, E8, !E8) ||
                 !make_map(&mv, a.kv.V, a.pool_rows, width, a.kv.ld_v, box_rows, E8, !E8))
        return QSA_ERR_CUDA;
    const WorkShape ws = work_shape(a, 2 * (kM / G), kN, kOver);
    constexpr size_t smem = tc_smem<E8>();
    if (ensure_kernel_attrs<dense_tc_kernel<E8, E4>>(smem) != cudaSuccess) return QSA_ERR_CUDA;
    int ctas = device_sm_count();
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    Split *splits = static_cast<Split *>(workspace);
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + kMaxCtas * sizeof(Split));
    const int64_t items = ((a.sv.n_tok + ws.rt - 1) / ws.rt + a.sv.n_seq) * a.kv.H_kv;
    const bool whole = whole_items<E8>(a, ws.rt, items, ctas);
    if (whole) ctas = (int)items;
    cudaError_t e = launch(dense_tc_kernel<E8, E4>, dim3((unsigned)ctas), dim3(Cfg<E8>::kThreads), smem, st, 1, mq,
                           mk, mv, a.kv, a.sv, ws, box_rows, a.H_q, a.scale * kLog2e,
                           static_cast<__nv_bfloat16 *>(a.out), a.lse, partial, splits,
                           (int)join_by_item(a, ws.rt, ctas), (int)whole, current_wait_ctl());
    if (e == cudaSuccess && !whole)
        e = launch_dense_join<__nv_bfloat16>(splits, partial, ctas, 2 * kM, kM / G, a, st);
    return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

qsa_status launch_dense_tc(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    if (a.kv_dtype == QSA_E2M1) return run_tc<true, true>(a, workspace, st);
    return a.kv_dtype == QSA_E4M3 ? run_tc<true>(a, workspace, st) : run_tc<false>(a, workspace, st);
}

}  // namespace qsa
