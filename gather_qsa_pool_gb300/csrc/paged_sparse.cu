// paged_sparse.cu -- attention of each token over the blocks listed for it, in place on a paged cache: a cluster of
// CTAs takes one token and one or more of its KV heads, its CTAs equal shares of the token's listed cells, which are
// joined through distributed shared memory (one launch, no workspace).
//
// Mathematics and a warp's products: few_cells.cuh.  Each warp runs a ring of stages of its own (cp.async) over its
// cells of every tile: warp w takes head w mod hpc and part w / hpc of a tile's 4 / hpc parts (hpc is 1, 2 or 4).
// A tile's list entries are looked up two turns ahead of its copies and their pages one turn ahead.
#include "few_cells.cuh"
#include "paged.cuh"

namespace qsa {
namespace few {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

// Stages of a warp's ring and CTAs per SM.
template <int C, int NB, int NT>
struct Plan {
    static constexpr int kCtas = NB == 4 || NB * NT == 4 ? 2 : C == QSA_E2M1 && NB * NT == 1 ? 4 : 3;
    static constexpr int kStages = C == QSA_E2M1 && NB * NT > 1 ? 3 : 2;
};

template <int NB>
__host__ __device__ constexpr size_t fin_bytes() { return (size_t)8 * NB * (kPitch + 2) * 4; }
template <int C, int NB, int NT>
__host__ __device__ constexpr size_t sparse_smem(int hpc)
{
    constexpr int S = kWarps * Plan<C, NB, NT>::kStages;
    return (size_t)S * Cell<C>::kStage + (Cell<C>::kF16 ? (size_t)S * 32 * 16 : 0) + hpc * (q_bytes<NB, NT>() + fin_bytes<NB>());
}

// CTAs of an SM as far as shared memory lets them (a CTA takes 1 KB besides, and what the kernel declares).
template <int C, int NB, int NT>
constexpr int ctas_that_fit(int hpc)
{
    const int n = (int)(228 * 1024 / (sparse_smem<C, NB, NT>(hpc) + 1024 + 128 + 3 * kWarps * 8 * NB * 4));
    return n < Plan<C, NB, NT>::kCtas ? n : Plan<C, NB, NT>::kCtas;
}
// KV heads of rows of codes that may share a CTA, as a power of two: as many CTAs fit an SM as with one.
template <int C, int NB, int NT>
constexpr int most_heads()
{
    const int one = ctas_that_fit<C, NB, NT>(1);
    if (!Cell<C>::kF16 || ctas_that_fit<C, NB, NT>(2) < one) return 0;
    return ctas_that_fit<C, NB, NT>(4) < one ? 1 : 2;
}

template <int C, typename TQ, int NB, int NT>
__global__ void __launch_bounds__(kThreads, (Plan<C, NB, NT>::kCtas))
paged_sparse_kernel(const KvView kv, const SeqView sv, const ListView lv, const TQ *__restrict__ q, int64_t ld_q, int H_q,
                    float scale_log2, float q_sign, TQ *__restrict__ out, float *__restrict__ lse, int hpc_log2, int kt_log2)
{
    using S = Cell<C>;
    constexpr int kRows = 8 * NB, kStages = Plan<C, NB, NT>::kStages, kKeys = S::kKeys;
    constexpr bool F16 = S::kF16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int bad_s;
    __shared__ float red_m[kWarps][kRows], red_l[kWarps][kRows];
    __shared__ __align__(16) float undo_s[kWarps][kRows];  // by head
    __shared__ uint32_t there_s[kWarps][kStages];          // cells of a stage that are there

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, c4 = lane & 3;
    unsigned char *const ring = smem + (size_t)warp * kStages * S::kStage;
    const int hpc = 1 << hpc_log2, head = warp & (hpc - 1), part = warp >> hpc_log2;
    // per cell of a stage (codes): 2^ke, exponent e of the value, 2^-e
    float4 *const exps = reinterpret_cast<float4 *>(smem + (size_t)kWarps * kStages * S::kStage) + warp * kStages * 32;
    uint4 *const q_all = reinterpret_cast<uint4 *>(smem + (size_t)kWarps * kStages * (S::kStage + (F16 ? 512 : 0)));  // by head
    const uint4 *const qf = q_all + head * (int)(q_bytes<NB, NT>() / 16);
    float *const fin = reinterpret_cast<float *>(q_all + hpc * (int)(q_bytes<NB, NT>() / 16));  // rows head by head

    pdl_wait();
    const TQ *qp = q;
    QSA_AFTER_WAIT(qp);
    pdl_trigger();

    const int G = H_q / kv.H_kv, groups = kv.H_kv >> hpc_log2;
    uint32_t rank, ranks;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const unsigned item = blockIdx.x / ranks;
    const int64_t tok = item / (unsigned)groups;
    const int group = (int)(item % (unsigned)groups), kv_head = (group << hpc_log2) + head;
    int seq, pos, cells;
    if (!token_place(sv, tok, seq, pos, cells)) return;  // (all CTAs of the cluster)
    const bool fits = cells_fit(kv, cells);
    const int n_list = (int)min((int64_t)max(lv.counts[tok], 0), lv.k_blk);
    const int32_t *const list = lv.blocks + tok * lv.k_blk;
    const int tiles = fits ? (n_list >> (kt_log2 - 2)) + 1 : 0;  // of 4 n_list + 4 cells
    const int share = (tiles + (int)ranks - 1) / (int)ranks;
    const int tile0 = min((int)rank * share, tiles), tile1 = min(tile0 + share, tiles);
    if (tid == 0) bad_s = 0;

    // ---- the ring: p_next, entry_next: this lane's cell of the next tile to issue, and its page; blk_next: the list
    // entry of its cell of the tile after that
    const int my_key = part * kKeys + (lane < kKeys ? lane : 0);
    bool bad = false, far = false;
    int32_t p_next = -1, entry_next = -1, blk_next = -1;
    auto look_list = [&](int tile) {
        const int i = (tile << kt_log2) + my_key;
        blk_next = tile < tile1 && (i >> 2) < n_list ? list[i >> 2] : -1;
    };
    // the cell of tile `tile`, whose entry is in blk_next; then the entry of the tile after it
    auto look_up = [&](int tile) {
        const int i = (tile << kt_log2) + my_key;
        p_next = -1;
        if (tile < tile1) {
            const int open = (pos + 1) & ~3;  // the open block's first cell
            if ((i >> 2) < n_list) p_next = blk_next >= 0 && blk_next <= ((pos - 3) >> 2) ? 4 * blk_next + (i & 3) : -1;
            else if ((i >> 2) == n_list && open + (i & 3) <= pos) p_next = open + (i & 3);
        }
        if (p_next >= 0) {
            const int64_t j = p_next >> kv.page_shift;
            entry_next = j < kv.ld_table ? kv.table[(int64_t)seq * kv.ld_table + j] : -1;
        }
        look_list(tile + 1);
    };
    auto row_next = [&]() -> int32_t {
        if (p_next < 0) return -1;  // not there: zeros
        if ((uint32_t)entry_next >= (uint32_t)kv.n_pages) {
            bad = true;
            return -1;
        }
        return (entry_next << kv.page_shift) | (p_next & ((1 << kv.page_shift) - 1));
    };
    int pend_k[kStages - 1], pend_v[kStages - 1];  // exponents of the next tiles, on their way
    const uint8_t *const Ke = F16 ? kv.K_exp + kv_head : nullptr, *const Ve = F16 ? kv.V_exp + kv_head : nullptr;
    auto load_exps = [&](int32_t row, int i) {
        const uint64_t at = (uint64_t)(uint32_t)row * (uint32_t)kv.H_kv;
        pend_k[i] = row >= 0 ? Ke[at] : kExpBias;
        pend_v[i] = row >= 0 ? Ve[at] : kExpBias;
    };
    auto keep_exps = [&](int stage) {  // the next tile's
        const int ek = min(max(pend_k[0] - kExpBias, kExpMin), kExpMax);
        const int ev = min(max(pend_v[0] - kExpBias, kExpMin), kExpMax);
        far = far || __any_sync(0xffffffffu, abs(ev) > (int)kFar);
        exps[stage * 32 + lane] = make_float4(two_to(ek), (float)ev, two_to(-ev), 0.0f);
#pragma unroll
        for (int i = 0; i + 1 < kStages - 1; ++i) {
            pend_k[i] = pend_k[i + 1];
            pend_v[i] = pend_v[i + 1];
        }
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
    auto note_there = [&](int stage) {
        const uint32_t there = __ballot_sync(0xffffffffu, p_next >= 0);
        if (lane == 0) there_s[warp][stage] = there;
    };
    look_list(tile0);
    look_up(tile0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        note_there(i);
        const int32_t row = row_next();
        look_up(tile0 + i + 1);
        if (tile0 + i < tile1) {
            issue(i, row);
            if constexpr (F16) load_exps(row, i);
        }
        cp_commit();
    }
    stage_queries<C, TQ, NB, NT, kWarps>(tid, qp + tok * ld_q + (int64_t)(group << hpc_log2) * G * kD, ld_q, G, G, hpc, q_sign,
                                         scale_log2, q_all, undo_s[0]);
    __syncthreads();
    Rows<C, NB, NT> w;
    w.clear();
    int slot = 0;
    for (int tile = tile0; tile < tile1; ++tile) {
        cp_wait<kStages - 2>();
        if constexpr (F16) keep_exps(slot);
        __syncwarp();
        const uint32_t there = there_s[warp][slot];
        const int nslot = slot == 0 ? kStages - 1 : slot - 1;
        // ---- issue the tile kStages - 1 ahead into the stage read in the last turn
        note_there(nslot);
        const int32_t row = row_next();
        look_up(tile + kStages);
        if (tile + kStages - 1 < tile1) {
            issue(nslot, row);
            if constexpr (F16) load_exps(row, kStages - 2);
        }
        cp_commit();
        constexpr uint32_t kAll = 0xffffffffu << (32 - kKeys);
        if (there << (32 - kKeys))
            w.tile(ring + slot * S::kStage, exps + slot * 32, qf, undo_s[head], scale_log2, far, there << (32 - kKeys) != kAll,
                   [&](int c, int, int) { return !((there >> c) & 1u); });
        __syncwarp();
        slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    cp_wait<0>();
    if (__any_sync(0xffffffffu, bad) && lane == 0) bad_s = 1;
    w.finish();
    if (g8 == 0) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                red_m[warp][8 * n + 2 * c4 + e] = w.ms[n][e];
                red_l[warp][8 * n + 2 * c4 + e] = w.l[n][e];
            }
    }
    __syncthreads();  // every warp is done with its ring
    // ---- join the warps of a head: rows of the CTA's heads, G of each
    const int heads = G << hpc_log2, rec_rows = kRows << hpc_log2;
    const bool nan_out = bad_s != 0 || !fits;
    constexpr int kTurn = NB > 2 ? 2 : NB;  // blocks that are joined at a time
    float *const ob = reinterpret_cast<float *>(smem);  // [warp][row][kPitch]
    static_assert((size_t)kWarps * 8 * kTurn * kPitch * 4 <= (size_t)kWarps * kStages * S::kStage, "the warps' sums fit over the ring");
    auto store = [&](int64_t at, int c, float m, float sum, const float (&v)[4]) {
        const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
        TQ *const dst = out + at * kD + c;
        if constexpr (sizeof(TQ) == 2)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv));
        else
            *reinterpret_cast<float4 *>(dst) = make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        if (c == 0 && lse) lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
    };
#pragma unroll
    for (int n0 = 0; n0 < NB; n0 += kTurn) {
        if (n0 > 0) __syncthreads();
#pragma unroll
        for (int n = n0; n < n0 + kTurn; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * c4 + e;
                float m = -INFINITY;
                for (int k = head; k < kWarps; k += hpc) m = fmaxf(m, red_m[k][r]);
                const float f = w.mx[n][e] == -INFINITY ? 0.0f : ex2_approx(w.mx[n][e] - (m == -INFINITY ? 0.0f : m));
                float *const dst = ob + (size_t)(warp * 8 * kTurn + r - 8 * n0) * kPitch;
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) dst[frag_dim<C>(t, g8, hf)] = w.o[t][n][2 * hf + e] * f;
            }
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < (8 * kTurn * (kD / 4)) << hpc_log2; i += kThreads) {
            const int rl = (i / (kD / 4)) % (8 * kTurn), h = i / (kD / 4 * 8 * kTurn), r = 8 * n0 + rl, c = (i % (kD / 4)) * 4;
            if (r >= G) continue;
            float m = -INFINITY, sum = 0.0f;
            for (int k = h; k < kWarps; k += hpc) m = fmaxf(m, red_m[k][r]);
            const float u = m == -INFINITY ? 0.0f : m;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k = h; k < kWarps; k += hpc) {
                sum += red_m[k][r] == -INFINITY ? red_l[k][r] : red_l[k][r] * ex2_approx(red_m[k][r] - u);
                const float4 y = *reinterpret_cast<const float4 *>(&ob[(size_t)(k * 8 * kTurn + rl) * kPitch + c]);
                v[0] += y.x; v[1] += y.y; v[2] += y.z; v[3] += y.w;
            }
            if (nan_out) sum = NAN;
            if (ranks == 1) {
                store(tok * H_q + group * heads + h * G + r, c, m, sum, v);
            } else {
                *reinterpret_cast<float4 *>(fin + (h * G + r) * kPitch + c) = make_float4(v[0], v[1], v[2], v[3]);
                if (c == 0) {
                    fin[rec_rows * kPitch + h * G + r] = m;
                    fin[rec_rows * kPitch + rec_rows + h * G + r] = sum;
                }
            }
        }
    }
    if (ranks == 1) return;
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
            const float f = km == -INFINITY ? 1.0f : ex2_approx(km - u);  // an unset side is zero or NaN
            float4 y;
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                         : "r"(there(k, r * kPitch + c))
                         : "memory");
            sum += kl * f;
            v[0] += y.x * f; v[1] += y.y * f; v[2] += y.z * f; v[3] += y.w * f;
        }
        store(tok * H_q + group * heads + r, c, m, sum, v);
    }
    // no CTA leaves while another reads its part
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

}  // namespace few

namespace {

template <int C, typename TQ, int NB, int NT>
cudaError_t run(const SparseArgs &a, cudaStream_t st)
{
    using P = few::Plan<C, NB, NT>;
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr auto kernel = few::paged_sparse_kernel<C, TQ, NB, NT>;
    constexpr int kMost = few::most_heads<C, NB, NT>();
    cudaError_t e = ensure_kernel_attrs<few::paged_sparse_kernel<C, TQ, NB, NT>>(few::sparse_smem<C, NB, NT>(1 << kMost));
    if (e != cudaSuccess) return e;
    // Two or four heads of a row go to one CTA, so that a row is read in larger pieces, where as many CTAs fit an SM as
    // with one and the GPU is filled twice. One head / several, us of a graph replayed cold, 2,052 cells, 4 KV heads in
    // groups of 8, 4-bit cells: chunks of 608 tokens 167 / 161, 1,024 272 / 269, 2,048 526 / 503, a token of 1,216
    // sequences (1,028 cells) 210 / 192; below that they lose as often as they win (512 tokens 148 / 143, 256 81 / 87; a
    // token of 256 sequences 63 / 56, of 456 89 / 99). 1,024 tokens in groups of 32, 4-bit cells 700 / 646, of 16, 8-bit
    // cells 450 / 401; fp32 queries in groups of 8, 8-bit cells 362 / 335 (four heads; two 339). Where fewer CTAs fit they
    // are kept apart: 1,024 tokens in groups of 8, 8-bit cells 253 / 286, of 32 708 / 968; of 16, 4-bit cells 390 / 435,
    // fp32 queries in groups of 8 340 / 386 (but a token of 1,216 sequences 318 / 286 and 275 / 258, with four).
    // CTAs of a token and its heads: as many as fill the GPU but for what clusters of their size leave of it, a tile each
    // at most, up to the portable cluster's eight.  (All of it instead of seven eighths, us: 38 tokens, 4-bit cells 37 and
    // not 30, bf16 51 and not 46, 14 tokens 8-bit 30 and not 21; 48 tokens 36 and not 37; otherwise alike.  Five eighths:
    // 64 tokens 4-bit 43 and not 40, 48 tokens 40 and not 34.  One each where tokens x heads are no fewer than SMs: 38
    // tokens bf16 54 and not 44.)
    const int64_t most = P::kCtas * device_sm_count();
    int hl = kMost;
    while (hl > 0 && (a.kv.H_kv % (1 << hl) || (a.sv.n_tok * a.kv.H_kv >> hl) < 2 * most)) --hl;
    const int kt_log2 = (C == QSA_BF16 ? 6 : 7) - hl;
    const int64_t items = a.sv.n_tok * (a.kv.H_kv >> hl), tiles = (a.k_blk >> (kt_log2 - 2)) + 1;
    int64_t parts = most * 7 / 8 / items;
    if (parts > tiles) parts = tiles;
    if (parts > 8) parts = 8;
    if (parts < 1) parts = 1;
    return launch(kernel, dim3((unsigned)(items * parts)), dim3(few::kThreads), few::sparse_smem<C, NB, NT>(1 << hl), st, (int)parts,
                  a.kv, a.sv, ListView{a.blocks, a.counts, a.k_blk}, static_cast<const TQ *>(a.q), a.ld_q, a.H_q, scale, q_sign,
                  static_cast<TQ *>(a.out), a.lse, hl, kt_log2);
}

template <int C>
cudaError_t run_cells(const SparseArgs &a, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv;
    // Terms: of fp32 queries as many as hold 22 or 24 bits; of bf16 queries, which one holds, one, so that a weight has 8
    // bits on bf16 cells (11 on codes): outputs are 0.0022 off in the 2-norm, 0.0017 with two (what the bf16 output's own
    // rounding is), but 1,024 tokens take 300 us and not 358, one token 17.5 and not 18.6 (a graph replayed cold).
    constexpr int NT = C == QSA_BF16 ? 3 : 2;
    if (a.q_dtype == QSA_F32) {
        if (G <= 8) return run<C, float, 1, NT>(a, st);
        return G <= 16 ? run<C, float, 2, NT>(a, st) : run<C, float, 4, NT>(a, st);
    }
    if (G <= 8) return run<C, __nv_bfloat16, 1, 1>(a, st);
    return G <= 16 ? run<C, __nv_bfloat16, 2, 1>(a, st) : run<C, __nv_bfloat16, 4, 1>(a, st);
}

}  // namespace

cudaError_t launch_paged_sparse(const SparseArgs &a, cudaStream_t st)
{
    // rows in 16-byte chunks, strides in 32 bits
    const int chunk = a.kv_dtype == QSA_E2M1 ? 32 : (a.kv_dtype == QSA_E4M3 ? 16 : 8);
    const bool fine = a.d == few::kD && a.H_q / a.kv.H_kv <= 32 && a.kv.ld_k % chunk == 0 && a.kv.ld_v % chunk == 0 &&
                      a.kv.ld_k <= (1 << 28) && a.kv.ld_v <= (1 << 28);
    if (fine && a.kv_dtype == QSA_BF16) return run_cells<QSA_BF16>(a, st);
    if (fine && a.kv_dtype == QSA_E4M3) return run_cells<QSA_E4M3>(a, st);
    if (fine && a.kv_dtype == QSA_E2M1) return run_cells<QSA_E2M1>(a, st);
    DenseArgs d;
    d.kv = a.kv;
    d.sv = a.sv;
    d.kv_dtype = a.kv_dtype;
    d.q_dtype = a.q_dtype;
    d.q = a.q;
    d.ld_q = a.ld_q;
    d.out = a.out;
    d.lse = a.lse;
    d.H_q = a.H_q;
    d.d = a.d;
    d.scale = a.scale;
    d.causal = 1;
    d.pool_rows = 0;
    d.list = {a.blocks, a.counts, a.k_blk};
    return launch_dense_attn(d, st);
}

}  // namespace qsa
