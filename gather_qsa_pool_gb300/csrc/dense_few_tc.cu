// dense_few_tc.cu -- attention of a few query rows per sequence (a token, or a token and its drafts)
// over a long paged or packed cache, bf16 queries, on the tcgen05 tensor cores: bound by the one pass
// over the cells' keys and values.
//
// Mathematics: as dense_attn.cu, one pass with a running reference m (an integer, in log2 units) and
// sum l per row; m moves, and what was summed so far is scaled, only when a weight would pass the
// range left above it, so almost no tile does that.  A part's (m, l, o) are joined by scaling to a
// common m (dense_join.cuh).
//
// Operands are swapped so that the cells fill the tensor cores' 128 rows and the few query rows (16 or
// 32: new tokens x heads of one KV head) are columns:
//   S' [cell][row]  = K Q'      A = the K tile as it lies in memory, B = the queries
//   O' [dim][row]  += V' P'     A = the V tile transposed by its descriptor, B = the weights
// so K and V go from TMA to the tensor cores without passing a register.  One thread holds a cell's
// logits (a row of S'), which makes the exponents of an e4m3 cell one multiplication and one addition
// a logit: x = s 2^ke + ve.
// e4m3 cells: the products run in 8 bits (kind::f8f6f4), A = the codes as they are.  A query, and a
// weight, is three e5m2 terms that lie beside each other as columns: e5m2 is the upper byte of fp16, so
// the terms of an fp16 number are its upper byte, the upper byte of what that leaves, and of what that
// leaves: 3 + 3 + 3 significant bits.  A bf16 query (8 bits) is exact in them down to 2^-31 of the
// row's largest (a row is scaled for itself).  Weights are rounded to 9 bits; what a weight's terms
// leave for the next is taken 8 times as large (and their products that much smaller), so that small
// weights are not cut off where e5m2 ends (2^-16) while the sum counts them: a weight is off by 2^-9
// of itself or by 3 * 2^-23, where the largest is at least 2^10.  The sum l adds 2^(x - ve), from the
// weight where |ve| is at most 50.
//
// Shape: one persistent CTA per SM, an equal share of the flattened list of (sequence, KV head, row
// tile) items in tiles of 128 cells (dense.cuh).  Warps 0-7: two groups that take the weights of the
// tiles in turn, a cell a thread, each with references, sums and output of its own, joined at the end of
// a part; warp 8 issues the MMAs, warps 9 and 10 the copies of K and of V (rings of 16 or 32 KB stages,
// one box per page; one warp for both could not keep up), warps 11 and 12 lay out the next part's
// queries, look the next part up for the others and see to the tiles where some row does not see some
// cell.  Per tile the tensor cores run O_g += V' P_g and S_g of the group's next tile, while the other
// group computes.
//
// What bounds it: bf16, the bytes (64 sequences of up to 8,000 cells, 32 / 4 heads, one token: 99 us,
// 5.4 TB/s; one of 255,181: 92 us).  e4m3, the weights' turn from logits to terms and back to the tensor
// cores, about 1,500 cycles a tile with two groups in flight where the bytes take 1,000 (48 sequences of
// up to 16,384 cells, 32 rows: 101 us; 16 rows: 86 us, 4.7 TB/s), and about 8,000 cycles at each end of a
// part (references, sums and outputs joined, the first references).
//
// Every mbarrier wait is bounded: after one gives up, nothing new is issued, what was issued is waited
// for, the rows not finished become NaN and the tensor memory is returned.
#include "dense_join.cuh"
#include "dense_tc.cuh"

namespace qsa {
namespace {

constexpr int kGroups = 2;      // of softmax warps, four each: a cell of a tile to a thread
constexpr int kSoftWarps = 4 * kGroups, kMmaWarp = kSoftWarps, kLoadWarp = kMmaWarp + 1, kAuxWarp = kLoadWarp + 2;
constexpr int kAuxWarps = 2;
constexpr int kThreads = 32 * (kAuxWarp + kAuxWarps);
constexpr int kMaxStages = 10;
constexpr int kBarVote = 1, kBarAll = 3, kBarAux = 4, kBarFirst = 5;  // named barriers: 1, 2 the groups'
constexpr float kUnset = 3.0e38f;  // -m of a row that has seen nothing: any logit moves it
// Exponents of V beyond this: the sum takes an exponential of its own (2^(x - m) times 2^-ve could
// start from a weight that is zero).
constexpr int kFar = 50;

template <bool E8, int NR>
struct Few {
    static constexpr int kTerms = E8 ? 3 : 1;
    static constexpr int kCols = kTerms * NR;                  // columns of S' and O'
    static constexpr uint32_t kStage = E8 ? kRawTile : kTileB;
    static constexpr uint32_t kQBytes = NR * 128 * (E8 ? 3 : 2);
    static constexpr uint32_t kPBytes = kN * 128;              // a cell's weights: 128 bytes, in part used
    // stages of K, of V
    static constexpr int kOfK = E8 ? 5 : 2, kOfV = E8 ? 5 : 3;
    static constexpr int kStages = kOfK + kOfV;
    static constexpr int kOver = E8 ? 7 : 4;                   // an item's fixed cost in tiles
    static constexpr uint32_t kStride = kCols <= 16 ? 16 : (kCols <= 32 ? 32 : (kCols <= 64 ? 64 : 128));
    static constexpr uint32_t kTmem = 2 * kGroups * kStride;
    // the weights' range: at most 2^kTop where m was set, 2^kMost before it moves (bf16: any; fp16 terms:
    // below 2^16)
    static constexpr float kTop = E8 ? 11.0f : 0.0f, kMost = E8 ? 32768.0f : 256.0f;
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages], raw[kMaxStages];  // of K's stages, then V's
    uint64_t part_full[kSlots];
    uint64_t s_full[kGroups], p_full[kGroups], o_full[kGroups], q_full[2], q_free[2], drain;
    uint32_t tmem, pad;
    int32_t odd[kSlots], bad[kSlots];  // number + 1 of the part that set it
    alignas(16) float qs[kSlots][32];  // what the part's rows of queries were divided by
    alignas(16) float nm[kGroups][32], mref[kGroups][32];  // -m, m of a group's rows
    float2 al[kGroups][32], fac[kGroups][32];  // factors 2^x as two, each in range
    alignas(16) float red[kGroups][4][32];
    float sum[kGroups][4][32];
    float inv[32];
    int32_t see[32];                   // last cell of a row
    int64_t at[32];                    // place of a row's results, -1: none
    Parts part[kSlots];                // the parts ahead, by number; more: there is one
    int32_t more[kSlots];
    int64_t per;                       // places of a CTA
    Parts now[2];                      // the part that a query warp is at
    Parts alone[2];                    // after a wait that gave up: the softmax warps' part, and the next
};

template <bool E8, int NR>
__host__ __device__ constexpr size_t few_smem()
{
    using F = Few<E8, NR>;
    return 1024 + (size_t)F::kStages * F::kStage + kGroups * F::kPBytes + 2 * F::kQBytes + sizeof(Bars);
}
static_assert(few_smem<false, 16>() <= 227 * 1024 && few_smem<true, 16>() <= 227 * 1024 &&
                  few_smem<false, 32>() <= 227 * 1024 && few_smem<true, 32>() <= 227 * 1024,
              "shared memory of one CTA");

// 2^e as two factors that fp32 holds; zero below 2^-252.
__device__ __forceinline__ float2 two_factors(float e)
{
    if (!(e > -252.0f)) return e != e ? make_float2(NAN, NAN) : make_float2(0.0f, 0.0f);
    const int i = (int)fminf(e, 252.0f), a = i >> 1;
    return make_float2(two_to(a), two_to(i - a));
}

__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, float *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_ld_async(uint32_t taddr, float *v)
{
    static_assert(N == 8 || N == 16, "columns of a load");
    if constexpr (N == 16) tmem_ld16_async(taddr, v);
    else tmem_ld8_async(taddr, v);
}

// N values (16 or 32) of each lane summed over the warp's lanes: lane i returns value i % N.  A step halves
// the values that a lane holds.
template <int N>
__device__ __forceinline__ float col_sum(float (&v)[N])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = N / 2; h > 0; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float keep = up ? v[i + h] : v[i], send = up ? v[i] : v[i + h];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, h);
        }
    }
    if constexpr (N == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
    return v[0];
}
// The largest over the warp's lanes, in every lane (a NaN counts for nothing).
__device__ __forceinline__ float lane_max(float v)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp16 numbers as their upper bytes, and what those leave.
__device__ __forceinline__ uint32_t less_upper(uint32_t h)
{
    const uint32_t u = h & 0xff00ff00u;
    const __half2 r = __hsub2(reinterpret_cast<const __half2 &>(h), reinterpret_cast<const __half2 &>(u));
    return reinterpret_cast<const uint32_t &>(r);
}
// The same, what is left 8 times as large (exact; of numbers of at most 2^15 it stays below 2^15).
__device__ __forceinline__ uint32_t less_upper_grown(uint32_t h)
{
    const uint32_t u = less_upper(h);
    const __half2 r = __hmul2(reinterpret_cast<const __half2 &>(u), __floats2half2_rn(8.0f, 8.0f));
    return reinterpret_cast<const uint32_t &>(r);
}

// Rows r0 .. of a tile of codes as scrub_tile takes them (a row is 128 bytes, 8 lanes).
__device__ __forceinline__ bool scrub_codes(unsigned char *tile, int r0, int r1, int first, int step)
{
    const int lane = threadIdx.x & 31;
    bool odd = false;
    for (int r = r0 + first + (lane >> 3); r < kN; r += step) {
        uint4 *w = reinterpret_cast<uint4 *>(tile + r * 128 + (lane & 7) * 16);
        if (r >= r1) {
            *w = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint4 v = *w;
        uint32_t *u = reinterpret_cast<uint32_t *>(&v);
        bool any = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t m = __vcmpeq4(u[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
            any |= m != 0;
            u[k] &= ~m;
        }
        if (any) *w = v;
        odd |= any;
    }
    return odd;
}

// A part's queries in the form that the products take, by kLanes threads (`at`: this one's number;
// barrier kBar is theirs): rows behind the part's last become zero.  e4m3: a row is scaled by a power of two of its
// own (one for the part would let a large query of one token or head take another's bits), undone by qs.  here: false
// when this thread's warp has given up; false for all is returned then.
template <bool E8, int NR, int kLanes, int kBar>
__device__ __forceinline__ bool lay_queries(const Parts &w, int at, bool here, const __nv_bfloat16 *q, int64_t ld_q,
                                            int G, uint32_t inv_g, float q_sign, unsigned char *dst, float *qs)
{
    constexpr int kUnits = NR * 8 / kLanes;  // 16 dims each
    const int rows = w.toks * G;
    uint4 raw[kUnits][2];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int r = (at + kLanes * i) >> 3;
        raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (here && r < rows) {
            const int tok = (int)((uint32_t)r * inv_g >> 16);
            const uint4 *src = reinterpret_cast<const uint4 *>(
                q + (w.t0 + w.tok0 + tok) * ld_q + (int64_t)(w.it.g * G + r - tok * G) * kD + (at & 7) * 16);
            raw[i][0] = src[0];
            raw[i][1] = src[1];
        }
    }
    if (named_or<kLanes>(kBar, !here)) return false;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int r = (at + kLanes * i) >> 3, u = at & 7;
        float mul = q_sign;
        if constexpr (E8) {
            // the row's largest finite magnitude, by its bits
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t x = (&raw[i][k >> 2].x)[k & 3];
                const uint32_t a = x & 0x7fffu, b = (x >> 16) & 0x7fffu;
                top = max(top, a < 0x7f80u ? a : 0u);
                top = max(top, b < 0x7f80u ? b : 0u);
            }
#pragma unroll
            for (int k = 1; k < 8; k <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
            // it becomes at least 2^14 and less than 2^15
            const int a = max(-100, (int)(top >> 7) - 141);
            mul *= two_to(-a);
            if (u == 0) *reinterpret_cast<volatile float *>(&qs[r]) = two_to(a);
        }
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t x = (&raw[i][k >> 2].x)[k & 3];
            const float lo = __uint_as_float(x << 16) * mul, hi = __uint_as_float(x & 0xffff0000u) * mul;
            if constexpr (E8) {
                const __half2 v = __floats2half2_rn(lo, hi);
                h[k] = reinterpret_cast<const uint32_t &>(v);
            } else {
                h[k] = pack_bf16(lo, hi);
            }
        }
        if constexpr (E8) {
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                uint4 o;
                o.x = __byte_perm(h[0], h[1], 0x7531);
                o.y = __byte_perm(h[2], h[3], 0x7531);
                o.z = __byte_perm(h[4], h[5], 0x7531);
                o.w = __byte_perm(h[6], h[7], 0x7531);
                *reinterpret_cast<uint4 *>(dst + (t * NR + r) * 128 + ((u ^ (r & 7)) << 4)) = o;
#pragma unroll
                for (int k = 0; k < 8; ++k) h[k] = less_upper(h[k]);
            }
        } else {
            unsigned char *row = dst + (u >> 2) * NR * 128 + r * 128;
            const int c = 2 * (u & 3);
            *reinterpret_cast<uint4 *>(row + ((c ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(row + (((c + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
    // written by this thread (generic proxy), read by the tensor cores (async proxy)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return true;
}

// The thread's number, as the compiler has not seen it: what follows from it is computed where it is
// needed and takes no register before.
__device__ __forceinline__ int thread_again()
{
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    return t;
}

template <bool E8, int NR>
__global__ void __launch_bounds__(kThreads, 1)
dense_few_kernel(const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                 const KvView kv, const SeqView sv, const WorkShape ws, int box_rows,
                 const __nv_bfloat16 *__restrict__ q, int64_t ld_q, int H_q, uint32_t inv_g, float scale_log2,
                 float q_sign, __nv_bfloat16 *__restrict__ out, float *__restrict__ lse, float *__restrict__ partial,
                 Split *__restrict__ splits, int by_item, const WaitCtl wc)
{
    using F = Few<E8, NR>;
    constexpr int kStages = F::kStages;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *sP = ring + (size_t)kStages * F::kStage;  // [group]
    unsigned char *sQ = sP + kGroups * F::kPBytes;                 // [part & 1]
    Bars &bars = *reinterpret_cast<Bars *>(sQ + 2 * F::kQBytes);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, as the compiler sees it
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
            mbar_init(&bars.raw[s], 1);
        }
        for (int g = 0; g < kGroups; ++g) {
            mbar_init(&bars.s_full[g], 1);
            mbar_init(&bars.p_full[g], 4);
            mbar_init(&bars.o_full[g], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.q_full[b], kAuxWarps);
            mbar_init(&bars.q_free[b], 1);
        }
        mbar_init(&bars.drain, 1);
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars.part_full[i], 1);
        for (int i = 0; i < kSlots; ++i) bars.odd[i] = bars.bad[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    QSA_AFTER_WAIT(q);
    pdl_trigger();

    Parts p;
    int64_t per;
    p.n = 0;
    if (!by_item && tid == 0) splits[blockIdx.x].s = -1;
    if (!work_share(sv, ws, blockIdx.x, gridDim.x, per, p.x, p.x1, p.it)) return;
    p.set(kv, sv, ws);
    if (p.tile1 <= p.tile0) {  // only places without a tile
        --p.n;
        if (!p.next(kv, sv, ws)) return;
    }

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars.tmem)),
                     "r"(F::kTmem)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        bars.part[0] = p;
        mbar_arrive(&bars.part_full[0]);  // (part 8 is its second)
        bars.per = per;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = bars.tmem;
    const int G = H_q / kv.H_kv;
    bool ok = true;
    // tensor memory: S of every group, then O of every group
    if (warp == kMmaWarp) {
        // ---- MMA issue (all lanes walk, one issues)
        const uint32_t lead = elect_leader();
        constexpr uint32_t id_s = E8 ? idesc_f8_m128(F::kCols, false, false) : idesc_m128(F::kCols, false);
        constexpr uint32_t id_o =
            E8 ? idesc_f8_m128(F::kCols, true, true) : idesc_m128(F::kCols, true) | (1u << 15);
        const uint64_t dk0 = desc_kmajor_sw128(smem_u32(ring));
        const uint64_t dv0 = desc_mnmajor_sw128(smem_u32(ring), kHalf);
        const uint64_t dq0 = desc_kmajor_sw128(smem_u32(sQ));
        const uint64_t dp0 = desc_mnmajor_sw128(smem_u32(sP), kHalf);
        // a stage, buffer or k step moves only the descriptors' start address (16-byte units, below
        // 2^14: the add does not carry out of the field)
        auto mma_s = [&](int g, int st, int buf) {
            const uint64_t dk = dk0 + (((uint32_t)st * F::kStage) >> 4), dq = dq0 + (((uint32_t)buf * F::kQBytes) >> 4);
            if constexpr (E8) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_m128_f8_ss_lead(tmem + (uint32_t)g * F::kStride, dk + 2 * k, dq + 2 * k, id_s, k ? 1u : 0u,
                                         lead);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    umma_m128_ss_lead(tmem + (uint32_t)g * F::kStride,
                                      dk + (((uint32_t)(k >> 2) * kHalf) >> 4) + 2 * (k & 3),
                                      dq + (((uint32_t)(k >> 2) * NR * 128) >> 4) + 2 * (k & 3), id_s, k ? 1u : 0u,
                                      lead);
            }
        };
        auto mma_o = [&](int g, int st, bool first) {
            const uint64_t dv = dv0 + (((uint32_t)st * F::kStage) >> 4), dp = dp0 + (((uint32_t)g * F::kPBytes) >> 4);
            const uint32_t d = tmem + (uint32_t)(kGroups + g) * F::kStride;
            if constexpr (E8) {
#pragma unroll
                for (int k = 0; k < kN / 32; ++k)
                    umma_m128_f8_ss_lead(d, dv + k * (4096 >> 4), dp + k * (4096 >> 4), id_o, (!first || k) ? 1u : 0u,
                                         lead);
            } else {
#pragma unroll
                for (int k = 0; k < kN / 16; ++k)
                    umma_m128_ss_lead(d, dv + k * (2048 >> 4), dp + k * (2048 >> 4), id_o, (!first || k) ? 1u : 0u,
                                      lead);
            }
        };
        uint32_t nk = 0, nv = 0, np = 0;  // K and V tiles so far; bit g: the phase of p_full[g]
        // (the stage of K or V tile i, once it is filled)
        auto k_ready = [&](uint32_t i) {
            return bar_wait(&bars.full[i % F::kOfK], (i / F::kOfK) & 1u, wc.limit_ns);
        };
        auto v_ready = [&](uint32_t i) {
            return bar_wait(&bars.full[F::kOfK + i % F::kOfV], (i / F::kOfV) & 1u, wc.limit_ns);
        };
        auto products_s = [&](int g, int buf) {
            ok = k_ready(nk);
            if (!ok) return;
            const int st = (int)(nk % F::kOfK);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            mma_s(g, st, buf);
            umma_commit_lead(&bars.s_full[g], lead);
            umma_commit_lead(&bars.empty[st], lead);
            ++nk;
        };
        do {
            const int tiles = p.tile1 - p.tile0, buf = p.n & 1;
            ok = bar_wait(&bars.q_full[buf], (uint32_t)(p.n >> 1) & 1u, wc.limit_ns);
            const int head = min(kGroups, tiles);
            for (int t = 0; ok && t < head; ++t) products_s(t, buf);
            if (!ok) break;
            if (tiles <= kGroups) umma_commit_lead(&bars.q_free[buf], lead);
            for (int t = 0; t < tiles; ++t) {
                const int g = t % kGroups;
                const int st = F::kOfK + (int)(nv % F::kOfV);
                ok = v_ready(nv) && bar_wait(&bars.p_full[g], (np >> g) & 1u, wc.limit_ns);
                if (!ok) break;
                ++nv;
                np ^= 1u << g;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                mma_o(g, st, t < kGroups);
                umma_commit_lead(&bars.empty[st], lead);
                if (t + kGroups < tiles) {
                    products_s(g, buf);
                    if (!ok) break;
                    if (t + kGroups + 1 == tiles) umma_commit_lead(&bars.q_free[buf], lead);
                } else {
                    umma_commit_lead(&bars.o_full[g], lead);
                }
            }
        } while (ok && p.next(kv, sv, ws));
        // every MMA issued has completed before the tensor memory is freed
        umma_commit_lead(&bars.drain, lead);
        if (!mbar_wait(&bars.drain, 0)) ok = false;
        __syncwarp();
    } else if (warp >= kLoadWarp && warp < kAuxWarp) {
        // ---- K tiles by one warp, V tiles by the other: box b of a tile is box_rows cells, by lane b
        const bool is_v = warp != kLoadWarp;
        const CUtensorMap *map = is_v ? &mapV : &mapK;
        const int boxes = kN / box_rows, first = is_v ? F::kOfK : 0, of = is_v ? F::kOfV : F::kOfK;
        uint32_t n = 0, edge_last = 0, raw_phase = 0;  // tiles so far; bits by stage
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
            for (int t = p.tile0; ok && t < p.tile1; ++t, ++n) {
                const int row = ahead[0].row(kv, p);
                ahead[0] = ahead[1];
                ahead[1] = look(t + 2);
                const uint32_t go = __ballot_sync(0xffffffffu, row >= 0);
                if (!is_v) {
                    if (__any_sync(0xffffffffu, row == -1) && lane == 0)
                        *reinterpret_cast<volatile int32_t *>(&bars.bad[p.n % kSlots]) = p.n + 1;
                    if (E8 && row >= 0) {
                        // the lines of the box's exponents, to L2
                        const int64_t at = (int64_t)row * kv.H_kv + p.it.g;
                        const int bytes = (box_rows - 1) * kv.H_kv;
                        for (int o = 0; o < bytes + 128; o += 128) {
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(kv.K_exp + at + min(o, bytes)));
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(kv.V_exp + at + min(o, bytes)));
                        }
                    }
                }
                const int i = (int)(n % of), s = first + i;
                if (n >= (uint32_t)of && !bar_wait_warp(&bars.empty[s], ((n / of) - 1) & 1u, wc.limit_ns)) {
                    ok = false;
                    break;
                }
                const bool edge = is_v && p.edge(t);
                uint64_t *bar = edge ? &bars.raw[s] : &bars.full[s];
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)__popc(go) * (uint32_t)box_rows * (E8 ? 128u : 256u));
                edge_last = edge ? edge_last | (1u << i) : edge_last & ~(1u << i);
                if (edge) raw_phase ^= 1u << i;
                __syncwarp();
                if (row >= 0) {
                    const uint32_t dst = smem_u32(ring) + (uint32_t)s * F::kStage + (uint32_t)(lane * box_rows) * 128;
                    tma_box(dst, map, p.it.g * kD, row, bar);
                    if constexpr (!E8) tma_box(dst + kHalf, map, p.it.g * kD + 64, row, bar);
                }
            }
        } while (ok && p.next(kv, sv, ws));
        // every copy issued has landed before the CTA may leave (a stage's earlier copies landed before
        // it was used again)
        if (lane == 0) {
            for (uint32_t k = n > (uint32_t)of ? n - of : 0; k < n; ++k) {  // a stage's last tile
                const int i = (int)(k % of), s = first + i;
                const bool done = (edge_last >> i) & 1u ? mbar_wait(&bars.raw[s], ((raw_phase >> i) & 1u) ^ 1u)
                                                       : mbar_wait(&bars.full[s], (k / of) & 1u);
                if (!done) ok = false;
            }
        }
        __syncwarp();
    } else if (warp >= kAuxWarp) {
        const int aux = warp - kAuxWarp;
        Parts ahead = p;
        uint32_t nv = 0, raw_phase = 0;  // V tiles so far
        bool more;
        do {
            __syncwarp();
            if (lane == 0) bars.now[aux] = ahead;
            __syncwarp();
            const volatile Parts &now = bars.now[aux];
            more = ahead.next(kv, sv, ws);
            if (aux == 0 && lane == 0) {
                bars.part[ahead.n % kSlots] = ahead;
                bars.more[ahead.n % kSlots] = more;
                mbar_arrive(&bars.part_full[ahead.n % kSlots]);
            }
            if (more) {
                // (the first part's are the softmax warps' work)
                const int buf = ahead.n & 1;
                if (ok && ahead.n >= 2)
                    ok = bar_wait_warp(&bars.q_free[buf], (uint32_t)((ahead.n >> 1) - 1) & 1u, wc.limit_ns);
                if (lay_queries<E8, NR, 32 * kAuxWarps, kBarAux>(ahead, aux * 32 + lane, ok, q, ld_q, G, inv_g, q_sign,
                                                                 sQ + (size_t)buf * F::kQBytes, bars.qs[ahead.n % kSlots])) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.q_full[buf]);
                } else {
                    ok = false;
                }
            }
            // ---- V tiles in which some row does not see some cell: values of cells that no row sees
            // become zero, and so do infinities and NaN of cells that only some rows see; the epilogue
            // adds those
            const int tiles = now.tile1 - now.tile0;
            for (int t = 0; ok && t < tiles; ++t) {
                const int c0 = (now.tile0 + t) * kN;  // the tile's first cell
                if (c0 + kN - 1 <= now.pos0) continue;
                const int i = (int)((nv + (uint32_t)t) % F::kOfV), s = F::kOfK + i;
                const bool here = bar_wait_warp(&bars.raw[s], (raw_phase >> i) & 1u, wc.limit_ns);
                if (named_or<32 * kAuxWarps>(kBarAux, !here)) {
                    ok = false;
                    break;
                }
                raw_phase ^= 1u << i;
                unsigned char *tile = ring + (size_t)s * F::kStage;
                const int r0 = max(0, now.pos0 + 1 - c0), r1 = now.n_see - c0;
                const bool odd = E8 ? scrub_codes(tile, r0, r1, 4 * aux, 4 * kAuxWarps)
                                    : scrub_tile(tile, r0, r1, 2 * aux, 2 * kAuxWarps);
                if (odd) *reinterpret_cast<volatile int32_t *>(&bars.odd[now.n % kSlots]) = now.n + 1;
                // written by this warp (generic proxy), read by the tensor cores (async proxy)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                named_sync<32 * kAuxWarps>(kBarAux);
                if (aux == 0 && lane == 0) mbar_arrive(&bars.full[s]);
            }
            nv += (uint32_t)tiles;
            // (one that gave up tells nothing more: it would overtake those who read)
        } while (ok && more);
        __syncwarp();
    } else {
        // ---- weights: this thread's cell is number r of every tile of group g
        const int g = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t colS = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)g * F::kStride;
        unsigned char *const prow = sP + (size_t)g * F::kPBytes + r * 128;
        uint32_t waits = 0;  // bit 0, 1: the phase of s_full, o_full
        // e4m3: the exponents of this group's tile, and the page of its next one's cell.  They are on their
        // way while the logits are (the copies' warp had them brought to L2); those of a part's first tile
        // while the part before ends.
        uint32_t ke1 = kExpBias, ve1 = kExpBias;
        PageAhead ahead = {0, -1};
        auto look = [&](const Parts &w, int k) {
            const int at = w.tile0 + kGroups * k + g;
            ahead.load(kv, w, at < w.tile1, (int64_t)at * kN + r);
        };
        auto fetch = [&](const Parts &w) {
            const int row = ahead.row(kv, w);
            ke1 = ve1 = kExpBias;
            if (row >= 0) {
                ke1 = kv.K_exp[(int64_t)row * kv.H_kv + w.it.g];
                ve1 = kv.V_exp[(int64_t)row * kv.H_kv + w.it.g];
            }
        };
        if constexpr (E8) look(p, 0);
        if (tid < NR * 8) {
            lay_queries<E8, NR, NR * 8, kBarFirst>(p, tid, true, q, ld_q, G, inv_g, q_sign, sQ, bars.qs[0]);
            named_sync<NR * 8>(kBarFirst);
            if (tid == 0) mbar_arrive_n(&bars.q_full[0], kAuxWarps);
        }
        if constexpr (E8) fetch(p);
        // the part is read where it lies: its fields would take the registers that the weights need
        int n = 0;
        bool alone = false;  // some wait gave up: the parts are looked up here, into places of their own
        do {
            const Parts &p = alone ? bars.alone[n & 1] : bars.part[n % kSlots];
            const int tiles = p.tile1 - p.tile0, mine = (tiles + kGroups - 1 - g) / kGroups;
            bool told;
            float l[NR];
#pragma unroll
            for (int c = 0; c < NR; ++c) l[c] = 0.0f;
            // (row r of the group: one thread's, here and where it moves)
            const bool keeper = r < NR;
            if (keeper) {
                bars.mref[g][r] = -INFINITY;
                bars.nm[g][r] = kUnset;
            }
            const float *nm = bars.nm[g];
            for (int k = 0; ok && k < mine; ++k) {
                const int t = p.tile0 + kGroups * k + g;
                const float *qs = bars.qs[n % kSlots];
                if constexpr (E8) {
                    if (k > 0) fetch(p);
                    look(p, k + 1);
                }
                bool here = bar_wait_warp(&bars.s_full[g], waits & 1u, wc.limit_ns);
                waits ^= 1u;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                float ks = scale_log2, vs = 0.0f, vi = 1.0f;
                bool far = false;
                if constexpr (E8) {
                    const int ke = min(max((int)ke1 - kExpBias, kExpMin), kExpMax);
                    const int ve = min(max((int)ve1 - kExpBias, kExpMin), kExpMax);
                    ks = two_to(ke) * scale_log2;
                    vs = (float)ve;
                    vi = two_to(-ve);
                    far = __any_sync(0xffffffffu, abs(ve) > kFar);
                }
                // the logits in log2 units (e4m3: with the exponent of the cell's values)
                float v[NR];
                constexpr int kStep = 8;  // columns of a term loaded together (16: 104.5 us instead of 99.2, registers)
                auto logits = [&]() {
                    const float2 k2 = make_float2(ks, ks), v2 = make_float2(vs, vs);
#pragma unroll
                    for (int at = 0; at < NR; at += kStep) {
                        float x[F::kTerms * kStep];
#pragma unroll
                        for (int i = 0; i < F::kTerms; ++i)
                            tmem_ld_async<kStep>(colS + (uint32_t)(i * NR + at), x + i * kStep);
                        tmem_wait_ld<F::kTerms * kStep>(x);
#pragma unroll
                        for (int c = 0; c < kStep; c += 2) {
                            float2 y = make_float2(x[c], x[c + 1]);
                            if constexpr (E8) {
                                y = add2(y, add2(make_float2(x[kStep + c], x[kStep + c + 1]), make_float2(x[2 * kStep + c], x[2 * kStep + c + 1])));
                                y = fma2(y, mul2(k2, *reinterpret_cast<const float2 *>(qs + at + c)), v2);
                            } else {
                                y = mul2(y, k2);
                            }
                            v[at + c] = y.x;
                            v[at + c + 1] = y.y;
                        }
                    }
                    if (p.edge(t)) {
                        const int64_t j = (int64_t)t * kN + r;
                        // the first row that sees cell j
                        const int c0 = j >= p.n_see ? NR : (ws.causal && j > p.pos0 ? (int)(j - p.pos0) * G : 0);
#pragma unroll
                        for (int c = 0; c < NR; ++c) v[c] = c >= c0 ? v[c] : -INFINITY;
                    }
                };
                // the weights relative to the references as they stand, in fp32 and as 16-bit pairs, whose
                // maximum says whether they may stay
                uint32_t h[NR / 2];
                uint32_t most;
                auto weights = [&]() {
                    most = 0;
#pragma unroll
                    for (int c = 0; c < NR; c += 4) {
                        const float4 m4 = *reinterpret_cast<const float4 *>(nm + c);
                        const float2 a0 = add2(make_float2(v[c], v[c + 1]), make_float2(m4.x, m4.y));
                        const float2 a1 = add2(make_float2(v[c + 2], v[c + 3]), make_float2(m4.z, m4.w));
                        v[c] = ex2_approx(a0.x);
                        v[c + 1] = ex2_approx(a0.y);
                        v[c + 2] = ex2_approx(a1.x);
                        v[c + 3] = ex2_approx(a1.y);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            uint32_t &u = h[(c + e) / 2];
                            if constexpr (E8) {
                                const __half2 x = __floats2half2_rn(v[c + e], v[c + e + 1]);
                                u = reinterpret_cast<const uint32_t &>(x);
                                const __half2 y = __hmax2(reinterpret_cast<const __half2 &>(most), x);
                                most = reinterpret_cast<const uint32_t &>(y);
                            } else {
                                u = pack_bf16(v[c + e], v[c + e + 1]);
                                const __nv_bfloat162 y = __hmax2(reinterpret_cast<const __nv_bfloat162 &>(most),
                                                                 reinterpret_cast<const __nv_bfloat162 &>(u));
                                most = reinterpret_cast<const uint32_t &>(y);
                            }
                        }
                    }
                };
                logits();
                bool move = k == 0;  // a part's first tile sets the references
                if (k > 0) {
                    weights();
                    if constexpr (E8) {
                        const float2 x = __half22float2(reinterpret_cast<const __half2 &>(most));
                        move = fmaxf(x.x, x.y) > F::kMost;
                    } else {
                        move = fmaxf(__uint_as_float(most << 16), __uint_as_float(most & 0xffff0000u)) > F::kMost;
                    }
                    move = named_or<128>(kBarVote + g, move || !here);
                }
                if (move) {
                    if (named_or<128>(kBarVote + g, !here)) {
                        ok = false;
                        break;
                    }
                    // ---- the references move
                    if (k > 0) logits();
                    const int tid = thread_again(), lane = tid & 31, quarter = (tid >> 5) & 3;
                    const uint32_t colO = tmem + ((uint32_t)(quarter * 32) << 16) + kGroups * F::kStride;
#pragma unroll
                    for (int c = 0; c < NR; c += 4) {
                        const float4 m4 = make_float4(lane_max(v[c]), lane_max(v[c + 1]), lane_max(v[c + 2]),
                                                      lane_max(v[c + 3]));
                        if (lane == 0) *reinterpret_cast<float4 *>(&bars.red[g][quarter][c]) = m4;
                    }
                    named_sync<128>(kBarVote + g);
                    if (keeper) {
                        const float m = bars.mref[g][r];
                        const float top = fmaxf(fmaxf(bars.red[g][0][r], bars.red[g][1][r]),
                                                fmaxf(bars.red[g][2][r], bars.red[g][3][r]));
                        float2 f = make_float2(1.0f, 1.0f);
                        // (of a row whose weights may stay, a little more room does no harm)
                        const float mn = ceilf(top) - F::kTop;
                        if (mn > m) {
                            if (m != -INFINITY) f = two_factors(m - mn);
                            bars.mref[g][r] = mn;
                            bars.nm[g][r] = -mn;
                        }
                        bars.al[g][r] = f;
                    }
                    named_sync<128>(kBarVote + g);
                    if (k > 0) {
#pragma unroll
                        for (int c = 0; c < NR; ++c) {
                            const float2 f = bars.al[g][c];
                            l[c] = l[c] * f.x * f.y;
                        }
                        // s_full follows this group's last product with V: o may be rescaled
#pragma unroll 1
                        for (int i = 0; i < NR / 8 * F::kTerms; ++i) {
                            const int c = 8 * (i % (NR / 8));
                            const uint32_t at = colO + (uint32_t)g * F::kStride + (uint32_t)(i / (NR / 8) * NR + c);
                            float o[8];
                            tmem_ld8_async(at, o);
                            tmem_wait_ld<8>(o);
                            uint32_t ou[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 f = bars.al[g][c + e];
                                ou[e] = __float_as_uint(o[e] * f.x * f.y);
                            }
                            tmem_st8(at, ou);
                        }
                        tmem_wait_st();
                    }
                    weights();
                }
                // ---- their sum, and their terms for the product
#pragma unroll
                for (int c = 0; c < NR; c += 2) {
                    float2 s2 = make_float2(l[c], l[c + 1]);
                    const float2 w2 = make_float2(v[c], v[c + 1]);
                    if constexpr (E8) {
                        if (!far) s2 = fma2(w2, make_float2(vi, vi), s2);
                    } else {
                        s2 = add2(s2, w2);
                    }
                    l[c] = s2.x;
                    l[c + 1] = s2.y;
                }
                if constexpr (E8) {
#pragma unroll
                    for (int c = 0; c < NR / 2; ++c) h[c] = (h[c] + 0x00020002u) & 0xfffcfffcu;  // nine bits
                    constexpr int kChunks = NR / 16;
                    #pragma unroll
                    for (int i = 0; i < 3; ++i) {
#pragma unroll
                        for (int ch = 0; ch < kChunks; ++ch) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                w[e] = __byte_perm(h[8 * ch + 2 * e], h[8 * ch + 2 * e + 1], 0x7531);
                            *reinterpret_cast<uint4 *>(prow + (((i * kChunks + ch) ^ (r & 7)) << 4)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        if (i < 2) {
#pragma unroll
                            for (int c = 0; c < NR / 2; ++c) h[c] = less_upper_grown(h[c]);
                        }
                    }
                    if (far) {
                        logits();
#pragma unroll
                        for (int c = 0; c < NR; ++c) l[c] += ex2_approx(v[c] - vs + nm[c]);
                    }
                } else {
#pragma unroll
                    for (int ch = 0; ch < NR / 8; ++ch)
                        *reinterpret_cast<uint4 *>(prow + ((ch ^ (r & 7)) << 4)) =
                            make_uint4(h[4 * ch], h[4 * ch + 1], h[4 * ch + 2], h[4 * ch + 3]);
                }
                // written by this thread (generic proxy), read by the tensor cores (async proxy)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[g]);
            }
            {
            // ---- the part's result: every group to the common reference R of a row.  On e4m3 cells a sum
            // (of 2^(x - m), in which V's exponent may be anything in +-100) is taken 2^30 smaller, so that
            // it stays between 2^-123 and 2^83 times the cells.
            constexpr float kLess = E8 ? 30.0f : 0.0f;
            const int tid = thread_again(), lane = tid & 31, warp = tid >> 5;
            const int g = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
            if constexpr (E8) {
#pragma unroll
                for (int c = 0; c < NR; ++c) l[c] *= 1.0f / (1 << 30);
            }
            {
                const float cm = col_sum(l);
                if (lane < NR) bars.sum[g][quarter][lane] = cm;
            }
            if (ok && mine > 0) {
                if (!bar_wait_warp(&bars.o_full[g], waits >> 1, wc.limit_ns)) ok = false;
                waits ^= 2u;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            // the next part as the query warps found it (its own look-up is a chain of loads)
            const int slot = (n + 1) % kSlots;
            const bool here = !alone && bar_wait_warp(&bars.part_full[slot], (uint32_t)((n + 1) / kSlots) & 1u, wc.limit_ns);
            told = !named_or<32 * kSoftWarps>(kBarAll, !ok || !here);
            ok = ok && told;
            if (E8 && told && bars.more[slot]) look(bars.part[slot], 0);
            const bool starts = p.tile0 == 0, ends = p.tile1 == p.it.tiles, whole = starts && ends;
            float *rec = partial + (2 * (int64_t)blockIdx.x + (starts ? 1 : 0)) * partial_floats(NR, kD);
            if (tid < NR) {
                float R = bars.mref[0][tid], s = 0.0f;
#pragma unroll
                for (int i = 1; i < kGroups; ++i) R = fmaxf(R, bars.mref[i][tid]);
                R += kLess;
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const float m = bars.mref[i][tid];
                    const float2 f = m == -INFINITY ? make_float2(0.0f, 0.0f) : two_factors(m - R);
                    bars.fac[i][tid] = f;
                    const float part = (bars.sum[i][0][tid] + bars.sum[i][1][tid]) +
                                       (bars.sum[i][2][tid] + bars.sum[i][3][tid]);
                    s += part * f.x * (E8 ? (float)(1 << 30) : 1.0f) * f.y;
                }
                if (!ok || !p.fits || *reinterpret_cast<volatile int32_t *>(&bars.bad[n % kSlots]) == n + 1) s = NAN;
                const int tok = (int)((uint32_t)tid * inv_g >> 16);
                const int64_t at = tid < p.toks * G ? (p.t0 + p.tok0 + tok) * H_q + p.it.g * G + tid - tok * G : -1;
                bars.at[tid] = at;
                bars.see[tid] = min(ws.causal ? p.pos0 + tok : p.cells - 1, p.n_see - 1);
                bars.inv[tid] = !whole ? 1.0f : (s > 0.0f ? 1.0f / s : (s == 0.0f ? 0.0f : s));
                if (at >= 0) {
                    if (!whole) {
                        rec[tid] = R;
                        rec[NR + tid] = s;
                    } else if (lse) {
                        lse[at] = s == 0.0f ? -INFINITY : (R + log2f(s)) * kLn2;
                    }
                }
            }
            named_sync<32 * kSoftWarps>(kBarAll);
            if (E8 && told && bars.more[slot]) fetch(bars.part[slot]);
            // dim r of the rows c0 .. c0 + kRows - 1
            constexpr int kRows = NR / kGroups;
            const int c0 = (warp >> 2) * kRows;
            const bool odd = ok && *reinterpret_cast<volatile int32_t *>(&bars.odd[n % kSlots]) == n + 1;
            float o[kRows];
#pragma unroll
            for (int c = 0; c < kRows; ++c) o[c] = 0.0f;
            if (ok) {
#pragma unroll 1
                for (int i = 0; i < kGroups && i < tiles; ++i) {
                    const uint32_t col = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(kGroups + i) * F::kStride +
                                         (uint32_t)c0;
                    float x[F::kTerms * kRows];
#pragma unroll
                    for (int j = 0; j < F::kTerms; ++j) tmem_ld_async<kRows>(col + (uint32_t)(j * NR), x + j * kRows);
                    tmem_wait_ld<F::kTerms * kRows>(x);
#pragma unroll
                    for (int c = 0; c < kRows; ++c) {
                        const float2 f = bars.fac[i][c0 + c];
                        float y = x[c];
                        if constexpr (E8) y = fmaf(fmaf(x[2 * kRows + c], 0.125f, x[kRows + c]), 0.125f, y);
                        o[c] += y * f.x * f.y;
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
#pragma unroll 1
            for (int c = 0; odd && c < kRows; ++c) {
                const int to = min(bars.see[c0 + c], p.tile1 * kN - 1);
                float y = 0.0f;
                for (int j = max(p.pos0 + 1, p.tile0 * kN); j <= to; ++j) {
                    const int64_t row = cell_row(kv, p.it.s, p.t0, j);
                    if (row >= 0) y += odd_value_at<E8>(kv, row * kv.ld_v + (int64_t)p.it.g * kD + r);
                }
#pragma unroll
                for (int e = 0; e < kRows; ++e) o[e] += e == c ? y : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < kRows; ++c) {
                const int64_t at = bars.at[c0 + c];
                if (at < 0) continue;
                if (whole) out[at * kD + r] = __float2bfloat16_rn(o[c] * bars.inv[c0 + c]);
                else rec[2 * NR + (int64_t)(c0 + c) * kD + r] = o[c];
            }
            if (starts && tid == 0)
                note_split(splits, by_item, p.it, ends, div_pos(p.it.start + ws.over + p.it.tiles - 1, bars.per));
            }
            // behind this barrier no group's output is read any more: its next weights let it be written
            named_sync<32 * kSoftWarps>(kBarAll);
            const int slot = (n + 1) % kSlots;
            if (!told) {
                Parts next = p;
                const bool more = next.next(kv, sv, ws);
                if (tid == 0) bars.alone[(n + 1) & 1] = next;
                named_sync<32 * kSoftWarps>(kBarAll);
                alone = true;
                if (!more) break;
            } else if (!bars.more[slot]) {
                break;
            }
            ++n;
        } while (true);
    }

    if (!ok) report_timeout(wc);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::kTmem)
                     : "memory");
}

constexpr int kMaxCtas = kTargetSMs;

template <bool E8, int NR>
qsa_status run_few(const DenseArgs &a, void *workspace, cudaStream_t st)
{
    using F = Few<E8, NR>;
    const int G = a.H_q / a.kv.H_kv;
    const int page = 1 << a.kv.page_shift;
    const int box_rows = a.kv.table && page < kN ? page : kN;
    CUtensorMap mk, mv;
    const int64_t width = (int64_t)a.kv.H_kv * kD;
    if (!make_map(&mk, a.kv.K, a.pool_rows, width, a.kv.ld_k, box_rows, E8, true) ||
        !make_map(&mv, a.kv.V, a.pool_rows, width, a.kv.ld_v, box_rows, E8, true))
        return QSA_ERR_CUDA;
    const WorkShape ws = work_shape(a, NR / G, kN, F::kOver);
    // the kernel takes a positive scale: a negative one turns the queries' signs, zero clears them
    const float scale = (a.scale == 0.0f ? 1.0f : fabsf(a.scale)) * kLog2e;
    const float q_sign = a.scale == 0.0f ? 0.0f : (a.scale < 0.0f ? -1.0f : 1.0f);
    constexpr size_t smem = few_smem<E8, NR>();
    if (ensure_kernel_attrs<dense_few_kernel<E8, NR>>(smem) != cudaSuccess) return QSA_ERR_CUDA;
    int ctas = device_sm_count();
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    Split *splits = static_cast<Split *>(workspace);
    float *partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + kMaxCtas * sizeof(Split));
    cudaError_t e = launch(dense_few_kernel<E8, NR>, dim3((unsigned)ctas), dim3(kThreads), smem, st, 1, mk, mv, a.kv,
                           a.sv, ws, box_rows, static_cast<const __nv_bfloat16 *>(a.q), a.ld_q, a.H_q, 65536u / (uint32_t)G + 1u, scale, q_sign,
                           static_cast<__nv_bfloat16 *>(a.out), a.lse, partial, splits,
                           (int)join_by_item(a, ws.rt, ctas), current_wait_ctl());
    if (e == cudaSuccess) e = launch_dense_join<__nv_bfloat16>(splits, partial, ctas, NR, ws.rt, a, st);
    return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

}  // namespace

bool dense_few_ok(const DenseArgs &a, int64_t max_q)
{
    const int G = a.H_q / a.kv.H_kv;
    const bool e8 = a.kv_dtype == QSA_E4M3;
    // (a TMA map's strides are multiples of 16 bytes, and below 2^40)
    if (a.kv.ld_k > kMaxStride || a.kv.ld_v > kMaxStride) return false;
    if (a.d != kD || a.q_dtype != QSA_BF16 || (!e8 && a.kv_dtype != QSA_BF16) || a.pool_rows <= 0 ||
        a.pool_rows > 0x7fffffffLL || (e8 && (a.kv.ld_k % 16 || a.kv.ld_v % 16)))
        return false;
    if (G > 32 || max_q * G > (e8 ? 64 : 32)) return false;
    // (e4m3: two row tiles read the cells twice and still beat the 128-row kernel, whose conversion bounds
    // it: 64 sequences of up to 8,000 cells, 64 rows, 142 us here and 243 there; bf16, 32 rows, 103 and 124)
    if (max_q * G > 16) return true;
    // Up to 16 rows over short contexts are dense_decode.cu's: a part costs more here, a cell less.  By what
    // the host knows, the most cells a sequence may have; measured there and here (us, one token, replayed
    // from a graph): bf16, one sequence of 4,000 cells and 2 KV heads 13.7 and 14.9, of 8,000 17.3 and 17.1,
    // eight of up to 2,050 and 4 KV heads 18.0 and 15.9, 64 of up to 500 and 2 18.6 and 20.0, of up to
    // 1,000 23.0 and 21.9; e4m3, one of 8,000 and 2 15.7 and 18.3, of 16,000 20.2 and 18.0, eight of up to
    // 8,000 20.0 and 18.1, 64 of up to 500 and 4 24.5 and 27.0, of up to 1,000 and 2 23.1 and 22.4.
    const int64_t cells = a.kv.table ? a.kv.ld_table << a.kv.page_shift : a.sv.n_tok;
    return cells >= (e8 ? 10240 : 6144) ||
           (cells >= 1024 && (double)cells * (double)a.sv.n_seq * a.kv.H_kv >= (e8 ? 1e5 : 6e4));
}

size_t dense_few_workspace()
{
    return kMaxCtas * sizeof(Split) + (size_t)2 * kMaxCtas * partial_floats(32, kD) * sizeof(float);
}

qsa_status launch_dense_few(const DenseArgs &a, int64_t max_q, void *workspace, cudaStream_t st)
{
    const int G = a.H_q / a.kv.H_kv;
    const bool small = G <= 16 && max_q * G <= 16;
    if (a.kv_dtype == QSA_E4M3)
        return small ? run_few<true, 16>(a, workspace, st) : run_few<true, 32>(a, workspace, st);
    return small ? run_few<false, 16>(a, workspace, st) : run_few<false, 32>(a, workspace, st);
}

}  // namespace qsa
