// draft_verify.cu -- verification of drafted tokens against the target's probabilities.
//
// Sequence s drafted tokens t_0 .. t_{n-1} from the rows q_j of its draft; the target gave the
// rows p_0 .. p_n.  Draft j is taken while u_j * q_j(t_j) < p_j(t_j) (that is, with probability
// min(1, p / q)); the number taken is a.  The next token comes from the weights
// w = max(p_a - q_a, 0) when draft a was refused and from w = p_n when all were taken: it is the
// first index whose running sum of w passes u_n' * sum(w), u_n' the sequence's last number.
// Taking with min(1, p/q) and drawing the refused mass from the difference leaves the tokens
// distributed as the target's.
//
// The product u * q is exact in 64 bits.  A running sum over a vocabulary in 32 bits would move
// the draw past small weights, so sums are kept as unevaluated pairs of 32-bit numbers (two-sum:
// the error of each addition is itself a 32-bit number) and joined in 64 bits; the difference
// p - q is carried the same way.  FP64 adds are scarce on this GPU (a few per SM and clock), the
// pairs cost six 32-bit adds each and hide behind the loads.
//
// One thread-block cluster per sequence: every CTA decides a itself (a few gathers), sums its
// slice of the row(s), and the warps of the CTA that holds the drawn point scan, a chunk each, the
// slice of the one warp that holds it (64 sequences, vocabulary of 131,072: 23.0 us; 31.7 with one
// warp scanning).  One launch, no workspace, no atomics: the same result every time.  Bound by one
// pass over one or two rows (10 of the 23.0 us, at the copy bandwidth) and the chain around it:
// token -> gather -> row, the cluster's barrier, the chunk.
#include <cooperative_groups.h>

#include "dense.cuh"
#include "draft_verify.cuh"

namespace qsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kChunk = 128;  // values a warp takes at once

// s + x as a pair: s the rounded sum, the rounding error added to c.
__device__ __forceinline__ void add_pair(float &s, float &c, float x)
{
    const float t = __fadd_rn(s, x);
    const float b = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(x, b)));
    s = t;
}

// A probability of the draft's: what is negative or NaN counts as 0.  (The target's needs no such step: with
// q >= 0 a p that is negative or NaN passes no comparison below.)
__device__ __forceinline__ float draft_prob(float q) { return fmaxf(q, 0.0f); }

// Weight of one index: max(p - q, 0) as a pair (d, e), q a draft_prob.
__device__ __forceinline__ void weight_of(float p, float q, float &d, float &e)
{
    d = __fsub_rn(p, q);
    const float b = __fsub_rn(d, p);
    e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
    if (!(d > 0.0f)) d = e = 0.0f;
}

__device__ __forceinline__ double warp_sum_f64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Row {
    const float *p, *q;  // q == NULL: the plain weights p
    int skip;            // index whose weight is 0 (the refused token of a draft without rows)
    __device__ __forceinline__ void weight(float pv, float qv, int64_t i, float &d, float &e) const
    {
        if (q) {
            weight_of(pv, draft_prob(qv), d, e);
        } else {
            d = pv > 0.0f && i != skip ? pv : 0.0f;
            e = 0.0f;
        }
    }
};

// The packed forms of the above: two indices at a time.
__device__ __forceinline__ float2 sub2(float2 a, float2 b)  // a + (-1) b: one rounding, as a - b
{
    return fma2(b, make_float2(-1.0f, -1.0f), a);
}

// Sum of the warp's chunks [c0, c1) of the row's weights; every lane gets it.
__device__ __forceinline__ double slice_sum(const Row &row, int64_t c0, int64_t c1, int64_t vocab, bool vec)
{
    const int lane = threadIdx.x & 31;
    float2 s = make_float2(0.0f, 0.0f), c = make_float2(0.0f, 0.0f);
    auto take = [&](float2 p, float2 q, int64_t i) {
        float2 d = p, e = make_float2(0.0f, 0.0f);
        if (row.q) {
            q = make_float2(draft_prob(q.x), draft_prob(q.y));
            d = sub2(p, q);
            const float2 b = sub2(d, p);
            e = sub2(sub2(p, sub2(d, b)), add2(q, b));
        }
        const bool x = d.x > 0.0f && i != row.skip, y = d.y > 0.0f && i + 1 != row.skip;
        d.x = x ? d.x : 0.0f;
        d.y = y ? d.y : 0.0f;
        e.x = x ? e.x : 0.0f;
        e.y = y ? e.y : 0.0f;
        const float2 t = add2(s, d), b = sub2(t, s);
        c = add2(c, add2(add2(sub2(s, sub2(t, b)), sub2(d, b)), e));
        s = t;
    };
    if (vec) {  // the vocabulary is a multiple of 4, rows are 16-byte aligned
        for (int64_t c_ = c0; c_ < c1; c_ += 4) {
            float4 p[4], q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t i = (c_ + u) * kChunk + 4 * lane;
                const bool on = c_ + u < c1 && i < vocab;
                p[u] = q[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (on) p[u] = *reinterpret_cast<const float4 *>(row.p + i);
                if (on && row.q) q[u] = *reinterpret_cast<const float4 *>(row.q + i);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t i = (c_ + u) * kChunk + 4 * lane;
                take(make_float2(p[u].x, p[u].y), make_float2(q[u].x, q[u].y), i);
                take(make_float2(p[u].z, p[u].w), make_float2(q[u].z, q[u].w), i + 2);
            }
        }
    } else {
        const int64_t end = min(c1 * kChunk, vocab);
        for (int64_t i0 = c0 * kChunk + 2 * lane; i0 < end; i0 += 256) {
            float2 p[4], q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t i = i0 + 64 * u;
                p[u].x = i < end ? row.p[i] : 0.0f;
                p[u].y = i + 1 < end ? row.p[i + 1] : 0.0f;
                q[u].x = row.q && i < end ? row.q[i] : 0.0f;
                q[u].y = row.q && i + 1 < end ? row.q[i + 1] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) take(p[u], q[u], i0 + 64 * u);
        }
    }
    return warp_sum_f64(((double)s.x + (double)s.y) + ((double)c.x + (double)c.y));
}

// First of `n` sums (n <= 32, lane i holds v) whose running sum passes x, and the sum before it;
// -1 when none does.  last: the last positive one.
__device__ __forceinline__ int first_over(double v, int n, double start, double x, double &before, int &last)
{
    const int lane = threadIdx.x & 31;
    if (lane >= n) v = 0.0;
    double incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    const uint32_t pos = __ballot_sync(0xffffffffu, v > 0.0);
    const uint32_t b = __ballot_sync(0xffffffffu, v > 0.0 && start + incl > x);
    last = pos ? 31 - __clz(pos) : -1;
    if (!b) return -1;
    const int j = __ffs(b) - 1;
    before = start + __shfl_sync(0xffffffffu, incl - v, j);
    return j;
}

// What the warps of a CTA tell one another while they look for the drawn point.
struct Search {
    double base, x;     // the sum before the slice, the point
    int64_t c0, c1;     // the slice's chunks; none when another CTA has it
    int end;            // the last weight is asked for, whatever x
    double sum[kWarps];
    int64_t last[kWarps];
};

// The first index of the slice whose running sum passes x; the last positive weight where none does;
// -1 without any.  A chunk a warp, kWarps at a time: returned to the warp that has it, -2 to the others.
__device__ __forceinline__ int64_t slice_find(const Row &row, Search &f, int64_t vocab)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const double x = f.x;
    const bool end = f.end != 0;
    double base = f.base;
    int64_t last = -1;
    for (int64_t cb = f.c0; cb < f.c1; cb += kWarps) {
        const int64_t i0 = (cb + warp) * kChunk + 4 * lane;
        // the lane's four weights and their sum as a pair
        float d[4], e[4], s = 0.0f, c = 0.0f;
        int pos = -1;  // the lane's last positive weight
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const bool on = cb + warp < f.c1 && i0 + k < vocab;
            const float pk = on ? row.p[i0 + k] : 0.0f, qk = on && row.q ? row.q[i0 + k] : 0.0f;
            row.weight(pk, qk, i0 + k, d[k], e[k]);
            if (d[k] > 0.0f) pos = k;
            add_pair(s, c, d[k]);
            c = __fadd_rn(c, e[k]);
        }
        const double sum = (double)s + (double)c, all = warp_sum_f64(sum);
        const uint32_t any = __ballot_sync(0xffffffffu, pos >= 0);
        const int tail = any ? 31 - __clz(any) : 0;
        const int64_t mine = any ? (cb + warp) * kChunk + 4 * tail + __shfl_sync(0xffffffffu, pos, tail) : -1;
        if (lane == 0) {
            f.sum[warp] = all;
            f.last[warp] = mine;
        }
        __syncthreads();
        double before = base;
        int lw;
        const int w = end ? -1 : first_over(lane < kWarps ? f.sum[lane] : 0.0, kWarps, base, x, before, lw);
        if (w >= 0) {
            if (warp != w) return -2;
            double incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const uint32_t b = __ballot_sync(0xffffffffu, pos >= 0 && before + incl > x);
            if (!b) return mine;  // (rounding: the chunk's last)
            const int j = __ffs(b) - 1;  // the lane whose weights pass x
            int hit = pos;
            if (lane == j) {
                double run = before + (incl - sum);
                hit = -1;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    run += (double)d[k] + (double)e[k];
                    if (hit < 0 && d[k] > 0.0f && run > x) hit = k;
                }
                if (hit < 0) hit = pos;
            }
            return (cb + w) * kChunk + 4 * j + __shfl_sync(0xffffffffu, hit, j);
        }
        for (int i = 0; i < kWarps; ++i) {
            base += f.sum[i];
            last = f.last[i] >= 0 ? f.last[i] : last;
        }
        __syncthreads();  // before the next turn's sums
    }
    return warp == 0 ? last : -2;
}

__global__ void __launch_bounds__(kThreads, 2)
draft_verify_kernel(const float *__restrict__ target, int64_t ld_t, const float *__restrict__ draft,
                    int64_t ld_d, const int32_t *__restrict__ tokens,
                    const int32_t *__restrict__ n_draft, const float *__restrict__ u,
                    int max_draft, int64_t vocab, int vec, int32_t *__restrict__ tokens_out,
                    int32_t *__restrict__ n_accepted)
{
    __shared__ double warp_w[kWarps];        // this CTA's slices
    __shared__ double cta_w[2][kMaxCluster];  // every CTA's total: of the weights, of the plain row
    __shared__ int taken_s, refused_s, empty_s, owner_s;
    __shared__ Search search;
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int64_t s = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto started = cl.barrier_arrive();  // waited for before the first access to another CTA
    pdl_wait();
    QSA_AFTER_WAIT(target);
    QSA_AFTER_WAIT(draft);
    QSA_AFTER_WAIT(tokens);
    QSA_AFTER_WAIT(n_draft);
    QSA_AFTER_WAIT(u);
    pdl_trigger();

    // ---- how many drafts are taken: the first refusal.  (The first 32 tokens and numbers are
    // loaded beside n_draft, not behind it.)
    if (warp == 0) {
        int n = max_draft, a = max_draft;
        for (int j0 = 0; j0 < n && a == n; j0 += 32) {
            const int j = j0 + lane;
            int t = -1;
            float uj = 0.0f;
            if (j < max_draft) {
                t = tokens[s * max_draft + j];
                uj = u[s * (max_draft + 1) + j];
            }
            if (j0 == 0 && n_draft) a = n = min(max(n_draft[s], 0), max_draft);
            bool refuse = j < n;  // a token outside the vocabulary is refused
            if (j < max_draft && t >= 0 && t < vocab) {
                const float p = target[(s * (max_draft + 1) + j) * ld_t + t];
                const float q = draft ? draft_prob(draft[(s * max_draft + j) * ld_d + t]) : 1.0f;
                refuse = j < n && !((double)uj * (double)q < (double)p);
            }
            const uint32_t b = __ballot_sync(0xffffffffu, refuse);
            if (b) a = j0 + __ffs(b) - 1;
        }
        if (lane == 0) {
            taken_s = a;
            refused_s = a < n;
        }
    }
    __syncthreads();
    const int a = taken_s;
    const bool refused = refused_s != 0;
    const int64_t chunks = (vocab + kChunk - 1) / kChunk;
    const int64_t per = (chunks + (int64_t)C * kWarps - 1) / ((int64_t)C * kWarps);
    const int64_t c0 = min(((int64_t)rank * kWarps + warp) * per, chunks);
    const int64_t c1 = min(c0 + per, chunks);
    const float r = fminf(fmaxf(u[s * (max_draft + 1) + max_draft], 0.0f), 1.0f);
    const int turned = refused && !draft ? tokens[s * max_draft + a] : -1;
    cl.barrier_wait(std::move(started));  // every CTA of the cluster runs

    // the weights after a refusal; then, only where they are zero everywhere (the two rows are
    // equal), the target's row itself
    for (int plain = refused ? 0 : 1; plain < 2; ++plain) {
        Row row;
        row.p = target + (s * (max_draft + 1) + a) * ld_t;
        row.q = !plain && draft ? draft + (s * max_draft + a) * ld_d : nullptr;
        row.skip = plain ? -1 : turned;
        const double mine = slice_sum(row, c0, c1, vocab, vec != 0);
        if (lane == 0) warp_w[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const double t = warp_sum_f64(lane < kWarps ? warp_w[lane] : 0.0);
            if (lane < C) *cl.map_shared_rank(&cta_w[plain][rank], lane) = t;
        }
        cl.sync();  // after the last turn's no CTA touches another's shared memory
        double total = 0.0;
        if (warp == 0) total = warp_sum_f64(lane < C ? cta_w[plain][lane] : 0.0);
        if (!plain) {  // (every CTA comes to the same answer)
            if (tid == 0) empty_s = !(total > 0.0);
            __syncthreads();
            if (empty_s) continue;
        }
        // ---- where the drawn point lies: the CTA, its warp's slice (warp 0), the index (all its warps)
        if (warp == 0) {
            const double x = (double)r * total;
            double before = 0.0, base = 0.0;
            int last, w = -1;
            int owner = first_over(lane < C ? cta_w[plain][lane] : 0.0, C, 0.0, x, before, last);
            const bool tail = owner < 0;  // rounding at the end: the last weight
            if (tail) owner = last;
            bool end = false;
            if (owner >= 0 && rank == owner) {
                w = tail ? -1 : first_over(lane < kWarps ? warp_w[lane] : 0.0, kWarps, before, x, base, last);
                end = w < 0;
                if (end) {
                    (void)first_over(lane < kWarps ? warp_w[lane] : 0.0, kWarps, 0.0, INFINITY, base, last);
                    w = last;
                }
            }
            if (lane == 0) {
                const int64_t d0 = w < 0 ? 0 : min(((int64_t)rank * kWarps + w) * per, chunks);
                search.base = base;
                search.x = x;
                search.c0 = d0;
                search.c1 = w < 0 ? 0 : min(d0 + per, chunks);
                search.end = end;
                owner_s = rank == (owner < 0 ? 0 : owner);
            }
        }
        __syncthreads();
        if (owner_s) {
            const int64_t token = slice_find(row, search, vocab);  // -1: no weight anywhere
            if (token >= -1) {
                int32_t *to = tokens_out + s * (max_draft + 1);
                for (int j = lane; j <= max_draft; j += 32)
                    to[j] = j < a ? tokens[s * max_draft + j] : (j == a ? (int)token : -1);
                if (lane == 0) n_accepted[s] = a;
            }
        }
        break;
    }
}

}  // namespace

cudaError_t launch_draft_verify(const float *target, int64_t ld_t, const float *draft, int64_t ld_d,
                                const int32_t *tokens, const int32_t *n_draft, const float *u,
                                int64_t n_seq, int64_t max_draft, int64_t vocab, int32_t *tokens_out,
                                int32_t *n_accepted, cudaStream_t st)
{
    const bool vec = vocab % 4 == 0 && ld_t % 4 == 0 && (!draft || ld_d % 4 == 0) &&
                     ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) & 15) == 0;
    // CTAs per sequence: as many as run at once (two per SM), while a warp still has more than one
    // chunk of the row
    int c = 1;
    while (c < kMaxCluster && n_seq * 2 * c <= 2 * (int64_t)device_sm_count() &&
           vocab > (int64_t)c * kWarps * kChunk)
        c *= 2;
    return launch(draft_verify_kernel, dim3((unsigned)(n_seq * c)), dim3(kThreads), 0, st, c, target,
                  ld_t, draft, ld_d, tokens, n_draft, u, (int)max_draft, vocab, (int)vec, tokens_out,
                  n_accepted);
}

}  // namespace qsa
