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
// slice of the row(s), and the CTA whose slice holds the drawn point scans the slice of the one
// warp that holds it.  One launch, no workspace, no atomics: the same result every time.  Bound
// by one pass over one or two rows; with few sequences by the chain token -> gather -> row.
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

// Weight of one index: max(p - q, 0) as a pair (d, e); a NaN or negative value counts as 0.
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
    const float *p, *q;  // q == NULL: no draft row
    int skip;            // index whose weight is 0 (the refused token of a draft without rows)
};

__device__ __forceinline__ void row_weight(const Row &r, int64_t i, int64_t vocab, bool difference,
                                           float &d, float &e)
{
    d = e = 0.0f;
    if (i >= vocab) return;
    const float p = r.p[i];
    if (difference && r.q) {
        weight_of(p, r.q[i], d, e);
    } else if (!(difference && i == r.skip)) {
        d = p > 0.0f ? p : 0.0f;
    }
}

__global__ void __launch_bounds__(kThreads)
draft_verify_kernel(const float *__restrict__ target, int64_t ld_t, const float *__restrict__ draft,
                    int64_t ld_d, const int32_t *__restrict__ tokens,
                    const int32_t *__restrict__ n_draft, const float *__restrict__ u,
                    int max_draft, int64_t vocab, int vec, int32_t *__restrict__ tokens_out,
                    int32_t *__restrict__ n_accepted)
{
    __shared__ double warp_w[kWarps], warp_p[kWarps];       // this CTA's slices: weights, plain p
    __shared__ double cta_w[kMaxCluster], cta_p[kMaxCluster];  // every CTA's total
    __shared__ int taken_s, refused_s;
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

    // ---- how many drafts are taken: the first refusal
    if (warp == 0) {
        const int n = n_draft ? min(max(n_draft[s], 0), max_draft) : max_draft;
        int a = n;
        for (int j0 = 0; j0 < n && a == n; j0 += 32) {
            const int j = j0 + lane;
            bool refuse = false;
            if (j < n) {
                const int t = tokens[s * max_draft + j];
                refuse = true;  // a token outside the vocabulary is refused
                if (t >= 0 && t < vocab) {
                    const float p = target[(s * (max_draft + 1) + j) * ld_t + t];
                    const float q = draft ? draft[(s * max_draft + j) * ld_d + t] : 1.0f;
                    refuse = !((double)u[s * (max_draft + 1) + j] * (double)q < (double)p);
                }
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
    Row row;
    row.p = target + (s * (max_draft + 1) + a) * ld_t;
    row.q = refused && draft ? draft + (s * max_draft + a) * ld_d : nullptr;
    row.skip = refused && !draft ? tokens[s * max_draft + a] : -1;

    // ---- sums of this warp's slice: whole chunks of 128 values
    const int64_t chunks = (vocab + kChunk - 1) / kChunk;
    const int64_t per = (chunks + (int64_t)C * kWarps - 1) / ((int64_t)C * kWarps);
    const int64_t c0 = min(((int64_t)rank * kWarps + warp) * per, chunks);
    const int64_t c1 = min(c0 + per, chunks);
    float ws = 0.0f, wc = 0.0f, ps = 0.0f, pc = 0.0f;
    auto take = [&](float p, float q, int64_t i) {
        float d, e = 0.0f;
        if (row.q) {
            weight_of(p, q, d, e);
        } else {
            d = p > 0.0f && i != row.skip ? p : 0.0f;
        }
        add_pair(ws, wc, d);
        wc = __fadd_rn(wc, e);
        if (refused) add_pair(ps, pc, p > 0.0f ? p : 0.0f);
    };
    if (vec) {
#pragma unroll 4
        for (int64_t c = c0; c < c1; ++c) {
            const int64_t i = c * kChunk + 4 * lane;
            if (i >= vocab) continue;  // vec: the vocabulary is a multiple of 4
            const float4 p = *reinterpret_cast<const float4 *>(row.p + i);
            float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (row.q) q = *reinterpret_cast<const float4 *>(row.q + i);
            take(p.x, q.x, i);
            take(p.y, q.y, i + 1);
            take(p.z, q.z, i + 2);
            take(p.w, q.w, i + 3);
        }
    } else {
#pragma unroll 4
        for (int64_t i = c0 * kChunk + lane; i < min(c1 * kChunk, vocab); i += 32)
            take(row.p[i], row.q ? row.q[i] : 0.0f, i);
    }
    const double wsum = warp_sum_f64((double)ws + (double)wc);
    const double psum = warp_sum_f64((double)ps + (double)pc);
    if (lane == 0) {
        warp_w[warp] = wsum;
        warp_p[warp] = psum;
    }
    __syncthreads();
    cl.barrier_wait(std::move(started));  // every CTA of the cluster runs
    if (tid == 0) {
        double tw = 0.0, tp = 0.0;
        for (int i = 0; i < kWarps; ++i) {
            tw += warp_w[i];
            tp += warp_p[i];
        }
        for (int c = 0; c < C; ++c) {
            *cl.map_shared_rank(&cta_w[rank], c) = tw;
            *cl.map_shared_rank(&cta_p[rank], c) = tp;
        }
    }
    cl.sync();  // after it no CTA touches another's shared memory

    // ---- where the drawn point lies
    if (warp == 0) {
        double total = 0.0, before = 0.0;
        for (int c = 0; c < C; ++c) total += cta_w[c];
        // nothing left of p - q (the two rows are equal): the token comes from p itself
        const bool difference = refused && total > 0.0;
        const double *cta = cta_w, *wsums = warp_w;
        if (refused && !difference) {
            cta = cta_p;
            wsums = warp_p;
            total = 0.0;
            for (int c = 0; c < C; ++c) total += cta_p[c];
        }
        const double r = fmin(fmax((double)u[s * (max_draft + 1) + max_draft], 0.0), 1.0);
        const double x = r * total;
        // the first slice whose running sum passes x, else the last one that holds any weight
        int owner = -1, ow = -1, last_c = -1;
        double run = 0.0;
        for (int c = 0; c < C; ++c) {
            if (cta[c] > 0.0) last_c = c;
            if (owner < 0 && run + cta[c] > x) {
                owner = c;
                before = run;
            }
            run += cta[c];
        }
        if (owner < 0) {
            owner = last_c;
            before = INFINITY;  // its last weight
        }
        int32_t *to = tokens_out + s * (max_draft + 1);
        if (rank == (owner < 0 ? 0 : owner)) {
            int token = -1;  // no weight anywhere
            if (owner >= 0) {
                run = before;
                int last_w = -1;
                for (int i = 0; i < kWarps; ++i) {
                    if (wsums[i] > 0.0) last_w = i;
                    if (ow < 0 && run + wsums[i] > x && wsums[i] > 0.0 && !isinf(run)) {
                        ow = i;
                        before = run;
                    }
                    run += wsums[i];
                }
                if (ow < 0) {
                    ow = last_w;
                    before = INFINITY;
                }
                const int64_t d0 = min(((int64_t)rank * kWarps + ow) * per, chunks);
                const int64_t d1 = min(d0 + per, chunks);
                const bool find_last = isinf(before);
                double base = find_last ? 0.0 : before;
                int64_t found = -1, last = -1;
                for (int64_t c = d0; c < d1 && found < 0; ++c) {
                    const int64_t i = c * kChunk + 4 * lane;
                    double w[4], sum = 0.0;
                    bool any_w[4];
                    int pos = -1;  // this lane's last positive weight
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float d, e;
                        row_weight(row, i + k, vocab, difference, d, e);
                        w[k] = (double)d + (double)e;
                        any_w[k] = w[k] > 0.0;
                        if (any_w[k]) pos = k;
                        sum += w[k];
                        w[k] = sum;
                    }
                    double incl = sum;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double v = __shfl_up_sync(0xffffffffu, incl, o);
                        if (lane >= o) incl += v;
                    }
                    const double start = base + (incl - sum);
                    int hit = 4;
#pragma unroll
                    for (int k = 3; k >= 0; --k)
                        if (any_w[k] && start + w[k] > x && !find_last) hit = k;
                    const uint32_t b = __ballot_sync(0xffffffffu, hit < 4);
                    const uint32_t any = __ballot_sync(0xffffffffu, pos >= 0);
                    if (any) {
                        const int j = 31 - __clz(any);
                        last = c * kChunk + 4 * j + __shfl_sync(0xffffffffu, pos, j);
                    }
                    if (b) {
                        const int j = __ffs(b) - 1;
                        found = c * kChunk + 4 * j + __shfl_sync(0xffffffffu, hit, j);
                    }
                    base += __shfl_sync(0xffffffffu, incl, 31);
                }
                token = (int)(found >= 0 ? found : last);
            }
            for (int j = lane; j <= max_draft; j += 32)
                to[j] = j < a ? tokens[s * max_draft + j] : (j == a ? token : -1);
            if (lane == 0) n_accepted[s] = a;
        }
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
    // CTAs per sequence: until the sequences fill the GPU twice, and while a warp still has more
    // than one chunk of the row
    int c = 1;
    while (c < kMaxCluster && n_seq * c < 2 * (int64_t)device_sm_count() &&
           vocab > (int64_t)c * kWarps * kChunk)
        c *= 2;
    return launch(draft_verify_kernel, dim3((unsigned)(n_seq * c)), dim3(kThreads), 0, st, c, target,
                  ld_t, draft, ld_d, tokens, n_draft, u, (int)max_draft, vocab, (int)vec, tokens_out,
                  n_accepted);
}

}  // namespace qsa
