// dense.cuh -- shared pieces of the paged key/value cache and of the dense attention over it
// (paged_rw.cu, dense_attn.cu, dense_decode.cu, dense_few_tc.cu, dense_attn_tc.cu): the device view of a cache,
// the row of a cell, the packed sequences and the flattened list of work.
#pragma once

#include <math.h>

#include "qsa_internal.cuh"

namespace qsa {

// Exponents of a QSA_E4M3 row: value = code * 2^(byte - 127), byte in [27, 227].
constexpr int kExpBias = 127;
constexpr int kExpMin = -100, kExpMax = 100;

// 2^e for e in [-126, 127], from its bits.
__host__ __device__ __forceinline__ float two_to(int e)
{
    union {
        uint32_t u;
        float f;
    } x;
    x.u = (uint32_t)(e + 127) << 23;
    return x.f;
}

// Eight consecutive values, 16-byte aligned.
__device__ __forceinline__ void load8(const float *p, float *x)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *x)
{
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}

// The views below hold plain pointers (not __restrict__): a load through one is an ordinary load,
// which the compiler does not move before a kernel's wait for its predecessor, so the kernels
// read the views where they lie, in the parameters.

// Keys and values as the attention kernels see them.  table != NULL: a paged pool, the cell at
// position p of sequence s lives in row table[s][p >> page_shift] << page_shift | (p & mask).
// table == NULL: packed sequences, the cell is row cu[s] + p.
struct KvView {
    const void *K, *V;
    const uint8_t *K_exp, *V_exp;  // [rows][H_kv], QSA_E4M3 only
    int64_t ld_k, ld_v;            // elements between rows
    const int32_t *table;
    int64_t ld_table;
    int32_t n_pages;
    int32_t page_shift;
    int32_t H_kv;
};

// Packed query tokens: sequence s has tokens cu[s] .. cu[s+1] - 1, the last of its kv_len[s]
// cells (kv_len == NULL: as many cells as tokens).
struct SeqView {
    const int32_t *cu;
    const int32_t *kv_len;
    int32_t n_seq;
    int64_t n_tok;  // tokens in the buffers: whatever cu says, none beyond is touched
};

// Tokens of a sequence, clipped to the buffers.
__device__ __forceinline__ void seq_tokens(const SeqView &sv, int s, int64_t &t0, int &len)
{
    int64_t a = sv.cu[s], b = sv.cu[s + 1];
    a = a < 0 ? 0 : (a > sv.n_tok ? sv.n_tok : a);
    b = b < a ? a : (b > sv.n_tok ? sv.n_tok : b);
    t0 = a;
    len = (int)(b - a);
}

__device__ __forceinline__ int seq_cells(const SeqView &sv, int s, int len)
{
    return sv.kv_len ? max(sv.kv_len[s], 0) : len;
}

// A paged sequence longer than its row of the table cannot be right: its outputs become NaN.  (Nor is one
// looked at whose last tile's end would pass 31 bits.)
constexpr int32_t kMostCells = 0x7fffff00;
__device__ __forceinline__ bool cells_fit(const KvView &kv, int cells)
{
    return cells <= kMostCells && (kv.table == nullptr || (int64_t)cells <= (kv.ld_table << kv.page_shift));
}

// Pool row of the cell at position p of sequence s; -1 when its page is not in the pool.
// first: cu[s] of packed sequences.
__device__ __forceinline__ int64_t cell_row(const KvView &kv, int s, int64_t first, int p)
{
    if (kv.table == nullptr) return first + p;
    const int64_t j = p >> kv.page_shift;
    if (j >= kv.ld_table) return -1;
    const int32_t page = kv.table[(int64_t)s * kv.ld_table + j];
    if ((uint32_t)page >= (uint32_t)kv.n_pages) return -1;
    return ((int64_t)page << kv.page_shift) | (p & ((1 << kv.page_shift) - 1));
}

// An infinite or NaN value of V (element i of the pool, bf16 or codes) as the attention kernels add it to the
// rows that see it, zero where it is finite.
template <bool E8>
__device__ __forceinline__ float odd_value_at(const KvView &kv, int64_t i)
{
    if constexpr (E8) {
        return (static_cast<const uint8_t *>(kv.V)[i] & 0x7f) == 0x7f ? NAN : 0.0f;
    } else {
        const float f = __bfloat162float(static_cast<const __nv_bfloat16 *>(kv.V)[i]);
        return isfinite(f) ? 0.0f : f;
    }
}

// ------------------------------------------------------------------ the flattened work list
// The rows of a sequence and KV head (its tokens times the G query heads of the KV head, token
// major) are cut into row tiles of `rt` tokens; a (sequence, KV head, row tile) is an item, and
// an item's work is its visible cells in tiles of `kt` cells (at least one, so that the rows of
// an item that sees nothing are written too).  Items are numbered sequence-major, then KV head,
// then row tile, and their tiles form one list, which is cut into equal shares: a CTA's share
// covers parts of at most a few items, and only its first and last part can be incomplete.
struct WorkShape {
    int32_t rt;      // query tokens per row tile
    int32_t kt;      // cells per tile; 0: every item is one tile (work that is not cut)
    int32_t over;    // what an item costs besides its tiles, in tiles: the list has that many
                     // places without a tile before each item's first
    int32_t H_kv;
    int32_t causal;
    int32_t most;    // the most cells a sequence may have: a longer one cannot be right, and nothing of it
                     // is looked at
};

// Cells that the tokens of row tile t see together.
__device__ __forceinline__ int item_cells(const WorkShape &w, int len, int cells, int t)
{
    if (cells > w.most) return 0;
    if (!w.causal) return cells;
    const int64_t last = (int64_t)(t + 1) * w.rt;
    const int64_t seen = (int64_t)cells - len + (last < len ? last : len);
    return seen < 0 ? 0 : (int)seen;
}

__device__ __forceinline__ int item_tiles(const WorkShape &w, int len, int cells, int t)
{
    if (w.kt == 0) return 1;
    const int n = item_cells(w, len, cells, t);
    return n > 0 ? (n - 1) / w.kt + 1 : 1;
}

// a / b, b > 0, with one 32-bit division where that is enough.
__device__ __forceinline__ int64_t div_pos(int64_t a, int64_t b)
{
    if (((uint64_t)a | (uint64_t)b) >> 32 == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

__device__ __forceinline__ int64_t floor_div(int64_t a, int64_t b)
{
    return a >= 0 ? div_pos(a, b) : -div_pos(-a + b - 1, b);
}

// Sum of floor((a i + b) / m) over 0 <= i < n (a, b >= 0, m > 0).  Whole multiples of m in a and b leave it
// in closed form; the rest counts the lattice points under a line, which counted along the other axis is a
// sum of the same kind with a and m exchanged: a few turns, as in Euclid's algorithm.
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b)
{
    int64_t sum = 0;
    for (;;) {
        if (a >= m) {
            const int64_t q = div_pos(a, m);
            sum += n * (n - 1) / 2 * q;
            a -= q * m;
        }
        if (b >= m) {
            const int64_t q = div_pos(b, m);
            sum += n * q;
            b -= q * m;
        }
        const int64_t y = a * n + b;
        if (y < m) return sum;
        n = div_pos(y, m);
        b = y - n * m;
        const int64_t t = a;
        a = m;
        m = t;
    }
}

// Tiles of the row tiles before t (t <= the last row tile) of one KV head of a sequence.  A row tile
// i < t sees c = cells - len + (i + 1) rt cells: one tile if that is none, else
// floor((c - 1) / kt) + 1; the sum is shortest when one of rt and kt divides the other (1, 2, 4 ...
// heads per KV head).  (Added up tile by tile for the others, a prompt of 65,536 tokens, 28 / 4 heads, took
// 23.1 ms instead of 20.7.)
__device__ __forceinline__ int64_t tiles_before(const WorkShape &w, int len, int cells, int t)
{
    if (!w.causal || w.kt == 0 || cells > w.most) return (int64_t)t * item_tiles(w, len, cells, 0);
    const int64_t base = (int64_t)cells - len;
    int64_t i0 = base < 0 ? div_pos(-base, w.rt) : 0;  // row tiles that see nothing
    if (i0 > t) i0 = t;
    const int64_t B = base + w.rt - 1;
    int64_t sum = t;
    if (w.rt % w.kt == 0) {
        const int64_t n = t - i0;
        sum += n * floor_div(B, w.kt) + (w.rt / w.kt) * (n * (i0 + t - 1) / 2);
    } else if (w.kt % w.rt == 0) {
        const int64_t r = w.kt / w.rt, v0 = floor_div(B, w.rt);
        // F(n) = sum of floor(v / r) over 0 <= v < n
        const int64_t n1 = v0 + t, n0 = v0 + i0, q1 = div_pos(n1, r), q0 = div_pos(n0, r);
        if (t > i0)
            sum += (r * (q1 * (q1 - 1) / 2) + q1 * (n1 - q1 * r)) -
                   (r * (q0 * (q0 - 1) / 2) + q0 * (n0 - q0 * r));
    } else {
        if (t > i0) sum += floor_sum(t - i0, w.kt, w.rt, B + i0 * w.rt);
    }
    return sum;
}

// Places of one KV head of a sequence.
__device__ __forceinline__ int64_t seq_places(const WorkShape &w, int len, int cells)
{
    const int nt = (len + w.rt - 1) / w.rt;
    return nt == 0 ? 0
                   : tiles_before(w, len, cells, nt - 1) + item_tiles(w, len, cells, nt - 1) +
                         (int64_t)nt * w.over;
}

struct WorkItem {
    int32_t s, g, t;        // sequence, KV head, row tile
    int32_t tiles;
    int64_t start;          // its first place in the list; its tiles begin `over` places on
    int64_t index;          // its number
};

// Places and items of one sequence.
__device__ __forceinline__ void seq_work(const SeqView &sv, const WorkShape &w, int s, int64_t &places,
                                         int64_t &items, int &len, int &cells)
{
    places = items = 0;
    len = cells = 0;
    if (s >= sv.n_seq) return;
    int64_t t0;
    seq_tokens(sv, s, t0, len);
    cells = seq_cells(sv, s, len);
    places = seq_places(w, len, cells) * w.H_kv;
    items = (int64_t)((len + w.rt - 1) / w.rt) * w.H_kv;
}

__device__ __forceinline__ int64_t warp_sum_i64(int64_t v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The item that holds place x of the list, among 32 sequences from s0 on whose lanes have their
// work (base, items before them: of the sequences before s0); false if it lies behind them.
__device__ __forceinline__ bool work_among(const WorkShape &w, int64_t x, int s0, int64_t mine, int64_t items,
                                           int len, int cells, int64_t &base, int64_t &before, WorkItem &it)
{
    const int lane = threadIdx.x & 31;
    int64_t incl = mine, inc_items = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o), u = __shfl_up_sync(0xffffffffu, inc_items, o);
        if (lane >= o) {
            incl += v;
            inc_items += u;
        }
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, x < base + incl);
    if (!hit) {
        base += __shfl_sync(0xffffffffu, incl, 31);
        before += __shfl_sync(0xffffffffu, inc_items, 31);
        return false;
    }
    const int j = __ffs(hit) - 1;  // the first lane whose prefix passes x
    const int64_t sbase = base + __shfl_sync(0xffffffffu, incl - mine, j);
    const int64_t stot = __shfl_sync(0xffffffffu, mine, j);
    const int64_t first_item = before + __shfl_sync(0xffffffffu, inc_items - items, j);
    len = __shfl_sync(0xffffffffu, len, j);
    cells = __shfl_sync(0xffffffffu, cells, j);
    const int64_t per_head = div_pos(stot, w.H_kv);
    it.s = s0 + j;
    it.g = (int32_t)div_pos(x - sbase, per_head);
    const int64_t at = sbase + it.g * per_head;
    // the last row tile that does not begin behind x
    const int nt = (len + w.rt - 1) / w.rt;
    int t = 0, hi = nt;
    while (hi - t > 1) {
        const int mid = (t + hi) >> 1;
        if (tiles_before(w, len, cells, mid) + (int64_t)mid * w.over <= x - at) t = mid;
        else hi = mid;
    }
    it.t = t;
    it.start = t == 0 ? at : at + tiles_before(w, len, cells, t) + (int64_t)t * w.over;
    it.tiles = item_tiles(w, len, cells, t);
    it.index = first_item + (int64_t)it.g * nt + t;
    return true;
}

// The share of CTA `cta` of `ctas`: places [x0, x1) of the list, and the item at x0.  False when
// there is none.  All 32 lanes of a warp call it and get the same values.
__device__ __forceinline__ bool work_share(const SeqView &sv, const WorkShape &w, int cta, int ctas, int64_t &per,
                                           int64_t &x0, int64_t &x1, WorkItem &it)
{
    const int lane = threadIdx.x & 31;
    int64_t mine, items, total;
    int len, cells;
    seq_work(sv, w, lane, mine, items, len, cells);
    total = mine;
    for (int s = 32 + lane; s < sv.n_seq; s += 32) {
        int64_t m, i;
        int l, c;
        seq_work(sv, w, s, m, i, l, c);
        total += m;
    }
    total = warp_sum_i64(total);
    per = div_pos(total + ctas - 1, ctas);
    x0 = cta * per;
    x1 = x0 + per < total ? x0 + per : total;
    if (x0 >= x1) return false;
    int64_t base = 0, before = 0;
    if (work_among(w, x0, 0, mine, items, len, cells, base, before, it)) return true;
    for (int s0 = 32; s0 < sv.n_seq; s0 += 32) {
        seq_work(sv, w, s0 + lane, mine, items, len, cells);
        if (work_among(w, x0, s0, mine, items, len, cells, base, before, it)) return true;
    }
    return false;
}

// The same with item number `cta` whole, for work of few, short items: the list is its own.
__device__ __forceinline__ bool work_item(const SeqView &sv, const WorkShape &w, int cta, int ctas, int64_t &per,
                                          int64_t &x0, int64_t &x1, WorkItem &it)
{
    WorkShape one = w;
    one.kt = one.over = 0;
    if (!work_share(sv, one, cta, ctas, per, x0, x1, it)) return false;
    int64_t t0;
    int len;
    seq_tokens(sv, it.s, t0, len);
    it.tiles = item_tiles(w, len, seq_cells(sv, it.s, len), it.t);
    it.start = x0 = 0;
    x1 = per = w.over + it.tiles;
    return true;
}

// The item after `it` in the list (its sequence's length and cells are looked up again).
// Returns false past the end.  All 32 lanes call it with the same item.
__device__ __forceinline__ bool work_next(const SeqView &sv, const WorkShape &w, WorkItem &it)
{
    int64_t t0;
    int len;
    seq_tokens(sv, it.s, t0, len);
    int cells = seq_cells(sv, it.s, len);
    const int nt = (len + w.rt - 1) / w.rt;
    it.start += it.tiles + w.over;
    ++it.index;
    if (++it.t >= nt) {
        it.t = 0;
        if (++it.g >= w.H_kv) {
            it.g = 0;
            do {
                if (++it.s >= sv.n_seq) return false;
                seq_tokens(sv, it.s, t0, len);
            } while (len == 0);
            cells = seq_cells(sv, it.s, len);
        }
    }
    it.tiles = item_tiles(w, len, cells, it.t);
    return true;
}

// Partial result of part of an item: one record per (CTA, first / last part), holding for each
// row the running maximum (log2 units), the sum and the unnormalised output.
__host__ __device__ inline int64_t partial_floats(int rows, int d) { return (int64_t)rows * (d + 2); }

// ------------------------------------------------------------------ launchers

struct DenseArgs {
    KvView kv;
    SeqView sv;
    qsa_dtype kv_dtype, q_dtype;  // out has q's type
    const void *q;
    int64_t ld_q;  // elements between tokens
    void *out;     // [n_tok][H_q][d] packed
    float *lse;    // [n_tok][H_q] or NULL
    int H_q, d;
    float scale;
    int causal;
    int64_t pool_rows;  // rows of K and V
};

// Row tiles of rt tokens, cells in tiles of kt, `over` places an item.
inline WorkShape work_shape(const DenseArgs &a, int rt, int kt, int over)
{
    const int64_t most = a.kv.table ? a.kv.ld_table << a.kv.page_shift : kMostCells;
    return {rt, kt, over, a.kv.H_kv, a.causal, (int32_t)(most < kMostCells ? most : kMostCells)};
}

// Any shape: d a multiple of 8 up to 256, fp32 arithmetic on the CUDA cores.
cudaError_t launch_dense_attn(const DenseArgs &a, cudaStream_t st);

// A few new tokens per sequence (max_q as the host knows it) over bf16 or e4m3 cells, d 128.
bool dense_decode_ok(const DenseArgs &a, int64_t max_q);
size_t dense_decode_workspace();
cudaError_t launch_dense_decode(const DenseArgs &a, void *workspace, cudaStream_t st);

// The same with bf16 queries on the tcgen05 tensor cores, up to 32 rows (tokens x heads of a KV head) over
// bf16 cells and up to 64, as two row tiles, over e4m3 cells; short contexts of up to 16 rows it leaves to
// the above.
bool dense_few_ok(const DenseArgs &a, int64_t max_q);
size_t dense_few_workspace();
qsa_status launch_dense_few(const DenseArgs &a, int64_t max_q, void *workspace, cudaStream_t st);

// Many query rows on the tensor cores: bf16 queries, d 128.
bool dense_tc_ok(const DenseArgs &a);
size_t dense_tc_workspace();
qsa_status launch_dense_tc(const DenseArgs &a, void *workspace, cudaStream_t st);

}  // namespace qsa
