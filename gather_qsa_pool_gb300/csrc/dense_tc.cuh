// dense_tc.cuh -- what the tcgen05 kernels of the attention over every visible cell share
// (dense_attn_tc.cu, dense_few_tc.cu): tiles and their TMA maps, bounded waits, packed arithmetic, the
// walk over a CTA's parts.  Only the library's own .cu files include this header.
#pragma once

#include <cuda.h>
#include <cuda_fp8.h>

#include "dense.cuh"
#include "mma_frag.cuh"
#include "umma.cuh"

namespace qsa {

constexpr int kD = 128;
constexpr int kN = 128;                  // cells of a tile
constexpr uint32_t kHalf = 128 * 128;    // 16 KB: 128 rows x 64 dims of bf16
constexpr uint32_t kTileB = 2 * kHalf;   // 32 KB: a K or V tile, or a group's queries
constexpr uint32_t kRawTile = 128 * 128;  // 16 KB: 128 cells of codes
constexpr int kTeamWarps = 3;             // warps that convert K tiles, and V tiles
constexpr float kMove = 8.0f;            // move the reference past 2^8 growth
constexpr int kSlots = 8;                // parts whose flags are kept
constexpr int64_t kMaxStride = 1 << 28;  // elements between rows that a tensor map takes

__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                         uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// mbar_wait and warp_wait for this kernel's many waiting warps: the hardware may suspend the
// thread up to 20 us a try (sixteen softmax warps that poll take issue slots from those that
// compute).
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    if (limit_ns == 0) return false;
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(a), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
        if ((i & 15) == 0) {
            const uint64_t t = global_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > limit_ns) return false;
        }
    }
}
__device__ __forceinline__ bool bar_wait_warp(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity, limit_ns)) != 0;
}

// One box of a 2D tensor map: 64 bf16 columns from x, the map's box rows from y.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// 32 columns of this warp's rows, without waiting.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float *v)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
          "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
          "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// The CTA's share of the list, part by part; every role walks the same parts.
struct Parts {
    WorkItem it;
    int64_t x, x1;
    int32_t n;             // parts so far
    // of the current part
    int32_t tile0, tile1;  // its tiles of the item
    int64_t t0;            // first token of the sequence
    int32_t len, cells, n_see, pos0, tok0, toks;
    bool fits;

    __device__ __forceinline__ void set(const KvView &kv, const SeqView &sv, const WorkShape &w)
    {
        const int64_t first = it.start + w.over;
        tile0 = x > first ? (int)(x - first) : 0;
        tile1 = x1 > first ? (int)min((int64_t)it.tiles, x1 - first) : 0;
        seq_tokens(sv, it.s, t0, len);
        cells = seq_cells(sv, it.s, len);
        fits = cells_fit(kv, cells);
        n_see = fits ? item_cells(w, len, cells, it.t) : 0;
        tok0 = it.t * w.rt;
        toks = min(w.rt, len - tok0);
        pos0 = w.causal ? cells - len + tok0 : cells - 1;
    }
    // The next part that has tiles.
    __device__ __forceinline__ bool next(const KvView &kv, const SeqView &sv, const WorkShape &w)
    {
        ++n;
        do {
            x = it.start + w.over + it.tiles;
            if (x >= x1 || !work_next(sv, w, it)) return false;
            set(kv, sv, w);
        } while (tile1 <= tile0);
        return true;
    }
    // cells behind pos0 (and behind n_see) are not seen by every row
    __device__ __forceinline__ bool edge(int t) const { return t * kN + kN - 1 > pos0; }
};

// A cell's page entry, loaded some tiles ahead and not looked at until then (packed rows: none), and
// the cell's row: -1 when its page is not in the pool, -2 when there is no such cell.
struct PageAhead {
    int32_t page;
    int32_t cell;  // below 0: none
    __device__ __forceinline__ void load(const KvView &kv, const Parts &p, bool on, int64_t j)
    {
        on = on && j < p.n_see;
        cell = on ? (int32_t)j : -1;
        page = 0;
        if (on && kv.table) {
            const int64_t k = j >> kv.page_shift;
            page = k < kv.ld_table ? kv.table[(int64_t)p.it.s * kv.ld_table + k] : -1;
        }
    }
    __device__ __forceinline__ int row(const KvView &kv, const Parts &p) const
    {
        if (cell < 0) return -2;
        if (!kv.table) return (int)p.t0 + cell;
        if ((uint32_t)page >= (uint32_t)kv.n_pages) return -1;
        return (page << kv.page_shift) | (cell & ((1 << kv.page_shift) - 1));
    }
};

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled()
{
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// Rows of `width` values at a stride of ld, in boxes of 128 bytes (64 bf16 values or 128 codes) x
// box_rows rows, in the 128-byte swizzle or row after row.  Zeros behind the last row.  L2 fetches a
// head's row and no more (with 256 bytes of codes the other heads' come along and go again: 570 MB
// instead of 420 for 411 MB of cells).
inline bool make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t width, int64_t ld, int box_rows, bool e8, bool swizzle)
{
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * (e8 ? 1 : 2)};
    const cuuint32_t box[2] = {e8 ? 128u : 64u, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, e8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              e8 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every tensor-memory load of this thread so far has arrived; the N values pass through it, so that no
// use of them moves before it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// Rows r0 .. of a swizzled V tile, rows `first` and every `step` after it: rows from r1 on, which no
// query row sees, become zero (their weight is zero, but zero times an infinity is not); infinities
// and NaN of those before, which only some see, become zero too, and true is returned: the epilogue
// adds them.  Lanes of a warp: 16 chunks of 16 bytes x two rows.
__device__ __forceinline__ bool scrub_tile(unsigned char *tile, int r0, int r1, int first, int step)
{
    const int lane = threadIdx.x & 31, c = lane & 15;
    bool odd = false;
    for (int r = r0 + first + (lane >> 4); r < kN; r += step) {
        uint4 *w = reinterpret_cast<uint4 *>(tile + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        if (r >= r1) {
            *w = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        uint4 v = *w;
        uint32_t *u = reinterpret_cast<uint32_t *>(&v);
        bool any = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t m = __vcmpeq2(u[k] & 0x7f807f80u, 0x7f807f80u);
            any |= m != 0;
            u[k] &= ~m;
        }
        if (any) *w = v;
        odd |= any;
    }
    return odd;
}

// A raw tile of e4m3 codes to a swizzled bf16 tile, value = code * 2^e (exact), by kLanes lanes (`at`:
// this one's number); rows from e0 on as in scrub_tile.  A lane's 16 codes c of rows r, r + kLanes / 8,
// ... are chunks 2 c and 2 c + 1 of the bf16 row; the lanes of the upper dim half write them in the
// other order, as both halves lie on the same banks.
template <int kLanes>
__device__ __forceinline__ bool convert_tile(const unsigned char *src, unsigned char *dst, const uint8_t *exps,
                                             int at, int e0, int e1)
{
    bool odd = false;
    const int c = at & 7;
    unsigned char *const w = dst + (c >> 2) * kHalf;
    const int first = 2 * (c & 3) + (c >> 2), second = first ^ 1;
    // (unrolled twice, a chunk of 1,024 tokens over 61,789 cells takes 1,317 us instead of 1,253: more
    // code than stays near)
#pragma unroll 1
    for (int r = at >> 3; r < kN; r += kLanes / 8) {
        uint4 v = *reinterpret_cast<const uint4 *>(src + r * 128 + c * 16);
        uint32_t u[4] = {v.x, v.y, v.z, v.w};
        if (r >= e0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t m = __vcmpeq4(u[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                odd |= m != 0 && r < e1;
                u[k] = r < e1 ? u[k] & ~m : 0u;
            }
        }
        const float f = two_to(min(max((int)exps[r] - kExpBias, kExpMin), kExpMax));
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const __half2_raw h =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
            const float2 x = mul2(__half22float2(__half2(h)), make_float2(f, f));
            o[k] = pack_bf16(x.x, x.y);
        }
        const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]);
        const uint4 hi = make_uint4(o[4], o[5], o[6], o[7]);
        *reinterpret_cast<uint4 *>(w + r * 128 + ((first ^ (r & 7)) << 4)) = c >> 2 ? hi : lo;
        *reinterpret_cast<uint4 *>(w + r * 128 + ((second ^ (r & 7)) << 4)) = c >> 2 ? lo : hi;
    }
    return odd;
}

// Barrier `id` of kLanes threads with the OR of `v` over them.
template <int kLanes>
__device__ __forceinline__ bool named_or(int id, bool v)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, c;\n\t"
        "setp.ne.u32 c, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, c;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "n"(kLanes)
        : "memory");
    return r != 0;
}
template <int kLanes>
__device__ __forceinline__ void named_sync(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kLanes) : "memory");
}

}  // namespace qsa
