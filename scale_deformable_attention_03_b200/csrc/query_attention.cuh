// Shared by the forward and the backward of msda_query_attention: the warp's
// matrix fragments, tile loads, visibility and the distance of points.
//
// A warp holds 16 rows of one side (queries; keys in the gradient of k and v)
// and walks tiles of 64 rows of the other, which the CTA's four warps share in
// shared memory.  With 32 channels per head a score takes 32 multiply-adds in
// each product but also an exponential (16 per clock and SM) and, with the
// bias, a square root and about ten instructions: the matrix pipe is not what
// binds (a third busy), and the fragments of mma.sync leave every score in the
// thread that computes on it.  A square root serves all heads of a warp.
//
// The same forward on tcgen05.mma (128 queries per CTA, scores, weights and
// outputs in tensor memory, one row per thread, one thread issuing) measured
// slower at this width: 970 us with tiles of 64 keys and two CTAs per SM, 801 us
// with tiles of 32 and three, where this one took 684 us at that time (100 x 100
// grid, 8 heads), and twice as long for 900 queries.  Its products have 32 or 64
// columns, too few to pay for the hand-over of each tile between the issuing
// thread and the warps that form the weights.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "msda.h"
#include "msda_launch.h"

namespace msda {
namespace attn {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kRows = 16 * kAttnWarps;  // rows of the own side per CTA
constexpr int kTile = 64;           // rows of the other side per step
constexpr int kDim = 32;
constexpr int kScan = 256;          // tiles whose visibility is looked up at once
// Groups that a bit each tells apart (10 000 queries in 100 groups, mixed: 955 us
// forward with bits, 991 us with the groups sorted, 1268 us looked through).
constexpr int kGroupBits = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sqrt_approx(float x)
{
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two neighbouring scores of a row go through the packed fp32 instructions:
// one issue slot for both.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair(const float (&c)[4], int half)
{
    return make_float2(c[2 * half], c[2 * half + 1]);
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v)
{
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What pack_bf16's rounding left over, packed likewise.
__device__ __forceinline__ uint32_t pack_rest(float2 v, uint32_t packed)
{
    return pack_bf16(v.x - __uint_as_float(packed << 16),
                     v.y - __uint_as_float(packed & 0xffff0000u));
}

// c += a b for a 16 x 16 by 16 x 8 product.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from zero (no registers to clear).
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool on)
{
    const int n = on ? kBytes : 0;  // the rest is filled with zeros
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src),
                     "n"(kBytes), "r"(n)
                     : "memory");
}

__device__ __forceinline__ void cp_async_all(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int kLeft>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// A head's tile: 64 rows of 64 bytes, the 16-byte chunk c of row r at place
// c ^ ((r >> 1) & 3), so that eight rows' same chunk falls in eight different
// bank groups.
__device__ __forceinline__ uint32_t tile_at(int row, int chunk)
{
    return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

constexpr int kTileBytes = kTile * 64;  // of one head

// Where a lane's rows of a fragment load start; rows 8 (16) further on are at
// plain offsets, since the places repeat every eight rows.
struct LaneAt {
    uint32_t cols;     // rows lane & 7, chunk lane >> 3
    uint32_t sum[2];   // rows lane & 15, chunks lane >> 4 and two further on
};

__device__ __forceinline__ LaneAt lane_at(int lane)
{
    return {tile_at(lane & 7, lane >> 3),
            {tile_at(lane & 15, lane >> 4), tile_at(lane & 15, 2 + (lane >> 4))}};
}

// B fragments of the product with a tile's rows as columns (scores): all 32
// channels of the rows 8j .. 8j + 7; r[0], r[1] for channels 0..15, r[2], r[3]
// for 16..31.
__device__ __forceinline__ void load_cols(uint32_t (&r)[4], uint32_t tile, int j, const LaneAt& at)
{
    ldsm(r, tile + at.cols + 512 * j);
}

// B fragments of the product that sums over a tile's rows 16k .. 16k + 15:
// r[0], r[1] for channels 16d .. 16d + 7, r[2], r[3] for the eight after them.
__device__ __forceinline__ void load_sum(uint32_t (&r)[4], uint32_t tile, int k, int d,
                                         const LaneAt& at)
{
    ldsm_t(r, tile + at.sum[d] + 1024 * k);
}

// Copies tiles of 64 rows of HP heads of two tensors (keys and values, or
// queries and their output's gradient) into shared memory.  A thread copies the
// 16-byte chunk `c` of the rows row, row + kStep, ...; only the start of a tile
// is computed anew.
template <int HP>
struct TileCopy {
    static constexpr int kChunks = 4 * HP, kStep = kAttnThreads / kChunks;
    const char *a, *b;        // this thread's chunk of the item's row `row`
    int64_t lda, ldb;         // bytes from row to row
    uint32_t to;              // its place in a stage
    int row, n;               // first row of a tile, rows of the item

    __device__ __forceinline__ TileCopy(const __nv_bfloat16* pa, int64_t la,
                                        const __nv_bfloat16* pb, int64_t lb, int rows)
    {
        const int c = threadIdx.x % kChunks;
        row = threadIdx.x / kChunks;
        n = rows;
        lda = 2 * la;
        ldb = 2 * lb;
        a = reinterpret_cast<const char*>(pa) + row * lda + c * 16;
        b = reinterpret_cast<const char*>(pb) + row * ldb + c * 16;
        to = (c / 4) * kTileBytes + tile_at(row, c % 4);
    }

    // `all` the tile's rows, or those of the item whose bit is set in `keep`, the
    // others as zeros.
    __device__ __forceinline__ void fetch(uint32_t sa, uint32_t sb, int tile, bool all,
                                          uint2 keep) const
    {
        const int64_t r0 = (int64_t)tile * kTile;
        const char *pa = a + r0 * lda, *pb = b + r0 * ldb;
        // (the places of a chunk repeat every eight rows, and kStep is a multiple of that)
        static_assert(kStep % 8 == 0, "");
        const uint32_t ta = sa + to, tb = sb + to;
        if (all) {
#pragma unroll
            for (int i = 0; i < kTile / kStep; ++i) {
                cp_async_all(ta + i * kStep * 64, pa);
                cp_async_all(tb + i * kStep * 64, pb);
                pa += kStep * lda;
                pb += kStep * ldb;
            }
            return;
        }
#pragma unroll 1
        for (int i = 0; i < kTile / kStep; ++i) {
            const int r = tile * kTile + row + i * kStep;
            const int at = row + i * kStep;
            const bool there = r < n && ((at < 32 ? keep.x : keep.y) >> (at & 31) & 1);
            cp_async<16>(ta + i * kStep * 64, there ? pa : a - row * lda, there);
            cp_async<16>(tb + i * kStep * 64, there ? pb : b - row * ldb, there);
            pa += kStep * lda;
            pb += kStep * ldb;
        }
    }
};

// A fragments of a warp's 16 rows of one head, straight from memory; a row
// that is not `on` reads as zero.
__device__ __forceinline__ void load_rows(uint32_t (&f)[8], const __nv_bfloat16* head,
                                          int64_t stride, int row, bool on0, bool on1, int t)
{
    const uint32_t* p = reinterpret_cast<const uint32_t*>(head + (int64_t)row * stride) + t;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(head + (int64_t)(row + 8) * stride) + t;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        f[4 * s] = on0 ? __ldg(p + 8 * s) : 0u;
        f[4 * s + 1] = on1 ? __ldg(q + 8 * s) : 0u;
        f[4 * s + 2] = on0 ? __ldg(p + 8 * s + 4) : 0u;
        f[4 * s + 3] = on1 ? __ldg(q + 8 * s + 4) : 0u;
    }
}

// The groups of the own side's rows; lo and hi: of those >= 0.
struct GroupRange {
    int lo, hi;
    bool zero, all_zero;  // some 0, all 0
};

__device__ __forceinline__ GroupRange warp_range(const int32_t* g, int count)
{
    int lo = INT32_MAX, hi = -1;
    bool zero = false, all = true;
    for (int i = threadIdx.x & 31; i < count; i += 32) {
        const int v = __ldg(g + i);
        if (v >= 0) {
            lo = min(lo, v);
            hi = max(hi, v);
        }
        zero |= v == 0;
        all &= v == 0;
    }
    return {__reduce_min_sync(0xffffffffu, lo), __reduce_max_sync(0xffffffffu, hi),
            (bool)__any_sync(0xffffffffu, zero), (bool)__all_sync(0xffffffffu, all)};
}

// What is looked up for kScan tiles of the other side at once: its rows that see
// or are seen by some row of the own side (`rows`; the others are not read, so
// that a weight of zero never meets what they hold), the tiles that have such a
// row (bit set in `need`), and those in which no pair is masked (`clear`).
struct TileBits {
    uint2 rows[kScan];
    uint32_t need[kScan / 32], clear[kScan / 32];
    // the own side's groups: a bit each, modulo kGroupBits, where they lie that close
    // together, else sorted
    union {
        uint32_t own[kGroupBits / 32];
        int32_t sorted[kRows];
    };
};

// kOwnKeys: the own side (`count` rows from `mine` on) are keys and the other
// (`n` rows from `other` on) queries.
template <bool kOwnKeys>
__device__ void scan_tiles(TileBits& bits, const int32_t* mine, int count, const int32_t* other,
                           int n, int first, int last)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const GroupRange own = warp_range(mine, count);
    for (int w = threadIdx.x; w < kScan / 32; w += kAttnThreads) bits.need[w] = bits.clear[w] = 0;
    const bool wide = own.hi >= 0 && own.hi - own.lo >= kGroupBits;
    const int mine_here = (int)threadIdx.x < count ? __ldg(mine + threadIdx.x) : -1;
    if (!wide) {
        for (int w = threadIdx.x; w < kGroupBits / 32; w += kAttnThreads) bits.own[w] = 0;
        __syncthreads();
        if (mine_here >= 0)
            atomicOr(&bits.own[mine_here / 32 % (kGroupBits / 32)], 1u << (mine_here & 31));
    } else if ((int)threadIdx.x < count) {
        int rank = 0;
        for (int i = 0; i < count; ++i) {
            const int v = __ldg(mine + i);
            rank += v < mine_here || (v == mine_here && i < (int)threadIdx.x);
        }
        bits.sorted[rank] = mine_here;
    }
    __syncthreads();
    const auto has = [&](int v) {  // whether the own side has this group
        if (v < own.lo || v > own.hi) return false;
        if (!wide) return (bool)(bits.own[v / 32 % (kGroupBits / 32)] >> (v & 31) & 1);
        int lo = 0, hi = count - 1;  // the last one is own.hi, so one at least is >= v
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (bits.sorted[mid] < v) lo = mid + 1;
            else hi = mid;
        }
        return bits.sorted[lo] == v;
    };
    for (int tile = first + warp; tile < min(last, first + kScan); tile += kAttnWarps) {
        uint32_t meet[2];
        bool clear = true;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = tile * kTile + 32 * half + lane;
            const int v = row < n ? __ldg(other + row) : -1;
            bool seen = v >= 0 && own.hi >= 0;
            if constexpr (kOwnKeys) {
                seen = seen && (own.zero || has(v));
                clear = clear && v >= 0;
            } else {
                seen = seen && (v == 0 || has(v));
                clear = clear && v == 0;
            }
            meet[half] = __ballot_sync(0xffffffffu, seen);
        }
        if constexpr (kOwnKeys) clear = clear && count == kTile && own.all_zero;
        clear = __all_sync(0xffffffffu, clear);
        if (lane == 0) {
            const int i = tile - first;
            bits.rows[i] = make_uint2(meet[0], meet[1]);
            if (meet[0] | meet[1]) atomicOr(&bits.need[i >> 5], 1u << (i & 31));
            if (clear) atomicOr(&bits.clear[i >> 5], 1u << (i & 31));
        }
    }
    __syncthreads();
}

// The first needed tile from `tile` on among those looked up, else `last`.
__device__ __forceinline__ int next_tile(const TileBits& bits, int tile, int first, int last)
{
    const int end = min(last, first + kScan) - first;
    int i = tile - first;
    while (i < end) {
        const uint32_t w = bits.need[i >> 5] >> (i & 31);
        if (w) {
            i += __ffs(w) - 1;
            return i < end ? first + i : last;
        }
        i = (i | 31) + 1;
    }
    return last;
}

// The tiles from `first` on, up to `last`: all of them without groups, those
// that have been looked up with.
template <bool kGroups>
struct Tiles {
    const TileBits& bits;
    int first, last;
    int full;  // without groups: tiles below it have no pair masked

    __device__ __forceinline__ int next(int tile) const
    {
        return kGroups ? next_tile(bits, tile, first, last) : min(tile, last);
    }
    __device__ __forceinline__ bool clear(int tile) const
    {
        const int i = tile - first;
        return kGroups ? (bits.clear[i >> 5] >> (i & 31)) & 1 : tile < full;
    }
    // The rows of a tile that are read; `clear` tiles are read as a whole.
    __device__ __forceinline__ uint2 rows(int tile) const
    {
        return kGroups ? bits.rows[tile - first] : make_uint2(~0u, ~0u);
    }
    // Where the tiles after these start.
    __device__ __forceinline__ int end() const { return kGroups ? first + kScan : last; }
};

__device__ __forceinline__ bool sees(int q_group, int k_group)
{
    return q_group >= 0 && k_group >= 0 && (k_group == 0 || k_group == q_group);
}

// Rows whose scores are far from zero: the logarithm of a weight is a score minus a
// reference, each times scale and log2 e; taken as one multiply-add it keeps the
// rounding of the reference's product, 2^-12 at kFarLog2 and without bound beyond.  Far
// rows take the reference off first.  (A row that sees nothing has -infinity here.)
constexpr float kFarLog2 = 4096.0f;
__device__ __forceinline__ bool is_far(float reference_log2)
{
    return fabsf(reference_log2) > kFarLog2 && fabsf(reference_log2) != INFINITY;
}

// tau, negated and in units of q . k
__device__ __forceinline__ float tau_units(float tau, float scale) { return -tau / scale; }

// A far row's lse, from its reference (a score in units of q . k) and the sum of its
// weights, and the logarithm of one of its weights from lse.  Neither is contracted, so
// that where the sum is 1 the key that lse comes from has the weight 1 at any size.
__device__ __forceinline__ float far_lse(float reference, float scale, float sum)
{
    return __fadd_rn(__fmul_rn(reference, scale), log2f(sum) * kLn2);
}

__device__ __forceinline__ float far_log2(float score, float scale, float lse)
{
    return __fmul_rn(__fsub_rn(__fmul_rn(score, scale), lse), kLog2e);
}

// Distances of a row's point (given negated, nx and ny) from two points.
__device__ __forceinline__ float2 distances(float nx, float ny, float2 x, float2 y)
{
    const float2 dx = __fadd2_rn(x, both(nx)), dy = __fadd2_rn(y, both(ny));
    const float2 d = __ffma2_rn(dx, dx, __fmul2_rn(dy, dy));
    return make_float2(sqrt_approx(d.x), sqrt_approx(d.y));
}

// The points of a tile, x and y apart so that two neighbours load as a pair.
struct Points {
    alignas(8) float x[kTile];
    alignas(8) float y[kTile];
};

// The points and groups of the tile's rows r0 .. r0 + 63 of an item.
template <bool kBias, bool kGroups>
__device__ __forceinline__ void load_columns(Points& pos, int32_t* group, const float2* points,
                                             const int32_t* groups, int64_t first, int r0, int n)
{
    if (threadIdx.x >= kTile) return;
    const int row = r0 + (int)threadIdx.x;
    const bool on = row < n;
    if constexpr (kBias) {
        const float2* src = on ? points + first + row : points;
        cp_async<4>(smem_addr(&pos.x[threadIdx.x]), &src->x, on);
        cp_async<4>(smem_addr(&pos.y[threadIdx.x]), &src->y, on);
    }
    if constexpr (kGroups)
        cp_async<4>(smem_addr(group + threadIdx.x), on ? groups + first + row : groups, on);
}

// The address of the word at `addr` of this CTA's shared memory in CTA `rank` of the
// cluster.
__device__ __forceinline__ uint32_t remote_addr(uint32_t addr, int rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float remote_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float2 remote_f32x2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float4 remote_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

constexpr int kMaxSplits = 8;  // CTAs of a cluster, on any GPU with clusters
constexpr int kSms = 148;

// How many CTAs share the keys of 64 queries, and how many heads a CTA has.
// Two heads share the distances, where that still fills the GPU (below it more
// and shorter CTAs are faster).  The keys are split until the CTAs fill a wave,
// down to two tiles per CTA, and of long rows where it evens out the last wave:
// 628 CTAs in waves of 592 take two of them (704 us for the 100 x 100 grid),
// quartered they take five a quarter as long (571 us).  With groups only the fill
// counts: the tiles that a CTA needs are few and lie together, and parts of a row
// without any still look them up (10 000 queries in seven equal documents one after
// the other: 267 us, with even waves 404 us; in one shared group 776 against 636 us).
struct Plan {
    int heads, splits, split_tiles;
};

// Whether the weights (and ds, in the gradient) keep 16 bits, as two bf16 in two
// products, instead of 8.  With 8 bits an output is off by sqrt(2) of its own
// rounding on average; over thousands of rows that is what it is, among the few of a
// decoding step a single one stands out.  Those leave most of the GPU idle, so
// that the second product costs them least: one query over 4097 keys, 16 heads,
// 15.0 us on the GPU instead of 13.9.  40 000 rows (5000 queries) are spared it: 203 us
// instead of 176, and 479 instead of 385 for the gradient's second kernel.
constexpr int64_t kExactRows = 1024;
inline bool exact_of(int64_t rows) { return rows <= kExactRows; }

Plan plan_of(int B, int Nq, int Nk, int H, bool bias, bool groups, int blocks);

// Device copy of the inputs.
struct Inputs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float2 *qp, *kp;
    const float* tau;
    const int32_t *qg, *kg;
    float scale;
    int B, Nq, Nk, H;
};

Inputs inputs_of(const msda_attention_t& p);
// The checks that the forward and the backward share.
msda_status_t check_inputs(const msda_attention_t* p, bool& empty);
// Whether [out, out + bytes) shares memory with the rows of q, k or v.
bool touches_inputs(const msda_attention_t* p, const void* out, size_t bytes);
msda_status_t check_workspace(const void* ws, size_t have, size_t need);

}  // namespace attn
}  // namespace msda
