// Shared by the forward and the backward of msda_query_attention: the warp's
// matrix fragments, tile loads, visibility and the distance of points.
//
// A warp holds 16 rows of one side (queries; keys in the gradient of k and v)
// and walks tiles of 64 rows of the other, which the CTA's four warps share in
// shared memory.  With 32 channels per head a score takes 32 multiply-adds in
// each product but also an exponential (16 per clock and SM) and, with the
// bias, a square root and about ten instructions: the matrix pipe is not what
// binds, and the fragments of mma.sync leave every score in the thread that
// computes on it.  A square root serves all heads of a warp.
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
constexpr int kScan = 2048;         // tiles whose visibility is looked up at once
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// c += a b for a 16 x 16 by 16 x 8 product.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// B fragments of the product with a tile's rows as columns (scores): all 32
// channels of the rows 8j .. 8j + 7; r[0], r[1] for channels 0..15, r[2], r[3]
// for 16..31.
__device__ __forceinline__ void load_cols(uint32_t (&r)[4], uint32_t tile, int j, int lane)
{
    ldsm(r, tile + tile_at(8 * j + (lane & 7), lane >> 3));
}

// B fragments of the product that sums over a tile's rows 16k .. 16k + 15:
// r[0], r[1] for channels 8d .. 8d + 7, r[2], r[3] for the eight after them.
__device__ __forceinline__ void load_sum(uint32_t (&r)[4], uint32_t tile, int k, int d, int lane)
{
    ldsm_t(r, tile + tile_at(16 * k + (lane & 15), d + (lane >> 4)));
}

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

// The groups on one side, as far as visibility goes: the range of those >= 0,
// whether 0 is among them, and whether all are 0.
struct GroupRange {
    int lo, hi;
    bool any, zero, all_zero;
};

__device__ __forceinline__ GroupRange warp_range(const int32_t* g, int64_t at, int count)
{
    int lo = INT32_MAX, hi = -1;
    bool zero = false, all = true;
    for (int i = threadIdx.x & 31; i < count; i += 32) {
        const int v = __ldg(g + at + i);
        if (v >= 0) {
            lo = min(lo, v);
            hi = max(hi, v);
        }
        zero |= v == 0;
        all &= v == 0;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    return {lo, hi, hi >= 0, (bool)__any_sync(0xffffffffu, zero),
            (bool)__all_sync(0xffffffffu, all)};
}

// Tiles of the other side that some row of the own side needs (bit set in
// `need`), and those in which no pair is masked (`clear`), for kScan tiles
// from `first` on.  kOwnKeys: the own side are keys and the other queries.
struct TileBits {
    uint32_t need[kScan / 32], clear[kScan / 32];
};

template <bool kOwnKeys>
__device__ void scan_tiles(TileBits& bits, const GroupRange& own, bool own_full,
                           const int32_t* other, int64_t at, int n, int first, int last)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = threadIdx.x; w < kScan / 32; w += kAttnThreads) bits.need[w] = bits.clear[w] = 0;
    __syncthreads();
    for (int tile = first + warp; tile < min(last, first + kScan); tile += kAttnWarps) {
        const int r0 = tile * kTile, count = min(kTile, n - r0);
        bool need = true, clear = count == kTile;
        if (other != nullptr) {
            const GroupRange g = warp_range(other, at + r0, count);
            const bool meet = g.any && own.any && g.lo <= own.hi && own.lo <= g.hi;
            if constexpr (kOwnKeys) {
                need = meet || (own.zero && g.any);
                clear = clear && own_full && own.all_zero && g.any &&
                        __all_sync(0xffffffffu, __ldg(other + at + r0 + min(lane, count - 1)) >= 0 &&
                                                    __ldg(other + at + r0 +
                                                          min(lane + 32, count - 1)) >= 0);
            } else {
                need = own.any && (meet || g.zero);
                clear = clear && g.all_zero;
            }
        } else if (kOwnKeys) {
            clear = clear && own_full;
        }
        if (lane == 0) {
            const int i = tile - first;
            if (need) atomicOr(&bits.need[i >> 5], 1u << (i & 31));
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

__device__ __forceinline__ bool sees(int q_group, int k_group)
{
    return q_group >= 0 && k_group >= 0 && (k_group == 0 || k_group == q_group);
}

__device__ __forceinline__ float distance(float2 a, float x, float y)
{
    const float dx = a.x - x, dy = a.y - y;
    return sqrt_approx(fmaf(dx, dx, dy * dy));
}

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
