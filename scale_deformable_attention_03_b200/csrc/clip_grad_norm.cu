// msda_clip_grad_norm: the global norm of a list of gradient tensors and their
// clipping by it.
//   total = scale * sqrt(sum g^2),  out = g * scale * min(1, max / (total + eps))
// Two passes, because every output needs the norm of all inputs: one reads the
// gradients and leaves one partial sum of squares per CTA, the other adds the
// partial sums (each CTA for itself, in the same order, so no flag, no atomic
// and no third launch), reads the gradients again and writes.  Both passes
// take the tensors as one row of tiles; the second walks it backwards, so that
// what the first read last is still in L2 (126 MB).
//
// Bound by memory: 4 bytes in and 4 out per fp32 value once; the second read
// comes from L2 as far as that reaches.  A square of an fp32 value is exact in
// double, and a conversion and a double fused multiply-add per value stay
// below the rate at which the values arrive (16 and 64 per clock and SM
// against about 6).
//
// The tensor table travels in the kernel's parameters (32 bytes a tensor): no
// copy to the device, so the call can be captured and the host array may go
// as soon as the call returns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "msda.h"
#include "msda_launch.h"

namespace msda {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipTile = 8192;        // values per tile: 32 per thread
constexpr int kClipMaxGrid = 2048;     // partial sums per launch
constexpr int kClipSmallTable = 64;    // a short list travels in 2 KB of parameters,
constexpr int kClipLargeTable = 960;   // a long one in 31 KB (the limit is 32764 bytes)

struct ClipEntry {
    const void* src;
    void* dst;
    int64_t numel;
    int32_t first_tile;
    uint8_t src_bf16, dst_bf16, mis;  // mis: values from the 16-byte boundary at or below src
    uint8_t co_aligned;               // dst moves in step with src's 16-byte groups
};

template <int N>
struct ClipTable {
    int32_t n, tiles;
    ClipEntry e[N];
};

__device__ __forceinline__ float bf16_bits(uint32_t h) { return __uint_as_float(h << 16); }

// Values per 16 bytes of the source type.
template <bool kBf16>
constexpr int kVec = kBf16 ? 8 : 4;

template <bool kBf16>
__device__ __forceinline__ void unpack(uint4 r, float (&v)[kVec<kBf16>])
{
    if constexpr (kBf16) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_bits(w[i]);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
}

template <bool kBf16>
__device__ __forceinline__ float load_one(const void* p, int64_t i)
{
    if constexpr (kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_one(void* p, int64_t i, float v, bool bf16)
{
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p)[i] = v;
}

// The tensor that holds a tile: the last whose first tile is at or below it
// (tensors without values have no tile and share the next one's first).
template <int N>
__device__ __forceinline__ int find_tensor(const ClipTable<N>& t, int tile)
{
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].first_tile <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Tile `k` of a tensor covers the values [k * kClipTile - mis, + kClipTile) of
// it: every group of kVec values in it starts on a 16-byte boundary, and only
// the tensor's first and last group can be cut.
template <bool kBf16>
__device__ __forceinline__ double tile_squares(const ClipEntry& e, int64_t k)
{
    constexpr int V = kVec<kBf16>, kIter = kClipTile / (kClipThreads * V);
    const int64_t base = k * kClipTile - e.mis;
    const char* src = static_cast<const char*>(e.src) + base * (kBf16 ? 2 : 4);
    uint4 r[kIter];
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int g = i * kClipThreads + (int)threadIdx.x;
        const int64_t at = base + (int64_t)g * V;
        r[i] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && at + V <= e.numel) r[i] = __ldg(reinterpret_cast<const uint4*>(src) + g);
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        float v[V];
        unpack<kBf16>(r[i], v);
#pragma unroll
        for (int j = 0; j < V; ++j) s = fma((double)v[j], (double)v[j], s);
    }
    // the cut groups: at most one at each end of the tensor
    if (base < 0 || base + kClipTile > e.numel) {
        for (int g = threadIdx.x; g < kClipTile / V; g += kClipThreads) {
            const int64_t at = base + (int64_t)g * V;
            if (at >= e.numel || at + V <= 0 || (at >= 0 && at + V <= e.numel)) continue;
            for (int j = 0; j < V; ++j)
                if (at + j >= 0 && at + j < e.numel) {
                    const double v = (double)load_one<kBf16>(e.src, at + j);
                    s = fma(v, v, s);
                }
        }
    }
    return s;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads) clip_squares_kernel(
    const __grid_constant__ ClipTable<N> t, double* __restrict__ partial)
{
    pdl_trigger();
    double s = 0.0;
    for (int tile = blockIdx.x; tile < t.tiles; tile += gridDim.x) {
        const int i = find_tensor(t, tile);
        const int64_t k = tile - t.e[i].first_tile;
        s += t.e[i].src_bf16 ? tile_squares<true>(t.e[i], k) : tile_squares<false>(t.e[i], k);
    }
    __shared__ double warp_sum[kClipThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kClipThreads / 32; ++w) s += warp_sum[w];
        partial[blockIdx.x] = s;
    }
}

template <bool kSrc, bool kDst>
__device__ __forceinline__ void tile_scale(const ClipEntry& e, int64_t k, float f)
{
    constexpr int V = kVec<kSrc>, kIter = kClipTile / (kClipThreads * V);
    const int64_t base = k * kClipTile - e.mis;
    if (!e.co_aligned) {  // out starts elsewhere in its 16 bytes: a value per lane
        for (int g = threadIdx.x; g < kClipTile; g += kClipThreads) {
            const int64_t at = base + g;
            if (at >= 0 && at < e.numel)
                store_one(e.dst, at, load_one<kSrc>(e.src, at) * f, kDst);
        }
        return;
    }
    const char* src = static_cast<const char*>(e.src) + base * (kSrc ? 2 : 4);
    char* dst = static_cast<char*>(e.dst) + base * (kDst ? 2 : 4);
    uint4 r[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int g = i * kClipThreads + (int)threadIdx.x;
        const int64_t at = base + (int64_t)g * V;
        if (at >= 0 && at + V <= e.numel) r[i] = *(reinterpret_cast<const uint4*>(src) + g);
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int g = i * kClipThreads + (int)threadIdx.x;
        const int64_t at = base + (int64_t)g * V;
        if (at >= 0 && at + V <= e.numel) {
            float v[V];
            unpack<kSrc>(r[i], v);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= f;
            if constexpr (kDst) {
                uint32_t w[V / 2];
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&h);
                }
                if constexpr (V == 8)
                    __stcs(reinterpret_cast<uint4*>(dst) + g, make_uint4(w[0], w[1], w[2], w[3]));
                else
                    __stcs(reinterpret_cast<uint2*>(dst) + g, make_uint2(w[0], w[1]));
            } else {
#pragma unroll
                for (int j = 0; j < V / 4; ++j)
                    __stcs(reinterpret_cast<float4*>(dst) + g * (V / 4) + j,
                           make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
            }
        }
    }
    if (base < 0 || base + kClipTile > e.numel) {
        for (int g = threadIdx.x; g < kClipTile / V; g += kClipThreads) {
            const int64_t at = base + (int64_t)g * V;
            if (at >= e.numel || at + V <= 0 || (at >= 0 && at + V <= e.numel)) continue;
            for (int j = 0; j < V; ++j)
                if (at + j >= 0 && at + j < e.numel)
                    store_one(e.dst, at + j, load_one<kSrc>(e.src, at + j) * f, kDst);
        }
    }
}

// (no __restrict__ on what the pass before writes while this one has begun)
template <int N>
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(
    const __grid_constant__ ClipTable<N> t, const double* partial, int partials, float max_norm,
    float eps, float scale, float* total_norm)
{
    __shared__ double warp_sum[kClipThreads / 32];
    __shared__ float factor;
    pdl_wait();
    double s = 0.0;
    for (int i = threadIdx.x; i < partials; i += kClipThreads) s += partial[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kClipThreads / 32; ++w) s += warp_sum[w];
        const double norm = sqrt(s) * (double)scale;
        double c = isinf(max_norm) ? 1.0 : (double)max_norm / (norm + (double)eps);
        if (c > 1.0) c = 1.0;  // a NaN stays
        factor = (float)(c * (double)scale);
        if (total_norm != nullptr && blockIdx.x == 0) *total_norm = (float)norm;
    }
    __syncthreads();
    const float f = factor;
    for (int tile = t.tiles - 1 - (int)blockIdx.x; tile >= 0; tile -= gridDim.x) {
        const int i = find_tensor(t, tile);
        const ClipEntry& e = t.e[i];
        // a gradient kept in place and not clipped is what it was
        if (e.dst == nullptr || (f == 1.0f && e.dst == e.src)) continue;
        const int64_t k = tile - e.first_tile;
        if (e.src_bf16) {
            if (e.dst_bf16) tile_scale<true, true>(e, k, f);
            else tile_scale<true, false>(e, k, f);
        } else {
            if (e.dst_bf16) tile_scale<false, true>(e, k, f);
            else tile_scale<false, false>(e, k, f);
        }
    }
}

int clip_grid(int tiles)
{
    // eight CTAs of 256 threads fill an SM; one CTA at least, for the norm of nothing
    return std::max(1, std::min(tiles, std::min(kClipMaxGrid, 8 * device_sm_count())));
}

int dtype_bytes(msda_dtype_t d) { return d == MSDA_BF16 ? 2 : 4; }

template <int N>
bool fill_table(ClipTable<N>& t, const msda_grad_t* g, int n)
{
    int64_t tiles = 0;
    t.n = n;
    for (int i = 0; i < n; ++i) {
        ClipEntry& e = t.e[i];
        const int sb = dtype_bytes(g[i].grad_dtype), ob = dtype_bytes(g[i].out_dtype);
        const int vec = 16 / sb;
        e.src = g[i].grad;
        e.dst = g[i].out;
        e.numel = g[i].numel;
        e.first_tile = (int32_t)tiles;
        e.src_bf16 = g[i].grad_dtype == MSDA_BF16;
        e.dst_bf16 = g[i].out_dtype == MSDA_BF16;
        e.mis = (uint8_t)(((uintptr_t)e.src % 16) / sb);
        // the store of one group: vec values of out, at most 16 bytes at a time
        e.co_aligned = ((uintptr_t)e.dst - (uintptr_t)e.mis * ob) % std::min(16, vec * ob) == 0;
        if (e.numel > 0) tiles += (e.numel + e.mis + kClipTile - 1) / kClipTile;
        if (tiles > INT32_MAX - 65536) return false;
    }
    t.tiles = (int32_t)tiles;
    return true;
}

struct ClipRange {
    uintptr_t lo, hi;
};

// No byte belongs to two tensors, or to one tensor's grad and its out (but for
// out == grad, which is one range here).
bool ranges_disjoint(std::vector<ClipRange>& r)
{
    const auto before = [](const ClipRange& a, const ClipRange& b) { return a.lo < b.lo; };
    if (!std::is_sorted(r.begin(), r.end(), before)) std::sort(r.begin(), r.end(), before);
    for (size_t i = 1; i < r.size(); ++i)
        if (r[i].lo < r[i - 1].hi) return false;
    return true;
}

template <int N>
msda_status_t run_clip(const msda_grad_t* tensors, int count, float max_norm, float eps,
                       float scale, double* partial, float* total_norm, cudaStream_t s)
{
    ClipTable<N> t;  // at most 31 KB of stack
    // (the first part is filled last, and first to be launched)
    for (int at = (count - 1) / N * N; at >= 0; at -= N)
        if (!fill_table(t, tensors + at, std::min(N, count - at)))
            return api_fail(MSDA_ERR_UNSUPPORTED, "the tensors hold too many values");
    int partials = 0;
    for (int at = 0; at == 0 || at < count; at += N) {
        if (at > 0) fill_table(t, tensors + at, std::min(N, count - at));
        const int grid = clip_grid(t.tiles);
        clip_squares_kernel<N><<<grid, kClipThreads, 0, s>>>(t, partial + partials);
        partials += grid;
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return api_cuda(e, "msda_clip_grad_norm");
    }
    for (int at = 0; at == 0 || at < count; at += N) {
        if (count > N) fill_table(t, tensors + at, std::min(N, count - at));
        // the first may begin while the last pass of sums ends; a later one
        // starts after its predecessor, which has waited for the sums
        cudaError_t e;
        if (at == 0) {
            e = launch_pdl(clip_scale_kernel<N>, dim3(clip_grid(t.tiles)), dim3(kClipThreads), 0,
                           s, t, partial, partials, max_norm, eps, scale, total_norm);
        } else {
            clip_scale_kernel<N><<<clip_grid(t.tiles), kClipThreads, 0, s>>>(
                t, partial, partials, max_norm, eps, scale, (float*)nullptr);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess) return api_cuda(e, "msda_clip_grad_norm");
    }
    return api_ok();
}

}  // namespace
}  // namespace msda

using namespace msda;

extern "C" size_t msda_clip_grad_norm_workspace_size(int32_t count)
{
    const size_t launches =
        count <= 0 ? 1 : ((size_t)count + kClipLargeTable - 1) / kClipLargeTable;
    return launches * kClipMaxGrid * sizeof(double);
}

extern "C" msda_status_t msda_clip_grad_norm(const msda_grad_t* tensors, int32_t count,
                                             float max_norm, float eps, float grad_scale,
                                             void* workspace, size_t workspace_bytes,
                                             float* total_norm, msda_stream_t stream)
{
    if (count < 0) return api_failf(MSDA_ERR_INVALID_ARG, "count = %d is negative", count);
    if (count > 0 && tensors == nullptr)
        return api_fail(MSDA_ERR_INVALID_ARG, "tensors is null");
    if (!(max_norm >= 0.0f))
        return api_failf(MSDA_ERR_INVALID_ARG, "max_norm = %g must be >= 0", (double)max_norm);
    if (!(eps > 0.0f) || std::isinf(eps))
        return api_failf(MSDA_ERR_INVALID_ARG, "eps = %g must be finite and > 0", (double)eps);
    if (!(grad_scale > 0.0f) || std::isinf(grad_scale))
        return api_failf(MSDA_ERR_INVALID_ARG, "grad_scale = %g must be finite and > 0",
                         (double)grad_scale);
    if (total_norm == nullptr || (uintptr_t)total_norm % 4)
        return api_fail(MSDA_ERR_INVALID_ARG, "total_norm is null or not 4-byte aligned");
    if (workspace == nullptr || workspace_bytes < msda_clip_grad_norm_workspace_size(count) ||
        (uintptr_t)workspace % 256)
        return api_failf(MSDA_ERR_WORKSPACE,
                         "workspace of %zu bytes: %zu bytes on a 256-byte boundary are needed",
                         workspace == nullptr ? (size_t)0 : workspace_bytes,
                         msda_clip_grad_norm_workspace_size(count));
    try {
        std::vector<ClipRange> ranges;
        ranges.reserve(2 * (size_t)count + 2);
        for (int i = 0; i < count; ++i) {
            const msda_grad_t& g = tensors[i];
            if (g.grad_dtype != MSDA_F32 && g.grad_dtype != MSDA_BF16)
                return api_failf(MSDA_ERR_INVALID_ARG, "tensor %d: unknown grad dtype %d", i,
                                 (int)g.grad_dtype);
            if (g.out_dtype != MSDA_F32 && g.out_dtype != MSDA_BF16)
                return api_failf(MSDA_ERR_INVALID_ARG, "tensor %d: unknown out dtype %d", i,
                                 (int)g.out_dtype);
            if (g.numel < 0 || g.numel > ((int64_t)1 << 44))
                return api_failf(MSDA_ERR_INVALID_ARG, "tensor %d has %lld values", i,
                                 (long long)g.numel);
            if (g.numel == 0) continue;
            const size_t sb = dtype_bytes(g.grad_dtype), ob = dtype_bytes(g.out_dtype);
            const uintptr_t src = (uintptr_t)g.grad, dst = (uintptr_t)g.out;
            if (src == 0) return api_failf(MSDA_ERR_INVALID_ARG, "tensor %d: grad is null", i);
            if (src % sb || dst % ob)
                return api_failf(MSDA_ERR_INVALID_ARG,
                                 "tensor %d is not aligned to its type", i);
            const bool in_place = src == dst;
            if (in_place && sb != ob)
                return api_failf(MSDA_ERR_INVALID_ARG, "tensor %d: in place, with two dtypes", i);
            ranges.push_back({src, src + (size_t)g.numel * sb});
            if (dst != 0 && !in_place) ranges.push_back({dst, dst + (size_t)g.numel * ob});
        }
        const uintptr_t ws = (uintptr_t)workspace, tn = (uintptr_t)total_norm;
        ranges.push_back({ws, ws + msda_clip_grad_norm_workspace_size(count)});
        ranges.push_back({tn, tn + sizeof(float)});
        if (!ranges_disjoint(ranges))
            return api_fail(MSDA_ERR_INVALID_ARG,
                            "two tensors overlap (or one is listed twice, or overlaps the "
                            "workspace or total_norm)");
    } catch (const std::bad_alloc&) {
        return api_fail(MSDA_ERR_INVALID_ARG, "no host memory to check the tensors");
    }
    double* partial = static_cast<double*>(workspace);
    const cudaStream_t s = (cudaStream_t)stream;
    return count <= kClipSmallTable
               ? run_clip<kClipSmallTable>(tensors, count, max_norm, eps, grad_scale, partial,
                                           total_norm, s)
               : run_clip<kClipLargeTable>(tensors, count, max_norm, eps, grad_scale, partial,
                                           total_norm, s);
}
