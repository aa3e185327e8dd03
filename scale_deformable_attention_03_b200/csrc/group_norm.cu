// msda_group_norm and its backward: group norm with an activation over the
// levels of channels-last rows [B, Nv, C].
//
// Forward, per (item, level, group) with N = rows * C/G values:
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//   y = act(gamma (x - mu) r + beta)
// Backward, with xh = (x - mu) r, dz = dy act'(z), t = gamma dz:
//   dgamma = sum dz xh, dbeta = sum dz, dx = r (t - mean(t) - xh mean(t xh))
//
// Both are two passes over the rows with a small merge between them: every
// value needs sums over its whole level.  A pass takes chunks of rows, one CTA
// each.  A thread holds eight neighbouring channels (16 bytes of bf16, 32 of
// fp32) of kRowsPerThread rows, so its channels' constants stay in registers
// and a warp reads whole rows.  The second pass walks the chunks backwards:
// what the first one read last is still in L2.  The launches are programmatic
// dependents of one another, so the second pass has its first rows in
// registers while the merge ends.
//
// Bound by memory.  The three sums over a chunk stay in registers, then in
// shared memory; a chunk leaves 16 bytes per group (forward) or 8 per channel
// (backward), about 1 % of the data.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "msda.h"
#include "msda_launch.h"

namespace msda {
namespace {

constexpr int kNormThreads = 256;
constexpr int kRowsPerThread = 8;
constexpr int kMaxC = MSDA_NORM_MAX_CHANNELS;
constexpr int kMergeThreads = 512;  // 32 groups or channels wide, 16 chunks at a time

struct NormShape {
    int B, Nv, C, L, G, cg;         // cg = C / G
    int tpr, slots, chunk_rows;     // threads per row, rows at a time, rows per chunk
    int chunks;                     // per item, over all levels
    int start[kMaxLevels], rows[kMaxLevels], chunk0[kMaxLevels + 1];
    int gaps, gap_chunks;           // runs of rows in no level
    int gap_start[kMaxLevels + 1], gap_rows[kMaxLevels + 1];
};

struct ChunkAt {
    int l, row, rows;  // level, first row within the item, rows
};

__device__ __forceinline__ ChunkAt chunk_at(const NormShape& n, int chunk)
{
    int l = 0;
    while (l + 1 < n.L && n.chunk0[l + 1] <= chunk) ++l;
    const int at = (chunk - n.chunk0[l]) * n.chunk_rows;
    return {l, n.start[l] + at, min(n.chunk_rows, n.rows[l] - at)};
}

struct Vec8 {
    float v[8];
};

template <bool kBf16>
struct Raw8 {  // eight values as they are stored
    uint4 a[kBf16 ? 1 : 2];
};

template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load8(const void* p, int64_t i)
{
    Raw8<kBf16> r;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) +
                                                    i * (kBf16 ? 2 : 4));
    r.a[0] = __ldg(q);
    if constexpr (!kBf16) r.a[1] = __ldg(q + 1);
    return r;
}

template <bool kBf16>
__device__ __forceinline__ Vec8 widen(const Raw8<kBf16>& r)
{
    Vec8 o;
    const uint32_t w[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
    if constexpr (kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.v[2 * i] = __uint_as_float(w[i] << 16);
            o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const uint32_t u[4] = {r.a[1].x, r.a[1].y, r.a[1].z, r.a[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o.v[i] = __uint_as_float(w[i]);
            o.v[4 + i] = __uint_as_float(u[i]);
        }
    }
    return o;
}

template <bool kBf16>
__device__ __forceinline__ void store8(void* p, int64_t i, const Vec8& o)
{
    if constexpr (kBf16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o.v[2 * j], o.v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<char*>(p) + i * 2),
               make_uint4(w[0], w[1], w[2], w[3]));
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<char*>(p) + i * 4);
        __stcs(q, make_float4(o.v[0], o.v[1], o.v[2], o.v[3]));
        __stcs(q + 1, make_float4(o.v[4], o.v[5], o.v[6], o.v[7]));
    }
}

__device__ __forceinline__ Vec8 load_channels(const float* p, int64_t i, float otherwise)
{
    Vec8 o;
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] = otherwise;
        return o;
    }
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p + i) + 1);
    o = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    return o;
}

// Adds the slots' sums of two quantities per channel: on return s[0][0][c] and
// s[1][0][c] hold the chunk's sums of channel c (for the thread that owns it,
// threads c mod kNormThreads; a barrier before others read them).
__device__ __forceinline__ void add_slots(float* s, int C, int slots)
{
    __syncthreads();
    float* s2 = s + kNormThreads * 8;
    for (int c = threadIdx.x; c < C; c += kNormThreads) {
        float a = s[c], b = s2[c];
        for (int k = 1; k < slots; ++k) {
            a += s[k * C + c];
            b += s2[k * C + c];
        }
        s[c] = a;
        s2[c] = b;
    }
}

__device__ __forceinline__ void put_slot(float* s, int C, int slot, int c, const Vec8& a,
                                         const Vec8& b)
{
    float* p = s + slot * C + c;
    float* q = p + kNormThreads * 8;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
        *reinterpret_cast<float4*>(p + j) = make_float4(a.v[j], a.v[j + 1], a.v[j + 2], a.v[j + 3]);
        *reinterpret_cast<float4*>(q + j) = make_float4(b.v[j], b.v[j + 1], b.v[j + 2], b.v[j + 3]);
    }
}

// ---------------------------------------------------------------- forward

// A chunk's mean and sum of squared distances from it, per group.  Within a
// channel both come from sums relative to the chunk's first row (which keeps
// their size that of the channel's spread), in fp32 over the chunk's rows; the
// channels are merged in double.
template <bool kX>
__global__ void __launch_bounds__(kNormThreads) norm_stats_kernel(const void* __restrict__ x,
                                                                  const NormShape n,
                                                                  double2* __restrict__ part)
{
    __shared__ __align__(16) float s[2 * kNormThreads * 8];
    __shared__ float first[kMaxC];
    pdl_trigger();
    const int b = blockIdx.x / n.chunks, chunk = blockIdx.x - b * n.chunks;
    const ChunkAt at = chunk_at(n, chunk);
    const int slot = threadIdx.x / n.tpr, c = (threadIdx.x - slot * n.tpr) * 8;
    const int64_t base = ((int64_t)b * n.Nv + at.row) * n.C + c;
    if (slot < n.slots) {
        const Raw8<kX> r0 = load8<kX>(x, base);
        Raw8<kX> r[kRowsPerThread];
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const int row = slot + i * n.slots;
            if (row < at.rows) r[i] = load8<kX>(x, base + (int64_t)row * n.C);
        }
        const Vec8 ref = widen(r0);
        Vec8 a{}, q{};
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            if (slot + i * n.slots < at.rows) {
                const Vec8 v = widen(r[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = v.v[j] - ref.v[j];
                    a.v[j] += d;
                    q.v[j] = fmaf(d, d, q.v[j]);
                }
            }
        }
        put_slot(s, n.C, slot, c, a, q);
        if (slot == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) first[c + j] = ref.v[j];
        }
    }
    add_slots(s, n.C, n.slots);
    __syncthreads();
    // lanes per group: a power of two, so that several small groups share a warp
    int seg = 1;
    while (seg < 32 && seg < n.cg) seg <<= 1;
    const int per_warp = 32 / seg, lane = threadIdx.x & 31, sub = lane / seg, in = lane - sub * seg;
    const double rows = (double)at.rows, inv_rows = 1.0 / rows;
    for (int g0 = (threadIdx.x >> 5) * per_warp; g0 < n.G; g0 += (kNormThreads / 32) * per_warp) {
        const int g = g0 + sub;
        const bool on = g < n.G;
        double sum = 0.0;
        for (int k = in; on && k < n.cg; k += seg) {
            const int ch = g * n.cg + k;
            sum += (double)first[ch] + (double)s[ch] * inv_rows;
        }
        for (int o = seg >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const double mean = sum / (double)n.cg;
        double m2 = 0.0;
        for (int k = in; on && k < n.cg; k += seg) {
            const int ch = g * n.cg + k;
            const double a = s[ch], d = (double)first[ch] + a * inv_rows - mean;
            m2 += (double)s[kNormThreads * 8 + ch] - a * a * inv_rows + rows * d * d;
        }
        for (int o = seg >> 1; o > 0; o >>= 1) m2 += __shfl_xor_sync(0xffffffffu, m2, o);
        if (on && in == 0) part[((int64_t)b * n.chunks + chunk) * n.G + g] = make_double2(mean, m2);
    }
}

// Merges the chunks of one (item, level), 32 groups per CTA, in double and
// relative to the first chunk's mean.  The mean is kept as two floats: what
// the second pass subtracts is then exact to 48 bits, whatever the mean.
__global__ void __launch_bounds__(kMergeThreads) norm_merge_kernel(
    const double2* __restrict__ part, const NormShape n, float eps, float4* __restrict__ stats,
    float* __restrict__ mean_out, float* __restrict__ rstd_out)
{
    __shared__ double2 s[kMergeThreads];
    pdl_trigger();
    const int b = blockIdx.x / n.L, l = blockIdx.x - b * n.L;
    const int lane = threadIdx.x & 31, slot = threadIdx.x >> 5, g = blockIdx.y * 32 + lane;
    const int k0 = n.chunk0[l], k1 = n.chunk0[l + 1];
    const double2* p = part + ((int64_t)b * n.chunks) * n.G + g;
    double a = 0.0, q = 0.0, ref = 0.0;
    pdl_wait();
    if (g < n.G) {
        ref = p[(int64_t)k0 * n.G].x;
#pragma unroll 4
        for (int k = k0 + slot; k < k1; k += kMergeThreads / 32) {
            const double2 v = p[(int64_t)k * n.G];
            const int rows = min(n.chunk_rows, n.rows[l] - (k - k0) * n.chunk_rows);
            const double w = (double)rows * n.cg, d = v.x - ref;
            a += w * d;
            q += v.y + w * d * d;
        }
    }
    s[threadIdx.x] = make_double2(a, q);
    __syncthreads();
    if (slot == 0 && g < n.G) {
        for (int k = 1; k < kMergeThreads / 32; ++k) {
            a += s[k * 32 + lane].x;
            q += s[k * 32 + lane].y;
        }
        const double N = (double)n.rows[l] * n.cg;
        const double mean = ref + a / N;
        double var = (q - a * a / N) / N;
        if (var < 0.0) var = 0.0;  // rounding only; a NaN stays
        const double r = 1.0 / sqrt(var + (double)eps);
        const float hi = (float)mean;
        const int64_t i = ((int64_t)b * n.L + l) * n.G + g;
        stats[i] = make_float4(hi, (float)(mean - (double)hi), (float)r, 0.0f);
        if (mean_out) mean_out[i] = hi;
        if (rstd_out) rstd_out[i] = (float)r;
    }
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + __expf(-z)); }

template <int kAct>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (kAct == MSDA_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (kAct == MSDA_ACT_SILU) return z * sigmoid(z);
    return z;
}

// Rows of no level: zeros.
template <bool kY>
__device__ void zero_gap(const NormShape& n, void* y, int b, int gap_chunk)
{
    int k = 0;
    for (; k < n.gaps; ++k) {
        const int c = (n.gap_rows[k] + n.chunk_rows - 1) / n.chunk_rows;
        if (gap_chunk < c) break;
        gap_chunk -= c;
    }
    if (k == n.gaps) return;
    const int row0 = gap_chunk * n.chunk_rows;
    const int rows = min(n.chunk_rows, n.gap_rows[k] - row0);
    const int64_t base = ((int64_t)b * n.Nv + n.gap_start[k] + row0) * n.C;
    for (int i = threadIdx.x; i < rows * n.tpr; i += kNormThreads)
        store8<kY>(y, base + (int64_t)i * 8, Vec8{});
}

template <bool kX, bool kY, int kAct>
__global__ void __launch_bounds__(kNormThreads) norm_apply_kernel(
    const void* __restrict__ x, const NormShape n, const float4* __restrict__ stats,
    const float* __restrict__ gamma, const float* __restrict__ beta, void* __restrict__ y)
{
    const int per = n.chunks + n.gap_chunks;
    const int id = gridDim.x - 1 - blockIdx.x;
    const int b = id / per, chunk = id - b * per;
    if (chunk >= n.chunks) {
        pdl_wait();
        zero_gap<kY>(n, y, b, chunk - n.chunks);
        return;
    }
    const ChunkAt at = chunk_at(n, chunk);
    const int slot = threadIdx.x / n.tpr, c = (threadIdx.x - slot * n.tpr) * 8;
    if (slot >= n.slots) return;
    const int64_t base = ((int64_t)b * n.Nv + at.row) * n.C + c;
    Raw8<kX> r[kRowsPerThread];
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
        const int row = slot + i * n.slots;
        if (row < at.rows) r[i] = load8<kX>(x, base + (int64_t)row * n.C);
    }
    const Vec8 ga = load_channels(gamma, (int64_t)at.l * n.C + c, 1.0f);
    const Vec8 be = load_channels(beta, (int64_t)at.l * n.C + c, 0.0f);
    Vec8 hi, lo, a;
    pdl_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float4 st = stats[((int64_t)b * n.L + at.l) * n.G + (c + j) / n.cg];
        hi.v[j] = st.x;
        lo.v[j] = st.y;
        a.v[j] = st.z * ga.v[j];
    }
#pragma unroll
    for (int i = 0; i < kRowsPerThread; ++i) {
        const int row = slot + i * n.slots;
        if (row < at.rows) {
            Vec8 v = widen(r[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v.v[j] = activate<kAct>(fmaf((v.v[j] - hi.v[j]) - lo.v[j], a.v[j], be.v[j]));
            store8<kY>(y, base + (int64_t)row * n.C, v);
        }
    }
}

// --------------------------------------------------------------- backward

// dz = dy act'(z).  The side of relu's border is taken exactly: z in fp32 is
// off by less than 2^-22 (|z| + |beta|), so its sign is sure outside a band of
// 1e-6 |beta|; inside it, it is formed again in double.
template <int kAct>
__device__ __forceinline__ float grad_z(float dy, float x, float mean, float rstd, float hat,
                                        float gamma, float beta)
{
    if constexpr (kAct == MSDA_ACT_NONE) return dy;
    const float z = fmaf(hat, gamma, beta);
    if constexpr (kAct == MSDA_ACT_RELU) {
        bool on = z > 0.0f;
        if (fabsf(z) <= fmaf(fabsf(beta), 1e-6f, 1e-37f))
            on = ((double)x - (double)mean) * (double)rstd * (double)gamma + (double)beta > 0.0;
        return on ? dy : 0.0f;
    }
    const float sg = sigmoid(z);
    return dy * sg * fmaf(z, 1.0f - sg, 1.0f);
}

// A thread's eight channels of one level.
struct Channels {
    Vec8 mean, rstd, gamma, beta;
};

__device__ __forceinline__ Channels load_constants(const NormShape& n, int b, int l, int c,
                                                   const float* mean, const float* rstd,
                                                   const float* gamma, const float* beta)
{
    Channels k;
    k.gamma = load_channels(gamma, (int64_t)l * n.C + c, 1.0f);
    k.beta = load_channels(beta, (int64_t)l * n.C + c, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = ((int64_t)b * n.L + l) * n.G + (c + j) / n.cg;
        k.mean.v[j] = __ldg(mean + i);
        k.rstd.v[j] = __ldg(rstd + i);
    }
    return k;
}

constexpr int kBackRows = 4;  // rows in flight: two tensors are read

template <bool kX, bool kDy, int kAct>
__global__ void __launch_bounds__(kNormThreads) norm_grad_sums_kernel(
    const void* __restrict__ x, const void* __restrict__ dy, const NormShape n,
    const float* __restrict__ mean, const float* __restrict__ rstd,
    const float* __restrict__ gamma, const float* __restrict__ beta, float* __restrict__ part)
{
    __shared__ __align__(16) float s[2 * kNormThreads * 8];
    pdl_trigger();
    const int b = blockIdx.x / n.chunks, chunk = blockIdx.x - b * n.chunks;
    const ChunkAt at = chunk_at(n, chunk);
    const int slot = threadIdx.x / n.tpr, c = (threadIdx.x - slot * n.tpr) * 8;
    if (slot < n.slots) {
        const int64_t base = ((int64_t)b * n.Nv + at.row) * n.C + c;
        const Channels k = load_constants(n, b, at.l, c, mean, rstd, gamma, beta);
        Vec8 a{}, q{};
#pragma unroll
        for (int i0 = 0; i0 < kRowsPerThread; i0 += kBackRows) {
            Raw8<kX> rx[kBackRows];
            Raw8<kDy> rd[kBackRows];
#pragma unroll
            for (int i = 0; i < kBackRows; ++i) {
                const int row = slot + (i0 + i) * n.slots;
                if (row < at.rows) {
                    rx[i] = load8<kX>(x, base + (int64_t)row * n.C);
                    rd[i] = load8<kDy>(dy, base + (int64_t)row * n.C);
                }
            }
#pragma unroll
            for (int i = 0; i < kBackRows; ++i) {
                if (slot + (i0 + i) * n.slots < at.rows) {
                    const Vec8 v = widen(rx[i]), d = widen(rd[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float hat = (v.v[j] - k.mean.v[j]) * k.rstd.v[j];
                        const float dz = grad_z<kAct>(d.v[j], v.v[j], k.mean.v[j], k.rstd.v[j],
                                                      hat, k.gamma.v[j], k.beta.v[j]);
                        a.v[j] += dz;
                        q.v[j] = fmaf(dz, hat, q.v[j]);
                    }
                }
            }
        }
        put_slot(s, n.C, slot, c, a, q);
    }
    add_slots(s, n.C, n.slots);
    float* out = part + ((int64_t)b * n.chunks + chunk) * 2 * n.C;
    for (int ch = threadIdx.x; ch < n.C; ch += kNormThreads) {  // the channels it has added itself
        out[ch] = s[ch];
        out[n.C + ch] = s[kNormThreads * 8 + ch];
    }
}

// Adds the chunks of one (item, level) per channel, in double, then the
// channels of each group: grid (B * L, blocks of whole groups), a block of
// groups at least 32 channels wide where the groups are smaller.
__global__ void __launch_bounds__(kMergeThreads) norm_grad_merge_kernel(
    const float* __restrict__ part, const NormShape n, int groups_per_block,
    const float* __restrict__ gamma, double2* __restrict__ chan, float2* __restrict__ coef)
{
    __shared__ double2 s[kMergeThreads];
    pdl_trigger();
    const int b = blockIdx.x / n.L, l = blockIdx.x - b * n.L;
    const int lane = threadIdx.x & 31, slot = threadIdx.x >> 5;
    const int g0 = blockIdx.y * groups_per_block;
    const int c0 = g0 * n.cg, c1 = min(n.C, (g0 + groups_per_block) * n.cg);
    const double inv = 1.0 / ((double)n.rows[l] * n.cg);
    const float* p = part + (int64_t)b * n.chunks * 2 * n.C;
    double t1 = 0.0, t2 = 0.0;  // a group wider than the block: its sums so far (lane 0)
    pdl_wait();
    for (int cb = c0; cb < c1; cb += 32) {
        const int c = cb + lane;
        double a = 0.0, q = 0.0;
        if (c < c1) {
#pragma unroll 4
            for (int k = n.chunk0[l] + slot; k < n.chunk0[l + 1]; k += kMergeThreads / 32) {
                a += (double)p[(int64_t)k * 2 * n.C + c];
                q += (double)p[(int64_t)k * 2 * n.C + n.C + c];
            }
        }
        s[threadIdx.x] = make_double2(a, q);
        __syncthreads();
        if (slot == 0) {
            for (int k = 1; k < kMergeThreads / 32; ++k) {
                a += s[k * 32 + lane].x;
                q += s[k * 32 + lane].y;
            }
            if (c < c1) chan[((int64_t)b * n.L + l) * n.C + c] = make_double2(a, q);
            const double w = c < c1 && gamma != nullptr ? (double)gamma[(int64_t)l * n.C + c] : 1.0;
            a *= w;
            q *= w;
            if (n.cg > 32) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    a += __shfl_xor_sync(0xffffffffu, a, o);
                    q += __shfl_xor_sync(0xffffffffu, q, o);
                }
                t1 += a;
                t2 += q;
            } else {
                __syncwarp();
                s[lane] = make_double2(a, q);
                __syncwarp();
                const int g = g0 + lane;
                if (lane < groups_per_block && g < n.G) {
                    double u1 = 0.0, u2 = 0.0;
                    for (int k = 0; k < n.cg; ++k) {
                        u1 += s[lane * n.cg + k].x;
                        u2 += s[lane * n.cg + k].y;
                    }
                    coef[((int64_t)b * n.L + l) * n.G + g] =
                        make_float2((float)(u1 * inv), (float)(u2 * inv));
                }
            }
        }
        __syncthreads();
    }
    if (n.cg > 32 && threadIdx.x == 0)
        coef[((int64_t)b * n.L + l) * n.G + g0] = make_float2((float)(t1 * inv), (float)(t2 * inv));
}

template <bool kX, bool kDy, bool kDx, int kAct>
__global__ void __launch_bounds__(kNormThreads) norm_grad_apply_kernel(
    const void* __restrict__ x, const void* __restrict__ dy, const NormShape n,
    const float* __restrict__ mean, const float* __restrict__ rstd,
    const float* __restrict__ gamma, const float* __restrict__ beta,
    const double2* __restrict__ chan, const float2* __restrict__ coef, void* __restrict__ dx,
    float* __restrict__ dgamma, float* __restrict__ dbeta)
{
    const int per = n.chunks + n.gap_chunks;
    const int id = n.B * per - 1 - (int)blockIdx.x;
    if (id < 0) {  // the CTAs behind the last chunk add the items' parameter gradients
        const int i = (-1 - id) * kNormThreads + (int)threadIdx.x;
        if (i >= n.L * n.C) return;
        pdl_wait();
        double a = 0.0, q = 0.0;
        for (int b = 0; b < n.B; ++b) {
            const double2 v = chan[(int64_t)b * n.L * n.C + i];
            a += v.x;
            q += v.y;
        }
        if (dbeta) dbeta[i] = (float)a;
        if (dgamma) dgamma[i] = (float)q;
        return;
    }
    const int b = id / per, chunk = id - b * per;
    if (chunk >= n.chunks) {
        pdl_wait();
        zero_gap<kDx>(n, dx, b, chunk - n.chunks);
        return;
    }
    const ChunkAt at = chunk_at(n, chunk);
    const int slot = threadIdx.x / n.tpr, c = (threadIdx.x - slot * n.tpr) * 8;
    if (slot >= n.slots) return;
    const int64_t base = ((int64_t)b * n.Nv + at.row) * n.C + c;
    const Channels k = load_constants(n, b, at.l, c, mean, rstd, gamma, beta);
    Vec8 c1, c2;
#pragma unroll
    for (int i0 = 0; i0 < kRowsPerThread; i0 += kBackRows) {
        Raw8<kX> rx[kBackRows];
        Raw8<kDy> rd[kBackRows];
#pragma unroll
        for (int i = 0; i < kBackRows; ++i) {
            const int row = slot + (i0 + i) * n.slots;
            if (row < at.rows) {
                rx[i] = load8<kX>(x, base + (int64_t)row * n.C);
                rd[i] = load8<kDy>(dy, base + (int64_t)row * n.C);
            }
        }
        if (i0 == 0) {
            pdl_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 v = coef[((int64_t)b * n.L + at.l) * n.G + (c + j) / n.cg];
                c1.v[j] = v.x;
                c2.v[j] = v.y;
            }
        }
#pragma unroll
        for (int i = 0; i < kBackRows; ++i) {
            const int row = slot + (i0 + i) * n.slots;
            if (row < at.rows) {
                const Vec8 v = widen(rx[i]), d = widen(rd[i]);
                Vec8 o;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hat = (v.v[j] - k.mean.v[j]) * k.rstd.v[j];
                    const float dz = grad_z<kAct>(d.v[j], v.v[j], k.mean.v[j], k.rstd.v[j], hat,
                                                  k.gamma.v[j], k.beta.v[j]);
                    // t rounded before the mean is taken off: exactly 0 where
                    // the group has one value
                    const float t = __fmul_rn(k.gamma.v[j], dz);
                    o.v[j] = k.rstd.v[j] * fmaf(-hat, c2.v[j], __fsub_rn(t, c1.v[j]));
                }
                store8<kDx>(dx, base + (int64_t)row * n.C, o);
            }
        }
    }
}

// ------------------------------------------------------------------- host

int norm_chunk_rows(int C)
{
    return std::max(1, kNormThreads / (C / 8)) * kRowsPerThread;
}

bool norm_sizes_ok(const msda_norm_dims_t& d)
{
    return d.B >= 0 && d.Nv >= 1 && d.C >= 8 && d.C % 8 == 0 && d.C <= kMaxC && d.L >= 1 &&
           d.L <= MSDA_MAX_LEVELS && d.G >= 1 && d.C % d.G == 0;
}

// Chunks per item, at most: whole ones over all rows and one cut per level.
int64_t norm_max_chunks(const msda_norm_dims_t& d)
{
    return d.Nv / norm_chunk_rows(d.C) + d.L;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

msda_status_t norm_shape(const msda_norm_dims_t& d, const int64_t* shapes, const int64_t* starts,
                         NormShape& n)
{
    if (d.B < 0 || d.Nv < 1)
        return api_failf(MSDA_ERR_INVALID_ARG, "B (%d) must be >= 0 and Nv (%d) >= 1", d.B, d.Nv);
    if (d.C < 8 || d.C % 8 || d.C > kMaxC)
        return api_failf(MSDA_ERR_UNSUPPORTED, "C = %d is not a multiple of 8 up to %d", d.C,
                         kMaxC);
    if (d.L < 1 || d.L > MSDA_MAX_LEVELS)
        return api_failf(MSDA_ERR_UNSUPPORTED, "L = %d outside 1..%d", d.L, MSDA_MAX_LEVELS);
    if (d.G < 1 || d.C % d.G)
        return api_failf(MSDA_ERR_INVALID_ARG, "G = %d does not divide C = %d", d.G, d.C);
    if (shapes == nullptr || starts == nullptr)
        return api_fail(MSDA_ERR_INVALID_ARG,
                        "spatial_shapes and level_start_index must be host arrays");
    n = NormShape{};
    n.B = d.B;
    n.Nv = d.Nv;
    n.C = d.C;
    n.L = d.L;
    n.G = d.G;
    n.cg = d.C / d.G;
    n.tpr = d.C / 8;
    n.slots = std::max(1, kNormThreads / n.tpr);
    n.chunk_rows = norm_chunk_rows(d.C);
    int order[MSDA_MAX_LEVELS];
    for (int l = 0; l < d.L; ++l) {
        const int64_t h = shapes[2 * l], w = shapes[2 * l + 1], st = starts[l];
        if (h < 1 || w < 1 || h > (1 << 24) || w > (1 << 24))
            return api_failf(MSDA_ERR_INVALID_ARG, "level %d has shape %lld x %lld", l,
                             (long long)h, (long long)w);
        if (st < 0 || h * w > d.Nv || st > d.Nv - h * w)
            return api_failf(MSDA_ERR_INVALID_ARG,
                             "level %d (start %lld, %lld x %lld) does not fit in Nv = %d", l,
                             (long long)st, (long long)h, (long long)w, d.Nv);
        n.start[l] = (int)st;
        n.rows[l] = (int)(h * w);
        n.chunk0[l] = n.chunks;
        n.chunks += (n.rows[l] + n.chunk_rows - 1) / n.chunk_rows;
        int k = l;  // the levels by their first row
        for (; k > 0 && n.start[order[k - 1]] > n.start[l]; --k) order[k] = order[k - 1];
        order[k] = l;
    }
    n.chunk0[d.L] = n.chunks;
    int at = 0;
    for (int k = 0; k <= d.L; ++k) {
        const int start = k < d.L ? n.start[order[k]] : d.Nv;
        if (start < at)
            return api_failf(MSDA_ERR_INVALID_ARG, "level %d shares rows with another", order[k]);
        if (start > at) {
            n.gap_start[n.gaps] = at;
            n.gap_rows[n.gaps++] = start - at;
            n.gap_chunks += (start - at + n.chunk_rows - 1) / n.chunk_rows;
        }
        if (k < d.L) at = start + n.rows[order[k]];
    }
    // chunks are counted in 32 bits over all items (elements in 64)
    if ((int64_t)d.B * (n.chunks + n.gap_chunks) > INT32_MAX - (1 << 20) ||
        (int64_t)d.B * d.L > INT32_MAX)
        return api_fail(MSDA_ERR_UNSUPPORTED, "too many rows");
    return MSDA_OK;
}

msda_status_t norm_ptr(const void* p, size_t align, const char* name, bool required)
{
    if (p == nullptr)
        return required ? api_failf(MSDA_ERR_INVALID_ARG, "%s is null", name) : MSDA_OK;
    if ((uintptr_t)p % align)
        return api_failf(MSDA_ERR_INVALID_ARG, "%s must be %zu-byte aligned", name, align);
    return MSDA_OK;
}

msda_status_t norm_workspace(const void* ws, size_t have, size_t need)
{
    if (ws != nullptr && have >= need && (uintptr_t)ws % 256 == 0) return MSDA_OK;
    return api_failf(MSDA_ERR_WORKSPACE,
                     "workspace of %zu bytes: %zu bytes on a 256-byte boundary are needed",
                     ws == nullptr ? (size_t)0 : have, need);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

size_t tensor_bytes(const msda_norm_dims_t& d, msda_dtype_t t)
{
    return (size_t)d.B * d.Nv * d.C * (t == MSDA_BF16 ? 2 : 4);
}

#define NORM_TRY(expr)                            \
    do {                                          \
        const msda_status_t st_ = (expr);         \
        if (st_ != MSDA_OK) return st_;           \
    } while (0)

msda_status_t norm_dtype(msda_dtype_t t, const char* name)
{
    if (t != MSDA_F32 && t != MSDA_BF16)
        return api_failf(MSDA_ERR_INVALID_ARG, "unknown %s %d", name, (int)t);
    return MSDA_OK;
}

template <bool kX, bool kY, int kAct>
cudaError_t apply_forward(const void* x, const NormShape& n, const float4* stats,
                          const float* gamma, const float* beta, void* y, cudaStream_t s)
{
    return launch_pdl(norm_apply_kernel<kX, kY, kAct>, dim3(n.B * (n.chunks + n.gap_chunks)),
                      dim3(kNormThreads), 0, s, x, n, stats, gamma, beta, y);
}

template <bool kX>
cudaError_t run_forward(const void* x, const NormShape& n, const float* gamma, const float* beta,
                        float eps, msda_activation_t act, bool y_bf16, void* y, float* mean,
                        float* rstd, double2* part, float4* stats, cudaStream_t s)
{
    norm_stats_kernel<kX><<<n.B * n.chunks, kNormThreads, 0, s>>>(x, n, part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_pdl(norm_merge_kernel, dim3(n.B * n.L, (n.G + 31) / 32), dim3(kMergeThreads), 0, s,
                   part, n, eps, stats, mean, rstd);
    if (e != cudaSuccess) return e;
    auto go = y_bf16 ? apply_forward<kX, true, MSDA_ACT_NONE> : apply_forward<kX, false, MSDA_ACT_NONE>;
    if (act == MSDA_ACT_RELU)
        go = y_bf16 ? apply_forward<kX, true, MSDA_ACT_RELU> : apply_forward<kX, false, MSDA_ACT_RELU>;
    if (act == MSDA_ACT_SILU)
        go = y_bf16 ? apply_forward<kX, true, MSDA_ACT_SILU> : apply_forward<kX, false, MSDA_ACT_SILU>;
    return go(x, n, stats, gamma, beta, y, s);
}

struct GradArgs {
    const void *x, *dy;
    NormShape n;
    const float *mean, *rstd, *gamma, *beta;
    float* part;
    double2* chan;
    float2* coef;
    void* dx;
    float *dgamma, *dbeta;
};

template <bool kX, bool kDy, bool kDx, int kAct>
cudaError_t run_backward(const GradArgs& a, cudaStream_t s)
{
    const NormShape& n = a.n;
    norm_grad_sums_kernel<kX, kDy, kAct><<<n.B * n.chunks, kNormThreads, 0, s>>>(
        a.x, a.dy, n, a.mean, a.rstd, a.gamma, a.beta, a.part);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int per_block = n.cg > 32 ? 1 : 32 / n.cg;
    e = launch_pdl(norm_grad_merge_kernel, dim3(n.B * n.L, (n.G + per_block - 1) / per_block),
                   dim3(kMergeThreads), 0, s, a.part, n, per_block, a.gamma, a.chan, a.coef);
    if (e != cudaSuccess) return e;
    const int extra = (n.L * n.C + kNormThreads - 1) / kNormThreads;
    return launch_pdl(norm_grad_apply_kernel<kX, kDy, kDx, kAct>,
                      dim3(n.B * (n.chunks + n.gap_chunks) + extra), dim3(kNormThreads), 0, s, a.x,
                      a.dy, n, a.mean, a.rstd, a.gamma, a.beta, a.chan, a.coef, a.dx, a.dgamma,
                      a.dbeta);
}

template <bool kX, bool kDy, bool kDx>
cudaError_t run_backward(const GradArgs& a, msda_activation_t act, cudaStream_t s)
{
    if (act == MSDA_ACT_RELU) return run_backward<kX, kDy, kDx, MSDA_ACT_RELU>(a, s);
    if (act == MSDA_ACT_SILU) return run_backward<kX, kDy, kDx, MSDA_ACT_SILU>(a, s);
    return run_backward<kX, kDy, kDx, MSDA_ACT_NONE>(a, s);
}

}  // namespace
}  // namespace msda

using namespace msda;

extern "C" size_t msda_group_norm_workspace_size(msda_norm_dims_t d)
{
    if (!norm_sizes_ok(d)) return 0;
    return up256(sizeof(double2) * d.B * norm_max_chunks(d) * d.G) +
           up256(sizeof(float4) * d.B * d.L * (size_t)d.G);
}

extern "C" size_t msda_group_norm_backward_workspace_size(msda_norm_dims_t d)
{
    if (!norm_sizes_ok(d)) return 0;
    return up256(sizeof(float) * 2 * d.B * norm_max_chunks(d) * d.C) +
           up256(sizeof(double2) * d.B * d.L * (size_t)d.C) +
           up256(sizeof(float2) * d.B * d.L * (size_t)d.G);
}

extern "C" msda_status_t msda_group_norm(const void* x, msda_dtype_t x_dtype,
                                         const int64_t* spatial_shapes,
                                         const int64_t* level_start_index, msda_norm_dims_t d,
                                         const float* gamma, const float* beta, float eps,
                                         msda_activation_t act, msda_dtype_t y_dtype, void* y,
                                         float* mean, float* rstd, void* workspace,
                                         size_t workspace_bytes, msda_stream_t stream)
{
    NormShape n;
    NORM_TRY(norm_shape(d, spatial_shapes, level_start_index, n));
    NORM_TRY(norm_dtype(x_dtype, "x_dtype"));
    NORM_TRY(norm_dtype(y_dtype, "y_dtype"));
    if (act < MSDA_ACT_NONE || act > MSDA_ACT_SILU)
        return api_failf(MSDA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    if (!(eps > 0.0f) || std::isinf(eps))
        return api_failf(MSDA_ERR_INVALID_ARG, "eps = %g must be finite and > 0", (double)eps);
    if (d.B == 0) return api_ok();
    NORM_TRY(norm_ptr(x, 16, "x", true));
    NORM_TRY(norm_ptr(y, 16, "y", true));
    NORM_TRY(norm_ptr(gamma, 16, "gamma", false));
    NORM_TRY(norm_ptr(beta, 16, "beta", false));
    NORM_TRY(norm_ptr(mean, 4, "mean", false));
    NORM_TRY(norm_ptr(rstd, 4, "rstd", false));
    if (overlap(x, tensor_bytes(d, x_dtype), y, tensor_bytes(d, y_dtype)))
        return api_fail(MSDA_ERR_INVALID_ARG, "y overlaps x");
    NORM_TRY(norm_workspace(workspace, workspace_bytes, msda_group_norm_workspace_size(d)));
    double2* part = static_cast<double2*>(workspace);
    float4* stats = reinterpret_cast<float4*>(
        static_cast<char*>(workspace) + up256(sizeof(double2) * d.B * norm_max_chunks(d) * d.G));
    const auto run = x_dtype == MSDA_BF16 ? run_forward<true> : run_forward<false>;
    return api_cuda(run(x, n, gamma, beta, eps, act, y_dtype == MSDA_BF16, y, mean, rstd, part,
                        stats, (cudaStream_t)stream),
                    "msda_group_norm");
}

extern "C" msda_status_t msda_group_norm_backward(
    const void* x, msda_dtype_t x_dtype, const int64_t* spatial_shapes,
    const int64_t* level_start_index, msda_norm_dims_t d, const float* gamma, const float* beta,
    const float* mean, const float* rstd, msda_activation_t act, const void* grad_y,
    msda_dtype_t gy_dtype, msda_dtype_t gx_dtype, void* grad_x, float* grad_gamma,
    float* grad_beta, void* workspace, size_t workspace_bytes, msda_stream_t stream)
{
    GradArgs a;
    NORM_TRY(norm_shape(d, spatial_shapes, level_start_index, a.n));
    NORM_TRY(norm_dtype(x_dtype, "x_dtype"));
    NORM_TRY(norm_dtype(gy_dtype, "gy_dtype"));
    NORM_TRY(norm_dtype(gx_dtype, "gx_dtype"));
    if (act < MSDA_ACT_NONE || act > MSDA_ACT_SILU)
        return api_failf(MSDA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    const cudaStream_t s = (cudaStream_t)stream;
    NORM_TRY(norm_ptr(grad_gamma, 4, "grad_gamma", false));
    NORM_TRY(norm_ptr(grad_beta, 4, "grad_beta", false));
    if (d.B == 0) {  // no items: the parameters' gradients are sums of nothing
        for (float* p : {grad_gamma, grad_beta}) {
            const cudaError_t e =
                p ? cudaMemsetAsync(p, 0, sizeof(float) * d.L * d.C, s) : cudaSuccess;
            if (e != cudaSuccess) return api_cuda(e, "msda_group_norm_backward");
        }
        return api_ok();
    }
    NORM_TRY(norm_ptr(x, 16, "x", true));
    NORM_TRY(norm_ptr(grad_y, 16, "grad_y", true));
    NORM_TRY(norm_ptr(grad_x, 16, "grad_x", true));
    NORM_TRY(norm_ptr(gamma, 16, "gamma", false));
    NORM_TRY(norm_ptr(beta, 16, "beta", false));
    NORM_TRY(norm_ptr(mean, 4, "mean", true));
    NORM_TRY(norm_ptr(rstd, 4, "rstd", true));
    if (overlap(x, tensor_bytes(d, x_dtype), grad_x, tensor_bytes(d, gx_dtype)) ||
        overlap(grad_y, tensor_bytes(d, gy_dtype), grad_x, tensor_bytes(d, gx_dtype)))
        return api_fail(MSDA_ERR_INVALID_ARG, "grad_x overlaps x or grad_y");
    NORM_TRY(norm_workspace(workspace, workspace_bytes,
                            msda_group_norm_backward_workspace_size(d)));
    char* w = static_cast<char*>(workspace);
    a.x = x;
    a.dy = grad_y;
    a.mean = mean;
    a.rstd = rstd;
    a.gamma = gamma;
    a.beta = beta;
    a.part = reinterpret_cast<float*>(w);
    w += up256(sizeof(float) * 2 * d.B * norm_max_chunks(d) * d.C);
    a.chan = reinterpret_cast<double2*>(w);
    w += up256(sizeof(double2) * d.B * d.L * (size_t)d.C);
    a.coef = reinterpret_cast<float2*>(w);
    a.dx = grad_x;
    a.dgamma = grad_gamma;
    a.dbeta = grad_beta;
    using Run = cudaError_t (*)(const GradArgs&, msda_activation_t, cudaStream_t);
    static constexpr Run runs[8] = {
        run_backward<false, false, false>, run_backward<false, false, true>,
        run_backward<false, true, false>,  run_backward<false, true, true>,
        run_backward<true, false, false>,  run_backward<true, false, true>,
        run_backward<true, true, false>,   run_backward<true, true, true>};
    const int k = 4 * (x_dtype == MSDA_BF16) + 2 * (gy_dtype == MSDA_BF16) +
                  (gx_dtype == MSDA_BF16);
    return api_cuda(runs[k](a, act, s), "msda_group_norm_backward");
}
