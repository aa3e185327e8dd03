// msda_group_norm and its backward: group norm with an activation over the
// levels of channels-last rows [B, Nv, C].
//
// Forward, per (item, level, group) with N = rows * C/G values:
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps),
//   y = act(gamma (x - mu) r + beta)
// Backward, with xh = (x - mu) r, dz = dy act'(z), t = gamma dz:
//   dgamma = sum dz xh, dbeta = sum dz, dx = r (t - mean(t) - xh mean(t xh))
//
// Both are two passes over the rows, one launch each: every value needs sums
// over its whole level.  The levels' rows of all items stand in one line, of
// which each CTA takes an even run, whatever the levels' sizes; a run is cut
// into spans at the levels' ends.  A thread holds two quads of channels of every
// slots-th row of a span, so that a channel's constants and sums stay in
// registers and only a span's end costs a reduction.  The quads are neighbours
// where all tensors are bf16, else half a row apart: either way neighbouring
// lanes' 16 bytes are neighbours (with the eight channels in one piece the two
// loads of fp32 each took half of every sector: 66 us instead of 33 us for the
// six cameras' first pass).  The first pass leaves one partial
// result per span and group; the second adds those of its span's level (each
// CTA for itself, in the same order: no atomic, no flag and no third launch)
// and then walks its run backwards: what the first pass read last is still in
// L2 (126 MB).  It is a programmatic dependent of the first.
//
// A few rows take one launch: a cluster of up to eight CTAs does both passes,
// with its barrier in between.
//
// Bound by memory: the rows are read twice, the second time from L2 as far as
// that reaches, and written once.  Six cameras (185 k rows of 256, fp32 to bf16):
// 85 us, 473 MB at 5.5 TB/s with next to nothing left in L2 for the second pass;
// taking the cameras in twos, so that a pass fits, costs as much in the ends of
// its launches as it saves.  The gradient of the same in fp32: 165 us, 946 MB at
// 5.7 TB/s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "msda.h"
#include "msda_launch.h"

namespace msda {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormWarps = kNormThreads / 32;
constexpr int kMaxC = MSDA_NORM_MAX_CHANNELS;
constexpr int kSms = 148;
constexpr int kMaxRuns = 2 * kSms;  // two CTAs per SM
constexpr int kCluster = 8;         // CTAs of the one-launch form (375 rows: 25.3 us a call, 28.4 us with two launches),
constexpr int kSmallRows = 8;       // which takes up to 8 rows per thread

struct NormShape {
    int B, Nv, C, L, G, cg;  // cg = C / G
    int tpr, slots;          // threads per row, rows side by side
    int runs;                // CTAs that share the rows
    bool small;              // and form one cluster
    int used;                // rows of an item in its levels, cum[L]
    int start[kMaxLevels], cum[kMaxLevels + 1];
    int gaps;                // runs of rows in no level
    int gap_start[kMaxLevels + 1], gap_rows[kMaxLevels + 1];
};

// Run i holds the rows [total i / runs, total (i + 1) / runs) of the line of
// all levels' rows.
__device__ __forceinline__ int64_t run_begin(const NormShape& n, int i)
{
    return (int64_t)n.B * n.used * i / n.runs;
}

__device__ __forceinline__ int run_of(const NormShape& n, int64_t row)
{
    return (int)(((row + 1) * n.runs - 1) / ((int64_t)n.B * n.used));
}

// A span: rows [at, at + rows) of the line, all of one (item, level).
struct Span {
    int b, l, rows;
    int64_t row;  // its first row among the tensor's B * Nv
};

__device__ __forceinline__ int level_of(const NormShape& n, int off)
{
    int l = 0;
    while (l + 1 < n.L && n.cum[l + 1] <= off) ++l;
    return l;
}

// The span that starts at `at` of a run that ends at `end`.
__device__ __forceinline__ Span span_from(const NormShape& n, int64_t at, int64_t end)
{
    const int b = (int)(at / n.used), off = (int)(at - (int64_t)b * n.used);
    const int l = level_of(n, off);
    return {b, l, (int)min((int64_t)(n.cum[l + 1] - off), end - at),
            (int64_t)b * n.Nv + n.start[l] + (off - n.cum[l])};
}

// The span that ends before `end` of a run that starts at `begin`.
__device__ __forceinline__ Span span_before(const NormShape& n, int64_t begin, int64_t end)
{
    const int b = (int)((end - 1) / n.used);
    const int l = level_of(n, (int)(end - 1 - (int64_t)b * n.used));
    const int64_t first = max(begin, (int64_t)b * n.used + n.cum[l]);
    return span_from(n, first, end);
}

// Where the partial results of run i's span of (item, level) bl lie: along the
// line i or bl grows from each span to the next, so i + bl is their own.
__device__ __forceinline__ int64_t span_slot(int run, int64_t bl) { return run + bl; }

struct Vec8 {
    float v[8];
};

// A thread's channels: [a, a + 4) and [b, b + 4).
struct Quads {
    int a, b;
};

template <bool kSplit>
__device__ __forceinline__ Quads quads_of(int C, int i)
{
    if constexpr (kSplit) return {4 * i, C / 2 + 4 * i};
    return {8 * i, 8 * i + 4};
}

__device__ __forceinline__ int channel(const Quads& q, int j) { return j < 4 ? q.a + j : q.b + j - 4; }

__device__ __forceinline__ void widen_pair(float* o, uint32_t w)
{
    o[0] = __uint_as_float(w << 16);
    o[1] = __uint_as_float(w & 0xffff0000u);
}

__device__ __forceinline__ Vec8 vec8(const float4& a, const float4& b)
{
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

template <bool kBf16>
__device__ __forceinline__ Vec8 load8(const void* p, int64_t row, const Quads& q)
{
    if constexpr (kBf16) {
        const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(p) + row;
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(h + q.a));
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(h + q.b));
        Vec8 o;
        widen_pair(o.v, a.x);
        widen_pair(o.v + 2, a.y);
        widen_pair(o.v + 4, b.x);
        widen_pair(o.v + 6, b.y);
        return o;
    } else {
        const float* f = static_cast<const float*>(p) + row;
        return vec8(__ldg(reinterpret_cast<const float4*>(f + q.a)),
                    __ldg(reinterpret_cast<const float4*>(f + q.b)));
    }
}

template <bool kBf16, bool kSplit>
__device__ __forceinline__ void store8(void* p, int64_t row, const Quads& q, const Vec8& o)
{
    if constexpr (kBf16) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o.v[2 * j], o.v[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        __nv_bfloat16* h = static_cast<__nv_bfloat16*>(p) + row;
        if constexpr (kSplit) {
            __stcs(reinterpret_cast<uint2*>(h + q.a), make_uint2(w[0], w[1]));
            __stcs(reinterpret_cast<uint2*>(h + q.b), make_uint2(w[2], w[3]));
        } else {
            __stcs(reinterpret_cast<uint4*>(h + q.a), make_uint4(w[0], w[1], w[2], w[3]));
        }
    } else {
        float* f = static_cast<float*>(p) + row;
        __stcs(reinterpret_cast<float4*>(f + q.a), make_float4(o.v[0], o.v[1], o.v[2], o.v[3]));
        __stcs(reinterpret_cast<float4*>(f + q.b), make_float4(o.v[4], o.v[5], o.v[6], o.v[7]));
    }
}

// A thread's rows on their way from memory: a ring in shared memory of kStages
// steps of 64 bytes per thread (kStepRows rows of one tensor, or of x and dy),
// written by asynchronous copies and read by the thread that asked for them
// (no barrier).  With registers as the landing place a warp either waits for
// its loads or computes: the memory then saw half of the requests it needs
// (4.4 TB/s, against 160 KB in flight per SM here).
constexpr int kStages = 5;
constexpr int kRingBytes = kStages * 64 * kNormThreads;

template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src)
{
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ void copy_wait()  // for the oldest of kStages steps
{
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
}

// A row's eight values in the ring: kPieces places of 16 bytes.
template <bool kBf16, bool kSplit>
struct RowCopy {
    static constexpr int kPieces = kBf16 ? 1 : 2;
    static __device__ __forceinline__ void fetch(uint4* to, const void* p, int64_t row,
                                                 const Quads& q)
    {
        if constexpr (!kBf16) {
            const float* f = static_cast<const float*>(p) + row;
            copy_async<16>(to, f + q.a);
            copy_async<16>(to + kNormThreads, f + q.b);
        } else if constexpr (kSplit) {
            const __nv_bfloat16* h = static_cast<const __nv_bfloat16*>(p) + row;
            copy_async<8>(to, h + q.a);
            copy_async<8>(reinterpret_cast<uint2*>(to) + 1, h + q.b);
        } else {
            copy_async<16>(to, static_cast<const __nv_bfloat16*>(p) + row + q.a);
        }
    }
    static __device__ __forceinline__ Vec8 take(const uint4* from)
    {
        if constexpr (kBf16) {
            const uint4 r = *from;
            Vec8 o;
            widen_pair(o.v, r.x);
            widen_pair(o.v + 2, r.y);
            widen_pair(o.v + 4, r.z);
            widen_pair(o.v + 6, r.w);
            return o;
        } else {
            return vec8(*reinterpret_cast<const float4*>(from),
                        *reinterpret_cast<const float4*>(from + kNormThreads));
        }
    }
};

// Rows of a thread whose sums are formed in fp32 before they join a double.
constexpr int kBlockRows = 8;

// Walks a thread's `count` rows, `step` values apart from the one that starts
// at `first` on, through the ring: start() asks for the first steps, run()
// calls use(row, x) or use(row, x, dy) for every row.  run_blocks() takes the
// rows in blocks of kBlockRows: use(x, leads) or use(x, dy, leads) for each, `leads`
// for a block's first, and join(rows) behind a block.
template <bool kX, bool kSplit>
struct Walk1 {
    using Copy = RowCopy<kX, kSplit>;
    static constexpr int kRows = 4 / Copy::kPieces;
    uint4* ring;
    const void* x;
    Quads q;
    int64_t first, step;
    int count;

    __device__ __forceinline__ uint4* at(int k, int i) const
    {
        return ring + ((k % kStages) * 4 + i * Copy::kPieces) * kNormThreads + threadIdx.x;
    }
    __device__ __forceinline__ void ask(int k) const
    {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (k * kRows + i < count)
                Copy::fetch(at(k, i), x, first + (int64_t)(k * kRows + i) * step, q);
        copy_commit();
    }
    __device__ __forceinline__ void start() const
    {
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) ask(k);
    }
    template <typename F>
    __device__ __forceinline__ void run(F use) const
    {
        for (int k = 0; k * kRows < count; ++k) {
            ask(k + kStages - 1);
            copy_wait();
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (k * kRows + i < count)
                    use(first + (int64_t)(k * kRows + i) * step, Copy::take(at(k, i)));
        }
    }
    template <typename F, typename J>
    __device__ __forceinline__ void run_blocks(F use, J join) const
    {
        for (int row = 0; row < count; row += kBlockRows) {
#pragma unroll
            for (int r = 0; r < kBlockRows; r += kRows) {
                if (row + r >= count) break;
                const int k = (row + r) / kRows;
                ask(k + kStages - 1);
                copy_wait();
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (row + r + i < count) use(Copy::take(at(k, i)), r + i == 0);
            }
            join(min(kBlockRows, count - row));
        }
    }
};

template <bool kX, bool kDy, bool kSplit>
struct Walk2 {
    using CopyX = RowCopy<kX, kSplit>;
    using CopyD = RowCopy<kDy, kSplit>;
    static constexpr int kPieces = CopyX::kPieces + CopyD::kPieces, kRows = 4 / kPieces;
    uint4* ring;
    const void *x, *dy;
    Quads q;
    int64_t first, step;
    int count;

    __device__ __forceinline__ uint4* at(int k, int i) const
    {
        return ring + ((k % kStages) * 4 + i * kPieces) * kNormThreads + threadIdx.x;
    }
    __device__ __forceinline__ void ask(int k) const
    {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (k * kRows + i < count) {
                const int64_t row = first + (int64_t)(k * kRows + i) * step;
                CopyX::fetch(at(k, i), x, row, q);
                CopyD::fetch(at(k, i) + CopyX::kPieces * kNormThreads, dy, row, q);
            }
        }
        copy_commit();
    }
    __device__ __forceinline__ void start() const
    {
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) ask(k);
    }
    template <typename F>
    __device__ __forceinline__ void run(F use) const
    {
        for (int k = 0; k * kRows < count; ++k) {
            ask(k + kStages - 1);
            copy_wait();
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                if (k * kRows + i < count)
                    use(first + (int64_t)(k * kRows + i) * step, CopyX::take(at(k, i)),
                        CopyD::take(at(k, i) + CopyX::kPieces * kNormThreads));
        }
    }
    template <typename F, typename J>
    __device__ __forceinline__ void run_blocks(F use, J join) const
    {
        for (int row = 0; row < count; row += kBlockRows) {
#pragma unroll
            for (int r = 0; r < kBlockRows; r += kRows) {
                if (row + r >= count) break;
                const int k = (row + r) / kRows;
                ask(k + kStages - 1);
                copy_wait();
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (row + r + i < count)
                        use(CopyX::take(at(k, i)),
                            CopyD::take(at(k, i) + CopyX::kPieces * kNormThreads), r + i == 0);
            }
            join(min(kBlockRows, count - row));
        }
    }
};

extern __shared__ uint4 ring_memory[];

__device__ __forceinline__ Vec8 load_channels(const float* p, int64_t row, const Quads& q,
                                              float otherwise)
{
    if (p != nullptr) return load8<false>(p, row, q);
    Vec8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = otherwise;
    return o;
}

// The sums of two quantities per channel and slot, in double: they lie where the
// ring was, whose rows have all been taken behind a barrier.
constexpr int kSumsPlane = kNormThreads * 8;
static_assert(2 * kSumsPlane * sizeof(double) <= kRingBytes, "");

__device__ __forceinline__ double* slot_sums() { return reinterpret_cast<double*>(ring_memory); }

struct Sums8 {
    double v[8];
};

__device__ __forceinline__ void put_slot(double* s, int C, int slot, const Quads& c,
                                         const Sums8& a, const Sums8& b)
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const int at = slot * C + channel(c, j);
        *reinterpret_cast<double2*>(s + at) = make_double2(a.v[j], a.v[j + 1]);
        *reinterpret_cast<double2*>(s + kSumsPlane + at) = make_double2(b.v[j], b.v[j + 1]);
    }
}

// Adds the slots' sums: on return s[c] and s[kSumsPlane + c] hold channel c's (for
// the thread that owns it, threads c mod kNormThreads; a barrier before others
// read them).
__device__ __forceinline__ void add_slots(double* s, int C, int slots)
{
    __syncthreads();
    double* s2 = s + kSumsPlane;
    for (int c = threadIdx.x; c < C; c += kNormThreads) {
        double a = s[c], b = s2[c];
        for (int k = 1; k < slots; ++k) {
            a += s[k * C + c];
            b += s2[k * C + c];
        }
        s[c] = a;
        s2[c] = b;
    }
}

// The 32 (or fewer) lanes that add up a group of cg channels: a power of two,
// so that several small groups share a warp.
struct GroupLanes {
    int seg, per_warp, sub, in;
};

__device__ __forceinline__ GroupLanes group_lanes(int cg)
{
    int seg = 1;
    while (seg < 32 && seg < cg) seg <<= 1;
    const int lane = threadIdx.x & 31;
    return {seg, 32 / seg, lane / seg, lane % seg};
}

__device__ __forceinline__ double add_lanes(double v, int seg)
{
    for (int o = seg >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------- forward

// A span's sums of x - m and of its square per group, m the mean of the group's
// channels in the level's first row: the same for all spans of the level, so
// that their sums add up.  m need not be near the group's mean: with N rows the
// row that it comes from makes 1 / N of the variance at least, so what cancels
// is N of the 2^53 of a double at most.  fp32 does not have such room, so it only holds
// sums of eight rows of a channel, relative to the first of the eight, whose
// distance from the mean is part of the same sum: they are off by less than 380
// roundings of the group's sum of squares whatever the data are (2^-16.4 of r).  They
// are moved to the channel's value in the level's first row, and then to m, in
// double.  (With all rows of a run summed in fp32 and relative to the level's first
// row, a blank first pixel under features 300 spreads from zero cost r 1e-3, and the
// six cameras took 2.7 us less: 1.5 us for the moves, the rest for sums of 64 bits in
// shared memory.  Blocks of 16 rows: 0.6 us less, and twice the bound.)
template <bool kX>
__device__ __forceinline__ void norm_stats(float* first, const void* __restrict__ x,
                                           const NormShape& n, double2* part, double* middle)
{
    constexpr bool kSplit = !kX;
    double* s = slot_sums();
    const int slot = threadIdx.x / n.tpr;
    const Quads c = quads_of<kSplit>(n.C, threadIdx.x - slot * n.tpr);
    const GroupLanes gl = group_lanes(n.cg);
    const int64_t end = run_begin(n, blockIdx.x + 1);
    for (int64_t at = run_begin(n, blockIdx.x); at < end;) {
        const Span sp = span_from(n, at, end);
        Vec8 ref{};
        Sums8 sum{}, square{};
        if (slot < n.slots) {
            const Walk1<kX, kSplit> walk{ring_memory,
                                         x,
                                         c,
                                         (sp.row + slot) * n.C,
                                         (int64_t)n.slots * n.C,
                                         (sp.rows - slot + n.slots - 1) / n.slots};
            walk.start();
            ref = load8<kX>(x, ((int64_t)sp.b * n.Nv + n.start[sp.l]) * n.C, c);
            Vec8 lead{}, a{}, q{};
            walk.run_blocks(
                [&](const Vec8& v, bool leads) {
                    if (leads) {
                        lead = v;
                        a = q = Vec8{};
                        return;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float d = v.v[j] - lead.v[j];
                        a.v[j] += d;
                        q.v[j] = fmaf(d, d, q.v[j]);
                    }
                },
                [&](int rows) {
                    const double k = (double)rows;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const double d = (double)lead.v[j] - (double)ref.v[j], s1 = (double)a.v[j];
                        const double moved = fma(k, d, s1);
                        sum.v[j] += moved;
                        square.v[j] += fma(d, s1 + moved, (double)q.v[j]);
                    }
                });
        }
        __syncthreads();  // the ring is free
        if (slot < n.slots) {
            put_slot(s, n.C, slot, c, sum, square);
            if (slot == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) first[channel(c, j)] = ref.v[j];
            }
        }
        add_slots(s, n.C, n.slots);
        __syncthreads();
        const double rows = (double)sp.rows;
        const int64_t bl = (int64_t)sp.b * n.L + sp.l, to = span_slot(blockIdx.x, bl) * n.G;
        const bool leads = at == (int64_t)sp.b * n.used + n.cum[sp.l];  // has the level's first row
        for (int g0 = (threadIdx.x >> 5) * gl.per_warp; g0 < n.G; g0 += kNormWarps * gl.per_warp) {
            const int g = g0 + gl.sub;
            const bool on = g < n.G;
            double m = 0.0, t1 = 0.0, t2 = 0.0;
            for (int k = gl.in; on && k < n.cg; k += gl.seg) m += (double)first[g * n.cg + k];
            m = add_lanes(m, gl.seg) / (double)n.cg;
            for (int k = gl.in; on && k < n.cg; k += gl.seg) {
                const int ch = g * n.cg + k;
                const double a = s[ch], d = (double)first[ch] - m;
                t1 += a + rows * d;
                t2 += s[kSumsPlane + ch] + d * (2.0 * a + rows * d);
            }
            t1 = add_lanes(t1, gl.seg);
            t2 = add_lanes(t2, gl.seg);
            if (on && gl.in == 0) {
                part[to + g] = make_double2(t1, t2);
                if (leads) middle[bl * n.G + g] = m;
            }
        }
        at += sp.rows;
        __syncthreads();  // the sums are read before the next span's are written
    }
}

// The partial results of all spans of an (item, level) for group g: one warp
// per share of the spans, 32 groups at a time.
struct Shares {
    double2 s[kNormWarps][32];
};

__device__ __forceinline__ double2 add_spans(Shares& sh, const double2* part, const NormShape& n,
                                             int b, int l, int g)
{
    const int64_t lo = (int64_t)b * n.used + n.cum[l], hi = (int64_t)b * n.used + n.cum[l + 1];
    const int r0 = run_of(n, lo), r1 = run_of(n, hi - 1);
    const int64_t bl = (int64_t)b * n.L + l;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double2 acc = make_double2(0.0, 0.0);
    if (g < n.G) {
#pragma unroll 8
        for (int r = r0 + warp; r <= r1; r += kNormWarps) {
            const double2 v = part[span_slot(r, bl) * n.G + g];
            acc.x += v.x;
            acc.y += v.y;
        }
    }
    sh.s[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
        for (int k = 1; k < kNormWarps; ++k) {
            acc.x += sh.s[k][lane].x;
            acc.y += sh.s[k][lane].y;
        }
    }
    return acc;  // for warp 0; a barrier before `sh` is used again
}

// An approximate reciprocal (one unit in the last place) instead of a division,
// which would bind the bf16 passes by instruction issue.
__device__ __forceinline__ float sigmoid(float z)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-z)));
    return r;
}

template <int kAct>
__device__ __forceinline__ float activate(float z)
{
    if constexpr (kAct == MSDA_ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (kAct == MSDA_ACT_SILU) return z * sigmoid(z);
    return z;
}

// Rows of no level: zeros, an even share per CTA.
template <bool kY>
__device__ void zero_gaps(const NormShape& n, void* y, int cta, int ctas)
{
    for (int k = 0; k < n.gaps; ++k) {
        const int64_t per = (int64_t)n.gap_rows[k] * n.tpr, all = per * n.B;
        for (int64_t i = (int64_t)cta * kNormThreads + threadIdx.x; i < all;
             i += (int64_t)ctas * kNormThreads) {
            const int64_t b = i / per;
            const int64_t at = (b * n.Nv + n.gap_start[k]) * n.C + (i - b * per) * 8;
            store8<kY, true>(y, at, {0, 4}, Vec8{});
        }
    }
}

struct ApplySmem {
    Shares shares;
    // the mean as two floats: what is subtracted is exact to 48 bits, whatever the mean
    float hi[kMaxC], lo[kMaxC], r[kMaxC];
};

struct NormOut {
    float eps;
    const float *gamma, *beta;
    void* y;
    float *mean, *rstd;
};

// The rows of a run, last ones first; `ready` is called before anything that the
// first pass wrote is read.
template <bool kX, bool kY, int kAct, typename Ready>
__device__ __forceinline__ void norm_apply(ApplySmem& sm, const void* __restrict__ x,
                                           const NormShape& n, const double2* part,
                                           const double* middle, const NormOut& out, int run,
                                           Ready ready)
{
    constexpr bool kSplit = !(kX && kY);
    Shares& shares = sm.shares;
    float *st_hi = sm.hi, *st_lo = sm.lo, *st_r = sm.r;
    const int slot = threadIdx.x / n.tpr;
    const Quads c = quads_of<kSplit>(n.C, threadIdx.x - slot * n.tpr);
    const int64_t begin = run_begin(n, run);
    bool waited = false;
    for (int64_t end = run_begin(n, run + 1); end > begin;) {
        const Span sp = span_before(n, begin, end);
        // the span's rows from its last on (what the pass before read last)
        const Walk1<kX, kSplit> walk{
            ring_memory,
            x,
            c,
            (sp.row + sp.rows - 1 - slot) * n.C,
            -(int64_t)n.slots * n.C,
            slot < n.slots ? (sp.rows - slot + n.slots - 1) / n.slots : 0};
        walk.start();
        if (!waited) ready();
        waited = true;
        const int64_t bl = (int64_t)sp.b * n.L + sp.l;
        for (int g0 = 0; g0 < n.G; g0 += 32) {
            const int g = g0 + (threadIdx.x & 31);
            const double2 acc = add_spans(shares, part, n, sp.b, sp.l, g);
            if (threadIdx.x < 32 && g < n.G) {
                const double N = (double)(n.cum[sp.l + 1] - n.cum[sp.l]) * n.cg;
                const double mean = middle[bl * n.G + g] + acc.x / N;
                double var = (acc.y - acc.x * acc.x / N) / N;
                if (var < 0.0) var = 0.0;  // rounding only; a NaN stays
                const float hi = (float)mean, r = (float)(1.0 / sqrt(var + (double)out.eps));
                st_hi[g] = hi;
                st_lo[g] = (float)(mean - (double)hi);
                st_r[g] = r;
                // the run with the level's first row writes the statistics
                if (begin <= (int64_t)sp.b * n.used + n.cum[sp.l]) {
                    if (out.mean) out.mean[bl * n.G + g] = hi;
                    if (out.rstd) out.rstd[bl * n.G + g] = r;
                }
            }
            __syncthreads();
        }
        if (slot < n.slots) {
            const Vec8 ga = load_channels(out.gamma, (int64_t)sp.l * n.C, c, 1.0f);
            const Vec8 be = load_channels(out.beta, (int64_t)sp.l * n.C, c, 0.0f);
            Vec8 hi, lo, a;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int g = channel(c, j) / n.cg;
                hi.v[j] = st_hi[g];
                lo.v[j] = st_lo[g];
                a.v[j] = st_r[g] * ga.v[j];
            }
            walk.run([&](int64_t at, Vec8 v) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v.v[j] = activate<kAct>(fmaf((v.v[j] - hi.v[j]) - lo.v[j], a.v[j], be.v[j]));
                store8<kY, kSplit>(out.y, at, c, v);
            });
        }
        end -= sp.rows;
        __syncthreads();  // the statistics are read before the next span's are written
    }
    zero_gaps<kY>(n, out.y, run, n.runs);
}

template <bool kX>
__global__ void __launch_bounds__(kNormThreads, 2) norm_stats_kernel(const void* __restrict__ x,
                                                                     const NormShape n,
                                                                     double2* __restrict__ part,
                                                                     double* __restrict__ middle)
{
    __shared__ float first[kMaxC];
    pdl_trigger();
    norm_stats<kX>(first, x, n, part, middle);
}

// (no __restrict__ on what the first pass writes while this one has begun)
template <bool kX, bool kY, int kAct>
__global__ void __launch_bounds__(kNormThreads, 2) norm_apply_kernel(
    const void* __restrict__ x, const NormShape n, const double2* part, const double* middle,
    const NormOut out)
{
    __shared__ ApplySmem sm;
    norm_apply<kX, kY, kAct>(sm, x, n, part, middle, out, n.runs - 1 - (int)blockIdx.x,
                             [] { pdl_wait(); });
}

// Both passes, for one cluster; a CTA's own rows come back from its L1 or L2.
template <bool kX, bool kY, int kAct>
__global__ void __launch_bounds__(kNormThreads, 2) norm_small_kernel(const void* __restrict__ x,
                                                                     const NormShape n,
                                                                     double2* part,
                                                                     double* middle,
                                                                     const NormOut out)
{
    __shared__ union {
        float first[kMaxC];
        ApplySmem apply;
    } sm;
    norm_stats<kX>(sm.first, x, n, part, middle);
    cluster_sync();
    norm_apply<kX, kY, kAct>(sm.apply, x, n, part, middle, out, blockIdx.x, [] {});
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

__device__ __forceinline__ Channels load_constants(const NormShape& n, int b, int l,
                                                   const Quads& c,
                                                   const float* mean, const float* rstd,
                                                   const float* gamma, const float* beta)
{
    Channels k;
    k.gamma = load_channels(gamma, (int64_t)l * n.C, c, 1.0f);
    k.beta = load_channels(beta, (int64_t)l * n.C, c, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = ((int64_t)b * n.L + l) * n.G + channel(c, j) / n.cg;
        k.mean.v[j] = __ldg(mean + i);
        k.rstd.v[j] = __ldg(rstd + i);
    }
    return k;
}

// A span's sums of dz and dz xh per channel (for the parameters' gradients) and,
// weighted with gamma, per group (for dx): fp32 over eight rows, double beyond.  A
// loss that is a mean has gradients of one sign and size, whose roundings in a long
// fp32 sum do not cancel (830 rows: 1e-5 of the sum).
struct GradIn {
    const void *x, *dy;
    const float *mean, *rstd, *gamma, *beta;
};

struct GradOut {
    void* dx;
    float *dgamma, *dbeta;
};

template <bool kX, bool kDy, int kAct>
__device__ __forceinline__ void norm_grad_sums(const GradIn& in, const NormShape& n,
                                               float* chan, double2* part)
{
    constexpr bool kSplit = !(kX && kDy);
    const void *__restrict__ x = in.x, *__restrict__ dy = in.dy;
    const float *mean = in.mean, *rstd = in.rstd, *gamma = in.gamma, *beta = in.beta;
    double* s = slot_sums();
    const int slot = threadIdx.x / n.tpr;
    const Quads c = quads_of<kSplit>(n.C, threadIdx.x - slot * n.tpr);
    const GroupLanes gl = group_lanes(n.cg);
    const int64_t end = run_begin(n, blockIdx.x + 1);
    for (int64_t at = run_begin(n, blockIdx.x); at < end;) {
        const Span sp = span_from(n, at, end);
        Sums8 sum{}, product{};
        if (slot < n.slots) {
            const Walk2<kX, kDy, kSplit> walk{ring_memory,
                                              x,
                                              dy,
                                              c,
                                              (sp.row + slot) * n.C,
                                              (int64_t)n.slots * n.C,
                                              (sp.rows - slot + n.slots - 1) / n.slots};
            walk.start();
            const Channels k = load_constants(n, sp.b, sp.l, c, mean, rstd, gamma, beta);
            Vec8 a{}, q{};
            walk.run_blocks(
                [&](const Vec8& v, const Vec8& d, bool) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float hat = (v.v[j] - k.mean.v[j]) * k.rstd.v[j];
                        const float dz = grad_z<kAct>(d.v[j], v.v[j], k.mean.v[j], k.rstd.v[j],
                                                      hat, k.gamma.v[j], k.beta.v[j]);
                        a.v[j] += dz;
                        q.v[j] = fmaf(dz, hat, q.v[j]);
                    }
                },
                [&](int) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        sum.v[j] += (double)a.v[j];
                        product.v[j] += (double)q.v[j];
                    }
                    a = q = Vec8{};
                });
        }
        __syncthreads();  // the ring is free
        if (slot < n.slots) put_slot(s, n.C, slot, c, sum, product);
        add_slots(s, n.C, n.slots);
        __syncthreads();
        const int64_t to = span_slot(blockIdx.x, (int64_t)sp.b * n.L + sp.l);
        for (int ch = threadIdx.x; ch < n.C; ch += kNormThreads) {
            chan[to * 2 * n.C + ch] = (float)s[ch];
            chan[to * 2 * n.C + n.C + ch] = (float)s[kSumsPlane + ch];
        }
        for (int g0 = (threadIdx.x >> 5) * gl.per_warp; g0 < n.G; g0 += kNormWarps * gl.per_warp) {
            const int g = g0 + gl.sub;
            const bool on = g < n.G;
            double t1 = 0.0, t2 = 0.0;
            for (int k = gl.in; on && k < n.cg; k += gl.seg) {
                const int ch = g * n.cg + k;
                const double w = gamma ? (double)__ldg(gamma + (int64_t)sp.l * n.C + ch) : 1.0;
                t1 += w * s[ch];
                t2 += w * s[kSumsPlane + ch];
            }
            t1 = add_lanes(t1, gl.seg);
            t2 = add_lanes(t2, gl.seg);
            if (on && gl.in == 0) part[to * n.G + g] = make_double2(t1, t2);
        }
        at += sp.rows;
        __syncthreads();
    }
}

// Level l's parameter gradients, 32 channels of them: the channel sums of all
// its spans in double, one warp per share of the spans.
__device__ __forceinline__ void add_parameters(Shares& sh, const float* chan, const NormShape& n,
                                               int l, int c, float* dgamma, float* dbeta)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double2 acc = make_double2(0.0, 0.0);
    for (int b = 0; b < n.B; ++b) {
        const int64_t lo = (int64_t)b * n.used + n.cum[l], hi = (int64_t)b * n.used + n.cum[l + 1];
        const int r0 = run_of(n, lo), r1 = run_of(n, hi - 1);
#pragma unroll 8
        for (int r = r0 + warp; c < n.C && r <= r1; r += kNormWarps) {
            const float* p = chan + span_slot(r, (int64_t)b * n.L + l) * 2 * n.C + c;
            acc.x += (double)p[0];
            acc.y += (double)p[n.C];
        }
    }
    sh.s[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && c < n.C) {
        for (int k = 1; k < kNormWarps; ++k) {
            acc.x += sh.s[k][lane].x;
            acc.y += sh.s[k][lane].y;
        }
        if (dbeta) dbeta[(int64_t)l * n.C + c] = (float)acc.x;
        if (dgamma) dgamma[(int64_t)l * n.C + c] = (float)acc.y;
    }
}

struct GradSmem {
    Shares shares;
    float c1[kMaxC], c2[kMaxC];
};

// Block i of the parameters' gradients: a level's 32 channels.
__device__ __forceinline__ int parameter_blocks(const NormShape& n) { return n.L * ((n.C + 31) / 32); }

__device__ __forceinline__ void parameter_block(Shares& sh, const float* chan, const NormShape& n,
                                                int i, const GradOut& out)
{
    const int blocks = (n.C + 31) / 32, l = i / blocks;
    add_parameters(sh, chan, n, l, (i - l * blocks) * 32 + (threadIdx.x & 31), out.dgamma,
                   out.dbeta);
}

template <bool kX, bool kDy, bool kDx, int kAct, typename Ready>
__device__ __forceinline__ void norm_grad_apply(GradSmem& sm, const GradIn& in, const NormShape& n,
                                                const double2* part, const GradOut& out, int run,
                                                Ready ready)
{
    constexpr bool kSplit = !(kX && kDy && kDx);
    const void *__restrict__ x = in.x, *__restrict__ dy = in.dy;
    const float *mean = in.mean, *rstd = in.rstd, *gamma = in.gamma, *beta = in.beta;
    Shares& shares = sm.shares;
    float *c1s = sm.c1, *c2s = sm.c2;
    const int slot = threadIdx.x / n.tpr;
    const Quads c = quads_of<kSplit>(n.C, threadIdx.x - slot * n.tpr);
    const int64_t begin = run_begin(n, run);
    bool waited = false;
    for (int64_t end = run_begin(n, run + 1); end > begin;) {
        const Span sp = span_before(n, begin, end);
        const Walk2<kX, kDy, kSplit> walk{
            ring_memory,
            x,
            dy,
            c,
            (sp.row + sp.rows - 1 - slot) * n.C,
            -(int64_t)n.slots * n.C,
            slot < n.slots ? (sp.rows - slot + n.slots - 1) / n.slots : 0};
        walk.start();
        if (!waited) ready();
        waited = true;
        const double inv = 1.0 / ((double)(n.cum[sp.l + 1] - n.cum[sp.l]) * n.cg);
        for (int g0 = 0; g0 < n.G; g0 += 32) {
            const int g = g0 + (threadIdx.x & 31);
            const double2 acc = add_spans(shares, part, n, sp.b, sp.l, g);
            if (threadIdx.x < 32 && g < n.G) {
                c1s[g] = (float)(acc.x * inv);
                c2s[g] = (float)(acc.y * inv);
            }
            __syncthreads();
        }
        if (slot < n.slots) {
            const Channels k = load_constants(n, sp.b, sp.l, c, mean, rstd, gamma, beta);
            Vec8 c1, c2;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c1.v[j] = c1s[channel(c, j) / n.cg];
                c2.v[j] = c2s[channel(c, j) / n.cg];
            }
            walk.run([&](int64_t at, const Vec8& v, const Vec8& d) {
                Vec8 o;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float hat = (v.v[j] - k.mean.v[j]) * k.rstd.v[j];
                    const float dz = grad_z<kAct>(d.v[j], v.v[j], k.mean.v[j], k.rstd.v[j], hat,
                                                  k.gamma.v[j], k.beta.v[j]);
                    // t rounded before the mean is taken off: exactly 0 where the
                    // group has one value
                    const float t = __fmul_rn(k.gamma.v[j], dz);
                    o.v[j] = k.rstd.v[j] * fmaf(-hat, c2.v[j], __fsub_rn(t, c1.v[j]));
                }
                store8<kDx, kSplit>(out.dx, at, c, o);
            });
        }
        end -= sp.rows;
        __syncthreads();
    }
    zero_gaps<kDx>(n, out.dx, run, n.runs);
}

template <bool kX, bool kDy, int kAct>
__global__ void __launch_bounds__(kNormThreads, 2) norm_grad_sums_kernel(
    const GradIn in, const NormShape n, float* __restrict__ chan, double2* __restrict__ part)
{
    pdl_trigger();
    norm_grad_sums<kX, kDy, kAct>(in, n, chan, part);
}

// The CTAs behind the runs take a block of the parameters' gradients each.
template <bool kX, bool kDy, bool kDx, int kAct>
__global__ void __launch_bounds__(kNormThreads, 2) norm_grad_apply_kernel(
    const GradIn in, const NormShape n, const float* chan, const double2* part, const GradOut out)
{
    __shared__ GradSmem sm;
    const int i = (int)blockIdx.x - n.runs;
    if (i >= 0) {
        pdl_wait();
        parameter_block(sm.shares, chan, n, i, out);
    } else {
        norm_grad_apply<kX, kDy, kDx, kAct>(sm, in, n, part, out, -1 - i, [] { pdl_wait(); });
    }
}

// Both passes, for one cluster.
template <bool kX, bool kDy, bool kDx, int kAct>
__global__ void __launch_bounds__(kNormThreads, 2) norm_grad_small_kernel(const GradIn in,
                                                                          const NormShape n,
                                                                          float* chan,
                                                                          double2* part,
                                                                          const GradOut out)
{
    __shared__ GradSmem sm;
    norm_grad_sums<kX, kDy, kAct>(in, n, chan, part);
    cluster_sync();
    norm_grad_apply<kX, kDy, kDx, kAct>(sm, in, n, part, out, blockIdx.x, [] {});
    for (int i = blockIdx.x; i < parameter_blocks(n); i += gridDim.x) {
        __syncthreads();  // the shares are free
        parameter_block(sm.shares, chan, n, i, out);
    }
}

// ------------------------------------------------------------------- host

bool norm_sizes_ok(const msda_norm_dims_t& d)
{
    return d.B >= 0 && d.Nv >= 1 && d.C >= 8 && d.C % 8 == 0 && d.C <= kMaxC && d.L >= 1 &&
           d.L <= MSDA_MAX_LEVELS && d.G >= 1 && d.C % d.G == 0;
}

// Spans, at most: each starts where a run or a level does.
size_t norm_max_spans(const msda_norm_dims_t& d)
{
    return (size_t)kMaxRuns + (size_t)d.B * d.L;
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
        // (levels that do not share rows hold Nv together at most)
        if (h * w > d.Nv - n.cum[l])
            return api_failf(MSDA_ERR_INVALID_ARG, "level %d shares rows with another", l);
        n.cum[l + 1] = n.cum[l] + (int)(h * w);
        int k = l;  // the levels by their first row
        for (; k > 0 && n.start[order[k - 1]] > n.start[l]; --k) order[k] = order[k - 1];
        order[k] = l;
    }
    n.used = n.cum[d.L];
    int at = 0;
    for (int k = 0; k <= d.L; ++k) {
        const int start = k < d.L ? n.start[order[k]] : d.Nv;
        if (start < at)
            return api_failf(MSDA_ERR_INVALID_ARG, "level %d shares rows with another", order[k]);
        if (start > at) {
            n.gap_start[n.gaps] = at;
            n.gap_rows[n.gaps++] = start - at;
        }
        if (k < d.L) at = start + n.cum[order[k] + 1] - n.cum[order[k]];
    }
    // rows are counted in 48 bits, so that their products with the runs fit 64
    if ((int64_t)d.B * d.Nv > ((int64_t)1 << 48) || (int64_t)d.B * d.L > INT32_MAX)
        return api_fail(MSDA_ERR_UNSUPPORTED, "too many rows");
    // four rows per thread at least; up to kSmallRows in one cluster
    const int64_t rows = (int64_t)d.B * n.used, least = (int64_t)n.slots * 4;
    n.small = rows <= (int64_t)kCluster * n.slots * kSmallRows;
    n.runs = (int)std::min<int64_t>(n.small ? kCluster : kMaxRuns, (rows + least - 1) / least);
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

struct NormArgs {
    const void* x;
    NormShape n;
    double2* part;
    double* middle;
    NormOut out;
};

template <bool kX, bool kY, int kAct>
cudaError_t run_forward(const NormArgs& a, cudaStream_t s)
{
    const dim3 block(kNormThreads);
    cudaError_t e;
    if (a.n.small) {
        e = allow_shared<norm_small_kernel<kX, kY, kAct>>(kRingBytes);
        if (e != cudaSuccess) return e;
        return launch_clusters(norm_small_kernel<kX, kY, kAct>, a.n.runs, dim3(a.n.runs), block,
                               kRingBytes, s, a.x, a.n, a.part, a.middle, a.out);
    }
    e = allow_shared<norm_stats_kernel<kX>>(kRingBytes);
    if (e == cudaSuccess) e = allow_shared<norm_apply_kernel<kX, kY, kAct>>(kRingBytes);
    if (e != cudaSuccess) return e;
    norm_stats_kernel<kX><<<a.n.runs, block, kRingBytes, s>>>(a.x, a.n, a.part, a.middle);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_apply_kernel<kX, kY, kAct>, dim3(a.n.runs), block, kRingBytes, s, a.x,
                      a.n, a.part, a.middle, a.out);
}

template <bool kX, bool kY>
cudaError_t run_forward(const NormArgs& a, msda_activation_t act, cudaStream_t s)
{
    if (act == MSDA_ACT_RELU) return run_forward<kX, kY, MSDA_ACT_RELU>(a, s);
    if (act == MSDA_ACT_SILU) return run_forward<kX, kY, MSDA_ACT_SILU>(a, s);
    return run_forward<kX, kY, MSDA_ACT_NONE>(a, s);
}

struct GradArgs {
    GradIn in;
    NormShape n;
    float* chan;
    double2* part;
    GradOut out;
};

template <bool kX, bool kDy, bool kDx, int kAct>
cudaError_t run_backward(const GradArgs& a, cudaStream_t s)
{
    const NormShape& n = a.n;
    const dim3 block(kNormThreads);
    cudaError_t e;
    if (n.small) {
        e = allow_shared<norm_grad_small_kernel<kX, kDy, kDx, kAct>>(kRingBytes);
        if (e != cudaSuccess) return e;
        return launch_clusters(norm_grad_small_kernel<kX, kDy, kDx, kAct>, n.runs, dim3(n.runs),
                               block, kRingBytes, s, a.in, n, a.chan, a.part, a.out);
    }
    e = allow_shared<norm_grad_sums_kernel<kX, kDy, kAct>>(kRingBytes);
    if (e == cudaSuccess) e = allow_shared<norm_grad_apply_kernel<kX, kDy, kDx, kAct>>(kRingBytes);
    if (e != cudaSuccess) return e;
    norm_grad_sums_kernel<kX, kDy, kAct><<<n.runs, block, kRingBytes, s>>>(a.in, n, a.chan, a.part);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_grad_apply_kernel<kX, kDy, kDx, kAct>,
                      dim3(n.runs + n.L * ((n.C + 31) / 32)), block, kRingBytes, s, a.in, n,
                      a.chan, a.part, a.out);
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
    return up256(sizeof(double2) * norm_max_spans(d) * d.G) +
           up256(sizeof(double) * d.B * d.L * (size_t)d.G);
}

extern "C" size_t msda_group_norm_backward_workspace_size(msda_norm_dims_t d)
{
    if (!norm_sizes_ok(d)) return 0;
    return up256(sizeof(double2) * norm_max_spans(d) * d.G) +
           up256(sizeof(float) * 2 * norm_max_spans(d) * d.C);
}

extern "C" msda_status_t msda_group_norm(const void* x, msda_dtype_t x_dtype,
                                         const int64_t* spatial_shapes,
                                         const int64_t* level_start_index, msda_norm_dims_t d,
                                         const float* gamma, const float* beta, float eps,
                                         msda_activation_t act, msda_dtype_t y_dtype, void* y,
                                         float* mean, float* rstd, void* workspace,
                                         size_t workspace_bytes, msda_stream_t stream)
{
    NormArgs a;
    NORM_TRY(norm_shape(d, spatial_shapes, level_start_index, a.n));
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
    a.x = x;
    a.part = static_cast<double2*>(workspace);
    a.middle = reinterpret_cast<double*>(static_cast<char*>(workspace) +
                                         up256(sizeof(double2) * norm_max_spans(d) * d.G));
    a.out = {eps, gamma, beta, y, mean, rstd};
    const auto run = x_dtype == MSDA_BF16
                         ? (y_dtype == MSDA_BF16 ? run_forward<true, true> : run_forward<true, false>)
                         : (y_dtype == MSDA_BF16 ? run_forward<false, true>
                                                 : run_forward<false, false>);
    return api_cuda(run(a, act, (cudaStream_t)stream), "msda_group_norm");
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
    a.in = {x, grad_y, mean, rstd, gamma, beta};
    a.part = reinterpret_cast<double2*>(w);
    a.chan = reinterpret_cast<float*>(w + up256(sizeof(double2) * norm_max_spans(d) * d.G));
    a.out = {grad_x, grad_gamma, grad_beta};
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
