// msda_query_attention: attention among object queries with a distance bias
// and group masks (forward).
//   s_ij = scale q_i . k_j - tau_i |p_i - p_j|,  out_i = sum_j softmax(s)_ij v_j
// One pass over the keys with the running maximum and sum of the softmax, in
// the base-2 logarithm's units.  A CTA takes 64 queries of one or (with the
// bias) two heads, so that a distance serves both; its keys come in tiles of
// 64 through a ring of asynchronous copies.  Tiles that no query of the CTA
// sees are skipped, tiles without a masked pair take no comparison.  Where the
// queries do not fill the GPU evenly the keys are split over the CTAs of a
// cluster, which join their sums through distributed shared memory.
//
// With 32 channels per head the products are not what binds: a score costs 64
// multiply-adds, but also an exponential, and a square root per pair of points
// and two heads, at 16 per clock and SM.  On the 100 x 100 grid with 8 heads (8e8
// pairs, 571 us) the exponential unit is busy half of the time, shared memory and
// instruction issue as well, the matrix pipe a third of it: no one unit binds,
// four warps per scheduler do not cover one another's latencies.
#include <algorithm>

#include "query_attention.cuh"

namespace msda {
namespace attn {
namespace {

constexpr int kBlocks = 4;  // CTAs per SM: 128 registers a thread (5 % faster than three)
constexpr int kStages = 3;  // tiles in shared memory
constexpr int kPart = 32;   // keys per step: scores and distances in registers

struct ForwardArgs {
    Inputs in;
    __nv_bfloat16* out;
    float* lse;
    int splits, split_tiles, q_tiles;
};

// Tiles that a CTA keeps where splits only even out the last wave (18 tiles in
// three parts: 37 us for the first pass of the gradient of 1100 queries, 29 us
// in one; 79 tiles in two: 155 us for 5000 queries, 181 us in one).
constexpr int kEvenTiles = 32;
constexpr int kPartRow = 36;  // floats of a row of split sums, padded for the banks

template <int HP>
struct ForwardSmem {
    alignas(128) unsigned char k[kStages][HP * kTileBytes];
    alignas(128) unsigned char v[kStages][HP * kTileBytes];
    Points pos[kStages];
    alignas(8) int32_t group[kStages][kTile];
    TileBits bits;
};

template <int HP, bool kBias, bool kGroups>
__device__ __forceinline__ void load_keys(ForwardSmem<HP>& sm, int stage, const Inputs& in,
                                          const TileCopy<HP>& copy,
                                          const Tiles<kGroups>& set, int b, int tile)
{
    copy.fetch(smem_addr(sm.k[stage]), smem_addr(sm.v[stage]), tile, set.clear(tile),
               set.rows(tile));
    load_columns<kBias, kGroups>(sm.pos[stage], sm.group[stage], in.kp, in.kg,
                                 (int64_t)b * in.Nk, tile * kTile, in.Nk);
    cp_commit();
}

// The queries of a warp (`row` the thread's first) and the tiles [begin, last) of the
// keys: the sums o of weighted values and l of weights (a thread's own), relative to the
// scores m, or in the units of the logarithm base.
//
// One multiply-add takes a reference off the scores, as `base`, its product with scale
// and log2 e.  That product's rounding is in every exponent (and in lse, which undoes
// it), and leaves fp32 as a power of 2 from scores of 1e9 on.  So a CTA that ends with a
// reference past kFarLog2 is walked again (kFar), with the references taken off the scores
// themselves, base being 0: a score equal to its reference has the weight 1 at any size.
// Always so would take 600 us for the 100 x 100 grid instead of 571, with a branch in
// this walk 642.
template <int HP, bool kBias, bool kGroups, bool kExact, bool kFar>
__device__ __forceinline__ void walk(ForwardSmem<HP>& sm, const Inputs& in,
                                     const uint32_t (&qf)[HP][8], const float2 (&p)[2],
                                     const float (&tau)[HP][2], int g0, int g1, int b, int h,
                                     int qt, int begin, int last, float (&o)[HP][4][4],
                                     float (&m)[HP][2], float (&base)[HP][2], float2 (&l)[HP][2])
{
    const int lane = threadIdx.x & 31, t = lane & 3;
    const float unit = in.scale * kLog2e;
    // The reference that is taken off stays the same until a score is 2^kSlack
    // times above it: weights up to 2^kSlack are as exact as weights up to 1, and
    // after the first tiles nothing has to be scaled again.
    constexpr float kSlack = 8.0f;
    const float slack = kSlack / unit;
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        // (a padding query's reference is never passed, so that what it holds moves no
        // other row's)
        m[hh][0] = g0 < 0 ? INFINITY : -INFINITY;
        m[hh][1] = g1 < 0 ? INFINITY : -INFINITY;
        base[hh][0] = base[hh][1] = 0.0f;
        l[hh][0] = l[hh][1] = both(0.0f);
#pragma unroll
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[hh][d][i] = 0.0f;
    }
    const LaneAt lanes = lane_at(lane);
    const TileCopy<HP> copy(in.k + (int64_t)b * in.Nk * in.ldk + h * kDim, in.ldk,
                            in.v + (int64_t)b * in.Nk * in.ldv + h * kDim, in.ldv, in.Nk);
    for (int first = begin; first < last;) {
        const Tiles<kGroups> set{sm.bits, first, last, in.Nk / kTile};
        first = set.end();
        if constexpr (kGroups) {
            __syncthreads();  // the bits of the tiles before are read
            scan_tiles<false>(sm.bits, in.qg + (int64_t)b * in.Nq + qt * kRows,
                              min(kRows, in.Nq - qt * kRows), in.kg + (int64_t)b * in.Nk, in.Nk,
                              set.first, last);
        }
        int tile = set.next(set.first), stage = 0;
        if (tile >= last) continue;
        load_keys<HP, kBias, kGroups>(sm, 0, in, copy, set, b, tile);
        cp_wait<0>();
        __syncthreads();
        int ahead = set.next(tile + 1);
        if (ahead < last) load_keys<HP, kBias, kGroups>(sm, 1, in, copy, set, b, ahead);

        // A step is 32 keys of a head.  Its products are asked for one step early,
        // so that the matrix pipe works while the weights of the step before are
        // formed; the step after a tile's last is the next tile's first.
        float c[4][4];      // products of the next step
        float2 dist[4][2];  // distances of the next step's keys
        float2 s[4][2];     // scores, then weights, of this one
        const auto products = [&](int st, int part, int hh) {
            const uint32_t sk = smem_addr(sm.k[st]) + hh * kTileBytes;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t r[4];
                load_cols(r, sk, 4 * part + j, lanes);
                mma_first(c[j], qf[hh], r[0], r[1]);
                mma(c[j], qf[hh] + 4, r[2], r[3]);
            }
            if (kBias && hh == 0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = kPart * part + 8 * j + 2 * t;
                    const float2 x = *reinterpret_cast<const float2*>(&sm.pos[st].x[at]);
                    const float2 y = *reinterpret_cast<const float2*>(&sm.pos[st].y[at]);
                    dist[j][0] = distances(p[0].x, p[0].y, x, y);
                    dist[j][1] = distances(p[1].x, p[1].y, x, y);
                }
            }
        };
        // Scores from the products, and their row's reference.
        const auto scores = [&](int st, int part, int hh, int of_tile) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    s[j][half] = pair(c[j], half);
                    if constexpr (kBias)
                        s[j][half] = __ffma2_rn(dist[j][half], both(tau[hh][half]), s[j][half]);
                }
            }
            if (!set.clear(of_tile)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = kPart * part + 8 * j + 2 * t;
                    const int key = of_tile * kTile + at;
                    int2 kg = make_int2(0, 0);
                    if constexpr (kGroups) kg = *reinterpret_cast<const int2*>(&sm.group[st][at]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int qg = half ? g1 : g0;
                        if (key >= in.Nk || !sees(qg, kg.x)) s[j][half].x = -INFINITY;
                        if (key + 1 >= in.Nk || !sees(qg, kg.y)) s[j][half].y = -INFINITY;
                    }
                }
            }
            float top[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top[half] = fmaxf(s[0][half].x, s[0][half].y);
#pragma unroll
                for (int j = 1; j < 4; ++j) top[half] = max3(top[half], s[j][half].x, s[j][half].y);
            }
            if (__any_sync(0xffffffffu,
                           top[0] > m[hh][0] + slack || top[1] > m[hh][1] + slack)) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float n = top[half];
                    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 1));
                    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 2));
                    n = fmaxf(n, m[hh][half]);
                    // (a row that has seen nothing has nothing to scale)
                    const float f =
                        m[hh][half] == -INFINITY ? 0.0f : exp2_approx((m[hh][half] - n) * unit);
                    m[hh][half] = n;
                    if constexpr (!kFar) base[hh][half] = n == -INFINITY ? 0.0f : n * unit;
                    l[hh][half] = __fmul2_rn(l[hh][half], both(f));
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        o[hh][d][2 * half] *= f;
                        o[hh][d][2 * half + 1] *= f;
                    }
                }
            }
            if constexpr (kFar) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float off = m[hh][half] == -INFINITY ? 0.0f : -m[hh][half];
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j][half] = __fadd2_rn(s[j][half], both(off));
                }
            }
        };
        products(0, 0, 0);
        scores(0, 0, 0, tile);
        while (tile < last) {
            const int next = stage == kStages - 1 ? 0 : stage + 1;
            const int after = ahead < last ? set.next(ahead + 1) : last;
#pragma unroll
            for (int u = 0; u < HP * (kTile / kPart); ++u) {
                const int part = u / HP, hh = u % HP;
                const bool ends = u + 1 == HP * (kTile / kPart);
                if (ends) {
                    cp_wait<0>();     // the next tile is here, and
                    __syncthreads();  // nobody reads the one before this any more
                    if (after < last)
                        load_keys<HP, kBias, kGroups>(sm, next == kStages - 1 ? 0 : next + 1, in, copy,
                                                      set, b, after);
                    products(next, 0, 0);  // (of no use behind the last tile)
                } else {
                    products(stage, (u + 1) / HP, (u + 1) % HP);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float2 sum = both(0.0f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = __ffma2_rn(s[j][half], both(unit), both(-base[hh][half]));
                        s[j][half] = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        sum = __fadd2_rn(sum, s[j][half]);
                    }
                    l[hh][half] = __fadd2_rn(l[hh][half], sum);
                }
                const uint32_t sv = smem_addr(sm.v[stage]) + hh * kTileBytes;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // the weights in bf16: the matrix instruction's type, v's own; 2^-8 of
                    // each at most, what out's own rounding may be (with kExact 2^-16)
                    const uint32_t pf[4] = {pack_bf16(s[2 * k][0]), pack_bf16(s[2 * k][1]),
                                            pack_bf16(s[2 * k + 1][0]),
                                            pack_bf16(s[2 * k + 1][1])};
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        uint32_t r[4];
                        load_sum(r, sv, 2 * part + k, d, lanes);
                        mma(o[hh][2 * d], pf, r[0], r[1]);
                        mma(o[hh][2 * d + 1], pf, r[2], r[3]);
                        if constexpr (kExact) {
                            const uint32_t pr[4] = {pack_rest(s[2 * k][0], pf[0]),
                                                    pack_rest(s[2 * k][1], pf[1]),
                                                    pack_rest(s[2 * k + 1][0], pf[2]),
                                                    pack_rest(s[2 * k + 1][1], pf[3])};
                            mma(o[hh][2 * d], pr, r[0], r[1]);
                            mma(o[hh][2 * d + 1], pr, r[2], r[3]);
                        }
                    }
                }
                if (!ends) scores(stage, (u + 1) / HP, (u + 1) % HP, tile);
                else if (ahead < last) scores(next, 0, 0, ahead);
            }
            tile = ahead;
            ahead = after;
            stage = next;
        }
    }
}

// Where a CTA leaves its sums for the others of its cluster: in the place of the tiles.
template <int HP>
__device__ __forceinline__ float* split_sums(ForwardSmem<HP>& sm)
{
    static_assert(HP * kRows * (kPartRow + 2) * sizeof(float) <= sizeof(sm.k) + sizeof(sm.v), "");
    return reinterpret_cast<float*>(&sm);
}

// All of a CTA's work but the join.  Returns whether it has to be done again with kFar.
template <int HP, bool kBias, bool kGroups, bool kExact, bool kFar>
__device__ __forceinline__ bool attend(ForwardSmem<HP>& sm, const ForwardArgs& a)
{
    const Inputs& in = a.in;
    const int split = blockIdx.x % a.splits;  // its place in the cluster
    int id = blockIdx.x / a.splits;
    const int qt = id % a.q_tiles;
    id /= a.q_tiles;
    const int hg = id % (in.H / HP), b = id / (in.H / HP);
    const int h = hg * HP, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int row = qt * kRows + warp * 16 + g;  // and row + 8
    const bool on0 = row < in.Nq, on1 = row + 8 < in.Nq;
    const int64_t q0 = (int64_t)b * in.Nq + row;

    uint32_t qf[HP][8];
#pragma unroll
    for (int hh = 0; hh < HP; ++hh)
        load_rows(qf[hh], in.q + (int64_t)b * in.Nq * in.ldq + (h + hh) * kDim, in.ldq, row, on0,
                  on1, t);
    // Scores are kept in units of the products q . k, and tau in the same units:
    // one multiply-add adds the bias, another takes the reference off and
    // changes to the base-2 logarithm.
    float2 p[2] = {};
    float tau[HP][2] = {};
    if constexpr (kBias) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (!(half ? on1 : on0)) continue;
            const float2 at = __ldg(in.qp + q0 + 8 * half);
            p[half] = make_float2(-at.x, -at.y);
#pragma unroll
            for (int hh = 0; hh < HP; ++hh)
                tau[hh][half] =
                    tau_units(__ldg(in.tau + (q0 + 8 * half) * in.H + h + hh), in.scale);
        }
    }
    int g0 = 0, g1 = 0;
    if constexpr (kGroups) {
        g0 = on0 ? __ldg(in.qg + q0) : -1;
        g1 = on1 ? __ldg(in.qg + q0 + 8) : -1;
    }
    const int tiles = (in.Nk + kTile - 1) / kTile;
    const int begin = split * a.split_tiles, last = min(tiles, begin + a.split_tiles);
    float o[HP][4][4], m[HP][2], base[HP][2];
    float2 l[HP][2];
    walk<HP, kBias, kGroups, kExact, kFar>(sm, in, qf, p, tau, g0, g1, b, h, qt, begin, last, o, m,
                                           base, l);
    // References on the way to the last one leave nothing behind where they were far, their
    // sums being scaled by 0, unless these had left fp32.
    bool far = false;
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
            far = far || ((half ? g1 : g0) >= 0 &&
                          (is_far(base[hh][half]) ||
                           !(l[hh][half].x + l[hh][half].y < INFINITY)));
    }
    far = __syncthreads_or(far);  // (and the tiles have been read)
    if (!kFar && far) return true;

    // split keys: a row's sums, and their reference and sum of weights (of a far walk the
    // reference as a score, told by the sum's sign)
    float* part = split_sums(sm);
    float2* part_ml = reinterpret_cast<float2*>(part + HP * kRows * kPartRow);
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float sum = l[hh][half].x + l[hh][half].y;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int q = row + 8 * half;
            // a padding query saw the keys of group 0: it is left out here
            const bool dead = sum == 0.0f || (half ? g1 : g0) < 0;
            if (a.splits > 1) {
                const int r = hh * kRows + warp * 16 + g + 8 * half;
                float2* dst = reinterpret_cast<float2*>(part + r * kPartRow);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    dst[4 * d + t] = make_float2(o[hh][d][2 * half], o[hh][d][2 * half + 1]);
                if (t == 0)
                    part_ml[r] = dead   ? make_float2(-INFINITY, 0.0f)
                                 : kFar ? make_float2(m[hh][half], -sum)
                                        : make_float2(base[hh][half], sum);
                continue;
            }
            if (!(half ? on1 : on0)) continue;
            const float w = dead ? 0.0f : 1.0f / sum;
            uint32_t* dst = reinterpret_cast<uint32_t*>(
                a.out + (((int64_t)b * in.Nq + q) * in.H + h + hh) * kDim);
#pragma unroll
            for (int d = 0; d < 4; ++d)
                dst[4 * d + t] =
                    dead ? 0u : pack_bf16(o[hh][d][2 * half] * w, o[hh][d][2 * half + 1] * w);
            if (a.lse != nullptr && t == 0)
                a.lse[((int64_t)b * in.H + h + hh) * in.Nq + q] =
                    dead   ? -INFINITY
                    : kFar ? far_lse(m[hh][half], in.scale, sum)
                           : (base[hh][half] + log2f(sum)) * kLn2;
        }
    }
    return false;
}

// The parts of up to kMost CTAs of a cluster: each CTA joins every splits-th 16 rows,
// eight lanes and four channels a row.
template <int HP, int kMost>
__device__ __forceinline__ void join_splits(ForwardSmem<HP>& sm, const ForwardArgs& a)
{
    const Inputs& in = a.in;
    const int split = blockIdx.x % a.splits;
    int id = blockIdx.x / a.splits;
    const int qt = id % a.q_tiles;
    id /= a.q_tiles;
    const int h = id % (in.H / HP) * HP, b = id / (in.H / HP);
    const float unit = in.scale * kLog2e;
    const float* part = split_sums(sm);
    const float2* part_ml = reinterpret_cast<const float2*>(part + HP * kRows * kPartRow);
    const int c = threadIdx.x & 7;
    for (int r = split * 16 + (int)(threadIdx.x >> 3); r < HP * kRows; r += 16 * a.splits) {
        const int q = qt * kRows + r % kRows, hh = h + r / kRows;
        if (q >= in.Nq) continue;
        const uint32_t at = smem_addr(part + r * kPartRow + 4 * c), at_ml = smem_addr(part_ml + r);
        // (all at once: one of these reads takes as long as all of them)
        float2 ml[kMost];
        float4 v[kMost];
#pragma unroll
        for (int s = 0; s < kMost; ++s) {
            ml[s] = make_float2(-INFINITY, 0.0f);
            if (s < a.splits) {
                ml[s] = remote_f32x2(remote_addr(at_ml, s));
                v[s] = remote_f32x4(remote_addr(at, s));
            }
        }
        bool far_row = false;  // of a CTA: then all references as scores
#pragma unroll
        for (int s = 0; s < kMost; ++s) far_row = far_row || ml[s].y < 0.0f;
        float m = -INFINITY;
#pragma unroll
        for (int s = 0; s < kMost; ++s) {
            if (far_row && ml[s].y > 0.0f) ml[s].x /= unit;
            m = fmaxf(m, ml[s].x);
        }
        float sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int s = 0; s < kMost; ++s) {
            // nothing seen: the sums may be those of a padding row
            if (s >= a.splits || ml[s].y == 0.0f) continue;
            const float w = exp2_approx(far_row ? (ml[s].x - m) * unit : ml[s].x - m);
            sum = fmaf(w, fabsf(ml[s].y), sum);
            acc.x = fmaf(w, v[s].x, acc.x);
            acc.y = fmaf(w, v[s].y, acc.y);
            acc.z = fmaf(w, v[s].z, acc.z);
            acc.w = fmaf(w, v[s].w, acc.w);
        }
        const float w = sum == 0.0f ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint2*>(a.out + (((int64_t)b * in.Nq + q) * in.H + hh) * kDim + c * 4) =
            make_uint2(pack_bf16(acc.x * w, acc.y * w), pack_bf16(acc.z * w, acc.w * w));
        if (a.lse != nullptr && c == 0)
            a.lse[((int64_t)b * in.H + hh) * in.Nq + q] =
                sum == 0.0f ? -INFINITY
                : far_row   ? far_lse(m, in.scale, sum)
                            : (m + log2f(sum)) * kLn2;
    }
}

template <int HP, bool kBias, bool kGroups, bool kExact>
__global__ void __launch_bounds__(kAttnThreads, kBlocks)
    attention_forward_kernel(const __grid_constant__ ForwardArgs a)
{
    extern __shared__ __align__(128) unsigned char smem[];
    ForwardSmem<HP>& sm = *reinterpret_cast<ForwardSmem<HP>*>(smem);
    if (attend<HP, kBias, kGroups, kExact, false>(sm, a))
        attend<HP, kBias, kGroups, kExact, true>(sm, a);
    if (a.splits == 1) return;
    cluster_sync();
    if (a.splits <= kMaxSplits / 2) join_splits<HP, kMaxSplits / 2>(sm, a);
    else join_splits<HP, kMaxSplits>(sm, a);
    cluster_sync();  // nobody's shared memory goes while others read it
}

template <int HP, bool kBias, bool kGroups, bool kExact>
cudaError_t run(const ForwardArgs& a, cudaStream_t s)
{
    constexpr auto kernel = attention_forward_kernel<HP, kBias, kGroups, kExact>;
    const cudaError_t e = allow_shared<kernel>(sizeof(ForwardSmem<HP>));
    if (e != cudaSuccess) return e;
    const int64_t ctas = (int64_t)a.q_tiles * a.in.B * (a.in.H / HP) * a.splits;
    return launch_clusters(kernel, a.splits, dim3((unsigned)ctas), dim3(kAttnThreads),
                           sizeof(ForwardSmem<HP>), s, a);
}

}  // namespace

Plan plan_of(int B, int Nq, int Nk, int H, bool bias, bool groups, int blocks)
{
    Plan p;
    const int64_t wave = blocks * kSms;
    const int tiles = (Nk + kTile - 1) / kTile;
    int64_t ctas = (int64_t)((Nq + kRows - 1) / kRows) * B * H;
    p.heads = bias && H % 2 == 0 && ctas >= 2 * wave ? 2 : 1;
    ctas /= p.heads;
    int64_t splits = wave / std::max<int64_t>(ctas, 1);
    if (splits <= 1) {
        // waves in units of a whole one, 2 % of a wave for each split's join
        double least = 1e30;
        for (int s = 1; s == 1 || (!groups && s <= 4 && tiles / s >= kEvenTiles); ++s) {
            const double cost = (double)((ctas * s + wave - 1) / wave) / s + 0.02 * (s - 1);
            if (cost < least) {
                least = cost;
                splits = s;
            }
        }
    }
    splits = std::max<int64_t>(1, std::min<int64_t>({splits, (tiles + 1) / 2, kMaxSplits}));
    p.split_tiles = std::max<int>(1, (tiles + (int)splits - 1) / (int)splits);
    p.splits = std::max(1, (tiles + p.split_tiles - 1) / p.split_tiles);
    return p;
}

Inputs inputs_of(const msda_attention_t& p)
{
    Inputs in;
    in.q = static_cast<const __nv_bfloat16*>(p.q);
    in.k = static_cast<const __nv_bfloat16*>(p.k);
    in.v = static_cast<const __nv_bfloat16*>(p.v);
    in.ldq = p.q_stride;
    in.ldk = p.k_stride;
    in.ldv = p.v_stride;
    in.qp = reinterpret_cast<const float2*>(p.q_points);
    in.kp = reinterpret_cast<const float2*>(p.k_points);
    in.tau = p.tau;
    in.qg = p.q_group;
    in.kg = p.k_group;
    in.scale = p.scale;
    in.B = p.B;
    in.Nq = p.Nq;
    in.Nk = p.Nk;
    in.H = p.H;
    return in;
}

msda_status_t check_inputs(const msda_attention_t* p, bool& empty)
{
    const auto bad = [](const char* m) { return api_fail(MSDA_ERR_INVALID_ARG, m); };
    if (p == nullptr) return bad("the inputs are null");
    if (p->B < 0 || p->Nq < 0 || p->Nk < 0 || p->H < 1)
        return api_failf(MSDA_ERR_INVALID_ARG,
                         "B (%d), Nq (%d) and Nk (%d) must be >= 0 and H (%d) >= 1", p->B, p->Nq,
                         p->Nk, p->H);
    if (!(p->scale >= 1e-6f && p->scale <= 1e6f))
        return api_failf(MSDA_ERR_INVALID_ARG, "scale = %g is outside 1e-6 .. 1e6",
                         (double)p->scale);
    if (p->H > (1 << 20))
        return api_failf(MSDA_ERR_UNSUPPORTED, "H = %d is above 2^20", p->H);
    // CTAs are counted in 32 bits (rows and elements in 64)
    const int64_t rows = std::max(p->Nq, p->Nk);
    if (rows > INT32_MAX - 1024 ||
        (__int128)(rows / kRows + 1) * p->B * p->H * kMaxSplits > INT32_MAX)
        return api_fail(MSDA_ERR_UNSUPPORTED, "too many rows");
    // (a tensor without values may have no address)
    const bool some_q = p->B > 0 && p->Nq > 0, some_k = p->B > 0 && p->Nk > 0;
    if ((p->q_points || p->k_points || p->tau) &&
        ((some_q && !(p->q_points && p->tau)) || (some_k && !p->k_points)))
        return bad("q_points, k_points and tau go together");
    if ((p->q_group || p->k_group) && ((some_q && !p->q_group) || (some_k && !p->k_group)))
        return bad("q_group and k_group go together");
    empty = p->B == 0 || p->Nq == 0;
    const struct {
        const void* ptr;
        int64_t stride;
        int rows;
        const char* name;
    } t[3] = {{p->q, p->q_stride, p->Nq, "q"},
              {p->k, p->k_stride, p->Nk, "k"},
              {p->v, p->v_stride, p->Nk, "v"}};
    for (const auto& x : t) {
        if (p->B == 0 || x.rows == 0) continue;
        if (x.ptr == nullptr) return api_failf(MSDA_ERR_INVALID_ARG, "%s is null", x.name);
        if ((uintptr_t)x.ptr % 16)
            return api_failf(MSDA_ERR_INVALID_ARG, "%s must be 16-byte aligned", x.name);
        if (x.stride < (int64_t)p->H * kDim || x.stride % 8 || x.stride > ((int64_t)1 << 32))
            return api_failf(MSDA_ERR_INVALID_ARG,
                             "%s_stride = %lld is not a multiple of 8 from H * 32 = %d on", x.name,
                             (long long)x.stride, p->H * kDim);
    }
    if ((uintptr_t)p->q_points % 8 || (uintptr_t)p->k_points % 8)
        return bad("q_points and k_points must be 8-byte aligned");
    if ((uintptr_t)p->tau % 4 || (uintptr_t)p->q_group % 4 || (uintptr_t)p->k_group % 4)
        return bad("tau, q_group and k_group must be 4-byte aligned");
    return MSDA_OK;
}

bool touches_inputs(const msda_attention_t* p, const void* out, size_t bytes)
{
    const auto meets = [&](const void* in, int64_t stride, int rows) {
        const uintptr_t a = (uintptr_t)in, o = (uintptr_t)out;
        const size_t n = (size_t)p->B * rows;
        if (in == nullptr || out == nullptr || n == 0 || bytes == 0) return false;
        const uintptr_t end = a + ((n - 1) * (size_t)stride + (size_t)p->H * kDim) * 2;
        return a < o + bytes && o < end;
    };
    return meets(p->q, p->q_stride, p->Nq) || meets(p->k, p->k_stride, p->Nk) ||
           meets(p->v, p->v_stride, p->Nk);
}

msda_status_t check_workspace(const void* ws, size_t have, size_t need)
{
    if (need == 0 || (ws != nullptr && have >= need && (uintptr_t)ws % 256 == 0)) return MSDA_OK;
    return api_failf(MSDA_ERR_WORKSPACE,
                     "workspace of %zu bytes: %zu bytes on a 256-byte boundary are needed",
                     ws == nullptr ? (size_t)0 : have, need);
}

}  // namespace attn
}  // namespace msda

using namespace msda;
using namespace msda::attn;

extern "C" msda_status_t msda_query_attention(const msda_attention_t* p, void* out, float* lse,
                                              msda_stream_t stream)
{
    bool empty = false;
    const msda_status_t st = check_inputs(p, empty);
    if (st != MSDA_OK) return st;
    if (empty) return api_ok();
    if (out == nullptr || (uintptr_t)out % 16)
        return api_fail(MSDA_ERR_INVALID_ARG, "out is null or not 16-byte aligned");
    if ((uintptr_t)lse % 4)
        return api_fail(MSDA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
    if (touches_inputs(p, out, (size_t)p->B * p->Nq * p->H * kDim * 2) ||
        touches_inputs(p, lse, (size_t)p->B * p->Nq * p->H * 4))
        return api_fail(MSDA_ERR_INVALID_ARG, "out or lse overlaps q, k or v");
    const Plan plan = plan_of(p->B, p->Nq, p->Nk, p->H, p->tau != nullptr,
                              p->q_group || p->k_group, kBlocks);
    ForwardArgs a;
    a.in = inputs_of(*p);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.q_tiles = (p->Nq + kRows - 1) / kRows;
    a.splits = plan.splits;
    a.split_tiles = plan.split_tiles;
    const cudaStream_t s = (cudaStream_t)stream;
    const bool groups = p->q_group || p->k_group;
    using Run = cudaError_t (*)(const ForwardArgs&, cudaStream_t);
    static constexpr Run runs[8] = {
        run<1, false, false, false>, run<1, false, false, true>, run<1, false, true, false>,
        run<1, false, true, true>,   run<1, true, false, false>, run<1, true, false, true>,
        run<1, true, true, false>,   run<1, true, true, true>};
    const Run call = plan.heads == 2
                         ? (groups ? run<2, true, true, false> : run<2, true, false, false>)
                         : runs[4 * (p->tau != nullptr) + 2 * groups +
                                exact_of((int64_t)p->B * p->Nq * p->H)];
    return api_cuda(call(a, s), "msda_query_attention");
}
