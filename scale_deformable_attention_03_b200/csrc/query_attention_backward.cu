// msda_query_attention_backward: with p_ij = exp(s_ij - lse_i),
// dp_ij = do_i . v_j, D_i = sum_j p_ij dp_ij and ds_ij = p_ij (dp_ij - D_i):
//   dq_i = scale sum_j ds_ij k_j,  dtau_i = -sum_j ds_ij |p_i - p_j|
//   dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// Every sum has one owner, so no atomic is needed.  A first kernel walks the
// keys for D (split over the CTAs of a cluster like the forward), the second
// has two kinds of CTAs, which run side by side so that neither leaves the GPU
// half empty at its end: 64 queries and all keys for dq and dtau, 64 keys and
// all queries for dk and dv.  D is formed from the same p and dp that ds uses
// (not from the rounded output of the forward): ds is then exact where one key
// takes all the weight, and dtau, an fp32 sum of it, keeps fp32's precision.
//
// Like the forward it is bound by no single unit (5000 queries, 8 heads: 152 us for
// D, exponential unit 66 % busy; 386 us for the gradients, shared memory 69 %,
// issue 55 %, exponentials 51 %, matrix pipe 44 %): an exponential and a square
// root per pair in each of the three walks, and nine products for the five that a
// single walk with atomics would take.
#include <algorithm>

#include "query_attention.cuh"

namespace msda {
namespace attn {
namespace {

// CTAs per SM: 128 registers a thread for D (1100 queries in groups: 23 us, with three
// CTAs 27 us; 5000 queries 155 us with either), 168 for the gradients.
constexpr int kDotBlocks = 4, kBlocks = 3;
constexpr int kHalf = 32;  // columns per step: scores, dp and distances in registers

struct BackwardArgs {
    Inputs in;
    const __nv_bfloat16* go;  // [B, Nq, H * 32]
    const float* lse;
    __nv_bfloat16 *dq, *dk, *dv;
    float* dtau;
    // [3, B, H, Nq]: -lse and -tau in units of log 2 (of a far query the logarithm of its
    // weights' sum, negated, in the place of tau), D
    float* rows;
    int q_tiles, k_tiles, splits, split_tiles;
};

template <int HP>
struct BackwardSmem {
    alignas(128) unsigned char a[2][HP * kTileBytes];  // keys, or queries
    alignas(128) unsigned char b[2][HP * kTileBytes];  // values, or the output's gradient
    alignas(8) float rows[2][HP][3][kTile];  // of the queries (keys' kernel): lse, tau, D
    float dots[HP][kTile];        // D's sums where the keys are split,
    float weights[HP][kTile];     // and those of the weights in a far walk
    Points pos[2];
    int32_t group[2][kTile];
    TileBits bits;
    int32_t far;                  // a query is far (keys' kernel)
};

template <int HP, bool kBias, bool kGroups>
__device__ __forceinline__ void load_keys(BackwardSmem<HP>& sm, int stage, const Inputs& in,
                                          const TileCopy<HP>& copy,
                                          const Tiles<kGroups>& set, int b, int tile)
{
    copy.fetch(smem_addr(sm.a[stage]), smem_addr(sm.b[stage]), tile, set.clear(tile),
               set.rows(tile));
    load_columns<kBias, kGroups>(sm.pos[stage], sm.group[stage], in.kp, in.kg,
                                 (int64_t)b * in.Nk, tile * kTile, in.Nk);
    cp_commit();
}

template <int HP, bool kBias, bool kGroups>
__device__ __forceinline__ void load_queries(BackwardSmem<HP>& sm, int stage,
                                             const BackwardArgs& a, const TileCopy<HP>& copy,
                                             const Tiles<kGroups>& set, int b, int h, int tile)
{
    const Inputs& in = a.in;
    const int r0 = tile * kTile;
    copy.fetch(smem_addr(sm.a[stage]), smem_addr(sm.b[stage]), tile, set.clear(tile),
               set.rows(tile));
    const int64_t plane = (int64_t)in.B * in.H * in.Nq;
#pragma unroll
    for (int i0 = 0; i0 < 3 * HP * kTile; i0 += kAttnThreads) {
        const int i = i0 + (int)threadIdx.x;
        if (3 * HP * kTile % kAttnThreads != 0 && i >= 3 * HP * kTile) break;
        const int k = i / (HP * kTile), hh = i / kTile % HP, row = r0 + i % kTile;
        const bool on = row < in.Nq;
        const float* src = a.rows + k * plane + ((int64_t)b * in.H + h + hh) * in.Nq + row;
        cp_async<4>(smem_addr(&sm.rows[stage][hh][k][i % kTile]), on ? src : a.rows, on);
    }
    load_columns<kBias, kGroups>(sm.pos[stage], sm.group[stage], in.qp, in.qg, (int64_t)b * in.Nq, r0,
                        in.Nq);
    cp_commit();
}

// A step's 16 x 32 products of a warp's rows with the tile's rows 32s..32s+31:
// c[j][half] are the columns 8j + 2t, + 1 of the row g + 8 half.
__device__ __forceinline__ void products(float2 (&c)[4][2], const uint32_t (&f)[8], uint32_t tile,
                                         int s, const LaneAt& lanes)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t r[4];
        load_cols(r, tile, 4 * s + j, lanes);
        float v[4];
        mma_first(v, f, r[0], r[1]);
        mma(v, f + 4, r[2], r[3]);
        c[j][0] = pair(v, 0);
        c[j][1] = pair(v, 1);
    }
}

// acc += w (16 x 32, rounded to bf16: the matrix instruction's type; what that leaves
// over in a second product with kExact) times the tile's rows 32s .. 32s + 31.
template <bool kExact>
__device__ __forceinline__ void accumulate(float (&acc)[4][4], const float2 (&w)[4][2],
                                           uint32_t tile, int s, const LaneAt& lanes)
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t f[4] = {pack_bf16(w[2 * k][0]), pack_bf16(w[2 * k][1]),
                               pack_bf16(w[2 * k + 1][0]), pack_bf16(w[2 * k + 1][1])};
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            uint32_t r[4];
            load_sum(r, tile, 2 * s + k, d, lanes);
            mma(acc[2 * d], f, r[0], r[1]);
            mma(acc[2 * d + 1], f, r[2], r[3]);
            if constexpr (kExact) {
                const uint32_t e[4] = {pack_rest(w[2 * k][0], f[0]), pack_rest(w[2 * k][1], f[1]),
                                       pack_rest(w[2 * k + 1][0], f[2]),
                                       pack_rest(w[2 * k + 1][1], f[3])};
                mma(acc[2 * d], e, r[0], r[1]);
                mma(acc[2 * d + 1], e, r[2], r[3]);
            }
        }
    }
}

__device__ __forceinline__ void store_rows(__nv_bfloat16* p, int64_t row, int64_t heads, int h,
                                           const float (&acc)[4][4], float w, bool on0, bool on1,
                                           int t)
{
    uint32_t* lo = reinterpret_cast<uint32_t*>(p + (row * heads + h) * kDim) + t;
    uint32_t* hi = reinterpret_cast<uint32_t*>(p + ((row + 8) * heads + h) * kDim) + t;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        if (on0) lo[4 * d] = pack_bf16(acc[d][0] * w, acc[d][1] * w);
        if (on1) hi[4 * d] = pack_bf16(acc[d][2] * w, acc[d][3] * w);
    }
}

// Replaces the values of a pair whose bits are set.
__device__ __forceinline__ void mask(float2& v, uint32_t bits, float by)
{
    if (bits & 1) v.x = by;
    if (bits & 2) v.y = by;
}

__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

// D of a far query from its sums, and what its weights' logarithms are moved by.
__device__ __forceinline__ float normalise(float& norm, float dot, float weights)
{
    if (!(weights > 0.0f && weights < INFINITY)) return norm = 0.0f, dot;  // (lse is another's)
    norm = -log2f(weights);
    return dot / weights;
}

// The logarithms of the weights of a warp's 16 queries, `row` the thread's first, from
// their products, where a query of theirs is far.  Past 2^24 lse holds nothing of the
// logarithm of the weights' sum (where keys tie), so with kNormed a far query's weights
// are divided by their sum, which the walk for D has found.
template <bool kBias, bool kNormed>
__device__ __forceinline__ void far_rows(float2 (&s)[4][2], const float2 (&dist)[4][2],
                                         const BackwardArgs& a, const float (&e)[2], int b, int h,
                                         int row)
{
    const Inputs& in = a.in;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const bool live = e[half] != -INFINITY;
        const int64_t q = (int64_t)row + 8 * half;
        const float lse = live ? __ldg(a.lse + ((int64_t)b * in.H + h) * in.Nq + q) : INFINITY;
        float tau = 0.0f;
        if (kBias && live)
            tau = tau_units(__ldg(in.tau + ((int64_t)b * in.Nq + q) * in.H + h), in.scale);
        float norm = 0.0f;
        if (kNormed && is_far(e[half]))
            norm = a.rows[((int64_t)in.B * in.H + (int64_t)b * in.H + h) * in.Nq + q];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (kBias) s[j][half] = __ffma2_rn(dist[j][half], both(tau), s[j][half]);
            s[j][half] = make_float2(far_log2(s[j][half].x, in.scale, lse) + norm,
                                     far_log2(s[j][half].y, in.scale, lse) + norm);
        }
    }
}

// The same with the queries as columns, step st of a tile; `e` and `norms` the tile's.
template <bool kBias>
__device__ __forceinline__ void far_columns(float2 (&s)[4][2], const float2 (&dist)[4][2],
                                            const BackwardArgs& a, const float* e,
                                            const float* norms, int b, int h, int tile, int st)
{
    const Inputs& in = a.in;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int at = kHalf * st + 8 * j + 2 * (threadIdx.x & 3) + c;
            const int64_t q = (int64_t)tile * kTile + at;
            const bool live = q < in.Nq && e[at] != -INFINITY;
            const float lse = live ? __ldg(a.lse + ((int64_t)b * in.H + h) * in.Nq + q) : INFINITY;
            float tau = 0.0f;
            if (kBias && live)
                tau = tau_units(__ldg(in.tau + ((int64_t)b * in.Nq + q) * in.H + h), in.scale);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float& x = c ? s[j][half].y : s[j][half].x;
                if constexpr (kBias) x = fmaf(c ? dist[j][half].y : dist[j][half].x, tau, x);
                x = far_log2(x, in.scale, lse) + (is_far(e[at]) ? norms[at] : 0.0f);
            }
        }
    }
}

// 64 queries and the tiles [begin, last) of the keys: D (and what the last
// kernel needs of the queries beside it), or with kGrad, given D, dq and dtau.
// Returns whether a query of theirs is far, and they have to be walked again with kFar:
// a walk of its own, since a branch in this one takes registers that it has not got (7 %
// of the gradient of 5000 queries).
template <int HP, bool kBias, bool kGroups, bool kGrad, bool kExact, bool kFar>
__device__ __forceinline__ bool walk_keys(BackwardSmem<HP>& sm, const BackwardArgs& a, int id,
                                          int split)
{
    const Inputs& in = a.in;
    const int qt = id % a.q_tiles;
    id /= a.q_tiles;
    const int h = id % (in.H / HP) * HP, b = id / (in.H / HP);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int row = qt * kRows + warp * 16 + g;
    const bool on0 = row < in.Nq, on1 = row + 8 < in.Nq;
    const int64_t q0 = (int64_t)b * in.Nq + row;

    uint32_t qf[HP][8], of[HP][8];
    float e[HP][2], tau[HP][2] = {};  // -lse, -tau in units of log 2
    float2 p[2] = {};
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        bool live[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int64_t i = ((int64_t)b * in.H + h + hh) * in.Nq + row + 8 * half;
            const float lse = (half ? on1 : on0) ? __ldg(a.lse + i) : -INFINITY;
            live[half] = lse != -INFINITY;
            // a row that sees nothing: weight exp2(s - infinity) = 0 everywhere
            e[hh][half] = live[half] ? -lse * kLog2e : -INFINITY;
            if constexpr (kBias) {
                if (live[half])
                    tau[hh][half] = -__ldg(in.tau + (q0 + 8 * half) * in.H + h + hh) * kLog2e;
            }
        }
        load_rows(qf[hh], in.q + (int64_t)b * in.Nq * in.ldq + (h + hh) * kDim, in.ldq, row,
                  live[0], live[1], t);
        load_rows(of[hh], a.go + ((int64_t)b * in.Nq * in.H + h + hh) * kDim,
                  (int64_t)in.H * kDim, row, live[0], live[1], t);
    }
    if constexpr (kBias) {  // (a row that sees nothing may have any point)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (e[0][half] == -INFINITY) continue;
            const float2 at = __ldg(in.qp + q0 + 8 * half);
            p[half] = make_float2(-at.x, -at.y);
        }
    }
    int g0 = 0, g1 = 0;
    if constexpr (kGroups) {
        g0 = on0 ? __ldg(in.qg + q0) : -1;
        g1 = on1 ? __ldg(in.qg + q0 + 8) : -1;
    }
    const float scale = in.scale * kLog2e;
    float D[HP][2] = {}, dt[HP][2] = {}, dq[HP][4][4] = {};
    float weights[HP][2] = {};  // their sums, of the far walk for D
    const int64_t plane = (int64_t)in.B * in.H * in.Nq;
    if constexpr (kGrad) {
#pragma unroll
        for (int hh = 0; hh < HP; ++hh)
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (half ? on1 : on0)
                    D[hh][half] = a.rows[2 * plane + ((int64_t)b * in.H + h + hh) * in.Nq + row +
                                         8 * half];
    }

    const int begin = kGrad ? 0 : split * a.split_tiles;
    const int last = kGrad ? a.k_tiles : min(a.k_tiles, begin + a.split_tiles);
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
        if (tile < last) load_keys<HP, kBias, kGroups>(sm, stage, in, copy, set, b, tile);
        while (tile < last) {
            const int ahead = set.next(tile + 1);
            if (ahead < last) {
                load_keys<HP, kBias, kGroups>(sm, stage ^ 1, in, copy, set, b, ahead);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
            const bool clear = set.clear(tile);
#pragma unroll
            for (int st = 0; st < kTile / kHalf; ++st) {
                float2 dist[4][2];
                uint32_t hide = 0;
                if constexpr (kBias) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = kHalf * st + 8 * j + 2 * t;
                        const float2 x = *reinterpret_cast<const float2*>(&sm.pos[stage].x[at]);
                        const float2 y = *reinterpret_cast<const float2*>(&sm.pos[stage].y[at]);
                        dist[j][0] = distances(p[0].x, p[0].y, x, y);
                        dist[j][1] = distances(p[1].x, p[1].y, x, y);
                    }
                }
                if (!clear) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int at = kHalf * st + 8 * j + 2 * t + c;
                            const bool in_range = tile * kTile + at < in.Nk;
                            const int kg = kGroups ? sm.group[stage][at] : 0;
                            hide |= (uint32_t)!(in_range && sees(g0, kg)) << (4 * j + c);
                            hide |= (uint32_t)!(in_range && sees(g1, kg)) << (4 * j + 2 + c);
                        }
                    }
                    if constexpr (kBias) {  // a masked point may be anything
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                mask(dist[j][half], hide >> (4 * j + 2 * half), 0.0f);
                    }
                }
#pragma unroll
                for (int hh = 0; hh < HP; ++hh) {
                    const uint32_t sk = smem_addr(sm.a[stage]) + hh * kTileBytes;
                    const uint32_t sv = smem_addr(sm.b[stage]) + hh * kTileBytes;
                    float2 s[4][2], dp[4][2];
                    products(s, qf[hh], sk, st, lanes);
                    products(dp, of[hh], sv, st, lanes);
                    if constexpr (kFar)
                        far_rows<kBias, kGrad>(s, dist, a, e[hh], b, h + hh, row);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float2 x = s[j][half];
                            if constexpr (!kFar) {
                                x = __ffma2_rn(x, both(scale), both(e[hh][half]));
                                if constexpr (kBias)
                                    x = __ffma2_rn(dist[j][half], both(tau[hh][half]), x);
                            }
                            if (!clear) mask(x, hide >> (4 * j + 2 * half), -INFINITY);
                            s[j][half] = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        }
                    }
                    float2 sum[2] = {both(0.0f), both(0.0f)};  // a step's own, then the total
                    if constexpr (!kGrad) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                sum[half] = __ffma2_rn(s[j][half], dp[j][half], sum[half]);
                        D[hh][0] += sum[0].x + sum[0].y;
                        D[hh][1] += sum[1].x + sum[1].y;
                        if constexpr (kFar) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int half = 0; half < 2; ++half)
                                    weights[hh][half] += s[j][half].x + s[j][half].y;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                s[j][half] = __fmul2_rn(
                                    s[j][half], __fadd2_rn(dp[j][half], both(-D[hh][half])));
                                if constexpr (kBias)
                                    sum[half] =
                                        __ffma2_rn(s[j][half], dist[j][half], sum[half]);
                            }
                        }
                        dt[hh][0] += sum[0].x + sum[0].y;
                        dt[hh][1] += sum[1].x + sum[1].y;
                        accumulate<kExact>(dq[hh], s, sk, st, lanes);
                    }
                }
            }
            __syncthreads();
            tile = ahead;
            stage ^= 1;
        }
    }
    if constexpr (!kGrad) {
#pragma unroll
        for (int hh = 0; hh < HP; ++hh) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                D[hh][half] = quad_sum(D[hh][half]);
                if constexpr (kFar) weights[hh][half] = quad_sum(weights[hh][half]);
                if (t != 0) continue;
                if (a.splits > 1) {
                    sm.dots[hh][warp * 16 + g + 8 * half] = D[hh][half];
                    if constexpr (kFar) sm.weights[hh][warp * 16 + g + 8 * half] = weights[hh][half];
                }
                if (split != 0 || !(half ? on1 : on0)) continue;
                const int64_t i = ((int64_t)b * in.H + h + hh) * in.Nq + row + 8 * half;
                a.rows[i] = e[hh][half];
                a.rows[plane + i] = tau[hh][half];
                if (a.splits == 1) {
                    if (kFar && is_far(e[hh][half]))
                        D[hh][half] = normalise(a.rows[plane + i], D[hh][half], weights[hh][half]);
                    a.rows[2 * plane + i] = D[hh][half];
                }
            }
        }
        if (a.splits > 1) {
            cluster_sync();
            for (int i = threadIdx.x; split == 0 && i < HP * kTile; i += kAttnThreads) {
                const int q = qt * kRows + i % kTile;
                if (q >= in.Nq) continue;
                float sum = 0.0f;
                for (int s = 0; s < a.splits; ++s)
                    sum += remote_f32(remote_addr(smem_addr(&sm.dots[0][i]), s));
                const int64_t at = ((int64_t)b * in.H + h + i / kTile) * in.Nq + q;
                if constexpr (kFar) {
                    float all = 0.0f;
                    for (int s = 0; s < a.splits; ++s)
                        all += remote_f32(remote_addr(smem_addr(&sm.weights[0][i]), s));
                    if (is_far(a.rows[at])) sum = normalise(a.rows[plane + at], sum, all);
                }
                a.rows[2 * plane + at] = sum;
            }
            cluster_sync();  // nobody's shared memory goes while others read it
        }
    } else {
#pragma unroll
        for (int hh = 0; hh < HP; ++hh) {
            store_rows(a.dq, q0, in.H, h + hh, dq[hh], in.scale, on0, on1, t);
            if constexpr (kBias) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float sum = quad_sum(dt[hh][half]);
                    if (t == 0 && (half ? on1 : on0))
                        a.dtau[(q0 + 8 * half) * in.H + h + hh] = -sum;
                }
            }
        }
    }
    bool far = false;
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) far = far || is_far(e[hh][0]) || is_far(e[hh][1]);
    return !kFar && __syncthreads_or(far);
}

// 64 keys and all queries: dk and dv.  Returns whether a query that was read is far, and
// they have to be walked again with kFar.
template <int HP, bool kBias, bool kGroups, bool kExact, bool kFar>
__device__ __forceinline__ bool walk_queries(BackwardSmem<HP>& sm, const BackwardArgs& a, int id)
{
    const Inputs& in = a.in;
    const int kt = id % a.k_tiles;
    id /= a.k_tiles;
    const int h = id % (in.H / HP) * HP, b = id / (in.H / HP);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int row = kt * kRows + warp * 16 + g;
    const bool on0 = row < in.Nk, on1 = row + 8 < in.Nk;
    const int64_t k0 = (int64_t)b * in.Nk + row;
    int g0 = on0 ? 0 : -1, g1 = on1 ? 0 : -1;
    const int own_rows = min(kRows, in.Nk - kt * kRows);
    if constexpr (kGroups) {
        if (on0) g0 = __ldg(in.kg + k0);
        if (on1) g1 = __ldg(in.kg + k0 + 8);
    }
    uint32_t kf[HP][8], vf[HP][8];
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        load_rows(kf[hh], in.k + (int64_t)b * in.Nk * in.ldk + (h + hh) * kDim, in.ldk, row,
                  g0 >= 0, g1 >= 0, t);
        load_rows(vf[hh], in.v + (int64_t)b * in.Nk * in.ldv + (h + hh) * kDim, in.ldv, row,
                  g0 >= 0, g1 >= 0, t);
    }
    float2 p[2] = {};
    if constexpr (kBias) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if ((half ? g1 : g0) < 0) continue;
            const float2 at = __ldg(in.kp + k0 + 8 * half);
            p[half] = make_float2(-at.x, -at.y);
        }
    }
    const float scale = in.scale * kLog2e;
    float dk[HP][4][4] = {}, dv[HP][4][4] = {};
    // (a barrier comes before the first tile; kFar writes nothing, since others may still be
    // reading it)
    if (!kFar && threadIdx.x == 0) sm.far = 0;

    const LaneAt lanes = lane_at(lane);
    const TileCopy<HP> copy(in.q + (int64_t)b * in.Nq * in.ldq + h * kDim, in.ldq,
                            a.go + ((int64_t)b * in.Nq * in.H + h) * kDim, (int64_t)in.H * kDim,
                            in.Nq);
    const int tiles = a.q_tiles;
    for (int first = 0; first < tiles;) {
        const Tiles<kGroups> set{sm.bits, first, tiles,
                                 own_rows == kRows ? in.Nq / kTile : 0};
        first = set.end();
        if constexpr (kGroups) {
            __syncthreads();
            scan_tiles<true>(sm.bits, in.kg + (int64_t)b * in.Nk + kt * kRows, own_rows,
                             in.qg + (int64_t)b * in.Nq, in.Nq, set.first, tiles);
        }
        int tile = set.next(set.first), stage = 0;
        if (tile < tiles) load_queries<HP, kBias, kGroups>(sm, stage, a, copy, set, b, h, tile);
        while (tile < tiles) {
            const int ahead = set.next(tile + 1);
            if (ahead < tiles) {
                load_queries<HP, kBias, kGroups>(sm, stage ^ 1, a, copy, set, b, h, ahead);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
            if (!kFar && (int)threadIdx.x < kTile) {
#pragma unroll
                for (int hh = 0; hh < HP; ++hh)
                    if (is_far(sm.rows[stage][hh][0][threadIdx.x])) sm.far = 1;
            }
            const bool clear = set.clear(tile);
#pragma unroll
            for (int st = 0; st < kTile / kHalf; ++st) {
                float2 dist[4][2];
                uint32_t hide = 0;
                if constexpr (kBias) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = kHalf * st + 8 * j + 2 * t;
                        const float2 x = *reinterpret_cast<const float2*>(&sm.pos[stage].x[at]);
                        const float2 y = *reinterpret_cast<const float2*>(&sm.pos[stage].y[at]);
                        dist[j][0] = distances(p[0].x, p[0].y, x, y);
                        dist[j][1] = distances(p[1].x, p[1].y, x, y);
                    }
                }
                if (!clear) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int at = kHalf * st + 8 * j + 2 * t + c;
                            const bool in_range = tile * kTile + at < in.Nq;
                            const int qg = kGroups ? sm.group[stage][at] : 0;
                            hide |= (uint32_t)!(in_range && sees(qg, g0)) << (4 * j + c);
                            hide |= (uint32_t)!(in_range && sees(qg, g1)) << (4 * j + 2 + c);
                        }
                    }
                }
#pragma unroll
                for (int hh = 0; hh < HP; ++hh) {
                    const uint32_t sq = smem_addr(sm.a[stage]) + hh * kTileBytes;
                    const uint32_t so = smem_addr(sm.b[stage]) + hh * kTileBytes;
                    float2 s[4][2], dp[4][2];
                    products(s, kf[hh], sq, st, lanes);
                    products(dp, vf[hh], so, st, lanes);
                    if constexpr (kFar)
                        far_columns<kBias>(s, dist, a, sm.rows[stage][hh][0],
                                           sm.rows[stage][hh][1], b, h + hh, tile, st);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = kHalf * st + 8 * j + 2 * t;
                        float2 r[3];
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            r[k] = *reinterpret_cast<const float2*>(&sm.rows[stage][hh][k][at]);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float2 x = s[j][half];
                            if constexpr (!kFar) {
                                x = __ffma2_rn(x, both(scale), r[0]);
                                if constexpr (kBias) x = __ffma2_rn(dist[j][half], r[1], x);
                            }
                            if (!clear) mask(x, hide >> (4 * j + 2 * half), -INFINITY);
                            s[j][half] = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                            dp[j][half] = __fmul2_rn(
                                s[j][half],
                                __fadd2_rn(dp[j][half], make_float2(-r[2].x, -r[2].y)));
                            // (a key that nobody sees may hold anything)
                            if (!clear) mask(dp[j][half], hide >> (4 * j + 2 * half), 0.0f);
                        }
                    }
                    accumulate<kExact>(dv[hh], s, so, st, lanes);
                    accumulate<kExact>(dk[hh], dp, sq, st, lanes);
                }
            }
            __syncthreads();
            tile = ahead;
            stage ^= 1;
        }
    }
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        store_rows(a.dk, k0, in.H, h + hh, dk[hh], in.scale, on0, on1, t);
        store_rows(a.dv, k0, in.H, h + hh, dv[hh], 1.0f, on0, on1, t);
    }
    __syncthreads();
    return !kFar && sm.far;
}

// (not inlined: the registers are for the walks that are taken)
template <int HP, bool kBias, bool kGroups, bool kGrad, bool kExact>
__device__ __noinline__ void far_keys(BackwardSmem<HP>& sm, const BackwardArgs& a, int id, int split)
{
    walk_keys<HP, kBias, kGroups, kGrad, kExact, true>(sm, a, id, split);
}

template <int HP, bool kBias, bool kGroups, bool kExact>
__device__ __noinline__ void far_queries(BackwardSmem<HP>& sm, const BackwardArgs& a, int id)
{
    walk_queries<HP, kBias, kGroups, kExact, true>(sm, a, id);
}

template <int HP, bool kBias, bool kGroups>
__global__ void __launch_bounds__(kAttnThreads, kDotBlocks)
    attention_dots_kernel(const __grid_constant__ BackwardArgs a)
{
    __shared__ BackwardSmem<HP> sm;
    const int id = blockIdx.x / a.splits, split = blockIdx.x - id * a.splits;
    if (walk_keys<HP, kBias, kGroups, false, false, false>(sm, a, id, split))
        far_keys<HP, kBias, kGroups, false, false>(sm, a, id, split);
}

template <bool kBias, bool kGroups, bool kExact>
__global__ void __launch_bounds__(kAttnThreads, kBlocks)
    attention_grad_kernel(const __grid_constant__ BackwardArgs a)
{
    __shared__ BackwardSmem<1> sm;
    const int keys = a.k_tiles * a.in.H * a.in.B;  // the longer ones first
    const int id = blockIdx.x;
    if (id < keys) {
        if (walk_queries<1, kBias, kGroups, kExact, false>(sm, a, id))
            far_queries<1, kBias, kGroups, kExact>(sm, a, id);
    } else {
        if (walk_keys<1, kBias, kGroups, true, kExact, false>(sm, a, id - keys, 0))
            far_keys<1, kBias, kGroups, true, kExact>(sm, a, id - keys, 0);
    }
}

template <bool kGroups>
cudaError_t run(const BackwardArgs& a, const Plan& plan, bool bias, cudaStream_t s)
{
    const int64_t items = (int64_t)a.in.B * a.in.H;
    cudaError_t e = cudaSuccess;
    if (a.in.Nq > 0) {
        const unsigned ctas = (unsigned)(items / plan.heads * a.q_tiles * a.splits);
        const auto kernel = plan.heads == 2 ? attention_dots_kernel<2, true, kGroups>
                            : bias          ? attention_dots_kernel<1, true, kGroups>
                                            : attention_dots_kernel<1, false, kGroups>;
        e = launch_clusters(kernel, a.splits, dim3(ctas), dim3(kAttnThreads), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    const unsigned ctas = (unsigned)(items * (a.q_tiles + a.k_tiles));
    // (few rows on one side: a gradient of the other is made of few terms)
    const bool exact = exact_of((int64_t)a.in.B * a.in.H * std::min(a.in.Nq, a.in.Nk));
    const auto grads = bias ? (exact ? attention_grad_kernel<true, kGroups, true>
                                     : attention_grad_kernel<true, kGroups, false>)
                            : (exact ? attention_grad_kernel<false, kGroups, true>
                                     : attention_grad_kernel<false, kGroups, false>);
    grads<<<ctas, kAttnThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn
}  // namespace msda

using namespace msda;
using namespace msda::attn;

extern "C" size_t msda_query_attention_backward_workspace_size(const msda_attention_t* p)
{
    if (p == nullptr || p->B <= 0 || p->Nq <= 0 || p->H < 1) return 0;
    return 3 * sizeof(float) * (size_t)p->B * p->H * p->Nq;
}

extern "C" msda_status_t msda_query_attention_backward(const msda_attention_t* p, const float* lse,
                                                       const void* grad_out, void* grad_q,
                                                       void* grad_k, void* grad_v,
                                                       float* grad_tau, void* workspace,
                                                       size_t workspace_bytes,
                                                       msda_stream_t stream)
{
    bool empty = false;
    const msda_status_t st = check_inputs(p, empty);
    if (st != MSDA_OK) return st;
    if (p->B == 0 || (p->Nq == 0 && p->Nk == 0)) return api_ok();
    const auto bad = [](const char* m) { return api_fail(MSDA_ERR_INVALID_ARG, m); };
    if (p->Nq > 0) {
        if (lse == nullptr || (uintptr_t)lse % 4) return bad("lse is null or not 4-byte aligned");
        if (grad_out == nullptr || (uintptr_t)grad_out % 16)
            return bad("grad_out is null or not 16-byte aligned");
        if (grad_q == nullptr || (uintptr_t)grad_q % 16)
            return bad("grad_q is null or not 16-byte aligned");
        if (p->tau != nullptr && (grad_tau == nullptr || (uintptr_t)grad_tau % 4))
            return bad("grad_tau is null or not 4-byte aligned");
        if (p->tau == nullptr && grad_tau != nullptr) return bad("grad_tau without tau");
    }
    if (p->Nk > 0 && (grad_k == nullptr || grad_v == nullptr || (uintptr_t)grad_k % 16 ||
                      (uintptr_t)grad_v % 16))
        return bad("grad_k or grad_v is null or not 16-byte aligned");
    const size_t rows_q = (size_t)p->B * p->Nq * p->H, rows_k = (size_t)p->B * p->Nk * p->H;
    if (touches_inputs(p, grad_q, rows_q * kDim * 2) || touches_inputs(p, grad_k, rows_k * kDim * 2) ||
        touches_inputs(p, grad_v, rows_k * kDim * 2) || touches_inputs(p, grad_tau, rows_q * 4))
        return bad("a gradient overlaps q, k or v");
    const msda_status_t ws = check_workspace(workspace, workspace_bytes,
                                             msda_query_attention_backward_workspace_size(p));
    if (ws != MSDA_OK) return ws;
    BackwardArgs a;
    a.in = inputs_of(*p);
    a.go = static_cast<const __nv_bfloat16*>(grad_out);
    a.lse = lse;
    a.dq = static_cast<__nv_bfloat16*>(grad_q);
    a.dk = static_cast<__nv_bfloat16*>(grad_k);
    a.dv = static_cast<__nv_bfloat16*>(grad_v);
    a.dtau = grad_tau;
    const Plan plan = plan_of(p->B, p->Nq, p->Nk, p->H, p->tau != nullptr,
                              p->q_group || p->k_group, kDotBlocks);
    a.rows = static_cast<float*>(workspace);
    a.splits = plan.splits;
    a.split_tiles = plan.split_tiles;
    a.q_tiles = (p->Nq + kTile - 1) / kTile;
    a.k_tiles = (p->Nk + kTile - 1) / kTile;
    const cudaStream_t s = (cudaStream_t)stream;
    const bool bias = p->tau != nullptr;
    const cudaError_t e = p->q_group || p->k_group ? run<true>(a, plan, bias, s)
                                                   : run<false>(a, plan, bias, s);
    return api_cuda(e, "msda_query_attention_backward");
}
