// msda_query_attention_backward: with p_ij = exp(s_ij - lse_i),
// dp_ij = do_i . v_j, D_i = sum_j p_ij dp_ij and ds_ij = p_ij (dp_ij - D_i):
//   dq_i = scale sum_j ds_ij k_j,  dtau_i = -sum_j ds_ij |p_i - p_j|
//   dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
// Two kernels, one per side, so that every sum has one owner and no atomic is
// needed.  The queries' kernel walks the keys twice: first for D, then for dq
// and dtau.  D is formed from the same p and dp that ds uses (not from the
// rounded output of the forward): ds is then exact where one key takes all the
// weight, and dtau, an fp32 sum of it, keeps fp32's precision.  It leaves
// (lse, tau, D) per head and query for the keys' kernel, which walks the
// queries once.
//
// Bound like the forward by instruction issue and the exponentials (three per
// pair, and three square roots per pair of points and CTA).
#include <algorithm>

#include "query_attention.cuh"

namespace msda {
namespace attn {
namespace {

constexpr int kHalf = 32;  // columns per step: scores, dp and distances in registers

struct BackwardArgs {
    Inputs in;
    const __nv_bfloat16* go;  // [B, Nq, H * 32]
    const float* lse;
    __nv_bfloat16 *dq, *dk, *dv;
    float* dtau;
    float4* rows;  // [B, H, Nq]: lse and tau in units of log 2, D
    int q_tiles, k_tiles;
};

template <int HP>
struct BackwardSmem {
    alignas(128) unsigned char a[2][HP * kTileBytes];  // keys, or queries
    alignas(128) unsigned char b[2][HP * kTileBytes];  // values, or the output's gradient
    float4 rows[2][HP][kTile];                         // of the queries (keys' kernel)
    float2 pos[2][kTile];
    int32_t group[2][kTile];
    TileBits bits;
};

template <int HP, bool kBias>
__device__ __forceinline__ void load_keys(BackwardSmem<HP>& sm, int stage, const Inputs& in, int b,
                                          int h, int tile)
{
    const int r0 = tile * kTile;
    const uint32_t sk = smem_addr(sm.a[stage]), sv = smem_addr(sm.b[stage]);
#pragma unroll
    for (int i = 0; i < 2 * HP; ++i) {
        const int id = i * kAttnThreads + (int)threadIdx.x;
        const int c = id % (4 * HP), row = id / (4 * HP);
        const int64_t key = (int64_t)b * in.Nk + r0 + row;
        bool on = r0 + row < in.Nk;
        if (on && in.kg != nullptr) on = __ldg(in.kg + key) >= 0;
        const uint32_t dst = (c / 4) * kTileBytes + tile_at(row, c % 4);
        cp_async<16>(sk + dst, on ? in.k + key * in.ldk + h * kDim + c * 8 : in.k, on);
        cp_async<16>(sv + dst, on ? in.v + key * in.ldv + h * kDim + c * 8 : in.v, on);
    }
    if (threadIdx.x < kTile) {
        const int row = r0 + threadIdx.x;
        const int64_t key = (int64_t)b * in.Nk + row;
        const bool on = row < in.Nk;
        if constexpr (kBias)
            cp_async<8>(smem_addr(&sm.pos[stage][threadIdx.x]), on ? in.kp + key : in.kp, on);
        if (in.kg != nullptr)
            cp_async<4>(smem_addr(&sm.group[stage][threadIdx.x]), on ? in.kg + key : in.kg, on);
    }
    cp_commit();
}

// Queries that see nothing (lse = -infinity) read as zero: whatever they and
// their gradient hold, p = 0 then has nothing to meet.
template <int HP, bool kBias>
__device__ __forceinline__ void load_queries(BackwardSmem<HP>& sm, int stage,
                                             const BackwardArgs& a, int b, int h, int tile)
{
    const Inputs& in = a.in;
    const int r0 = tile * kTile;
    const uint32_t sq = smem_addr(sm.a[stage]), so = smem_addr(sm.b[stage]);
#pragma unroll
    for (int i = 0; i < 2 * HP; ++i) {
        const int id = i * kAttnThreads + (int)threadIdx.x;
        const int c = id % (4 * HP), row = id / (4 * HP);
        const int64_t q = (int64_t)b * in.Nq + r0 + row;
        bool on = r0 + row < in.Nq;
        if (on)
            on = __ldg(a.lse + ((int64_t)b * in.H + h + c / 4) * in.Nq + r0 + row) != -INFINITY;
        const uint32_t dst = (c / 4) * kTileBytes + tile_at(row, c % 4);
        cp_async<16>(sq + dst, on ? in.q + q * in.ldq + h * kDim + c * 8 : in.q, on);
        cp_async<16>(so + dst, on ? a.go + (q * in.H + h) * kDim + c * 8 : a.go, on);
    }
    for (int i = threadIdx.x; i < HP * kTile; i += kAttnThreads) {
        const int hh = i / kTile, row = r0 + i % kTile;
        const bool on = row < in.Nq;
        const float4* src = a.rows + ((int64_t)b * in.H + h + hh) * in.Nq + row;
        cp_async<16>(smem_addr(&sm.rows[stage][hh][i % kTile]), on ? src : a.rows, on);
    }
    if (threadIdx.x < kTile) {
        const int row = r0 + threadIdx.x;
        const int64_t q = (int64_t)b * in.Nq + row;
        const bool on = row < in.Nq;
        if constexpr (kBias)
            cp_async<8>(smem_addr(&sm.pos[stage][threadIdx.x]), on ? in.qp + q : in.qp, on);
        if (in.qg != nullptr)
            cp_async<4>(smem_addr(&sm.group[stage][threadIdx.x]), on ? in.qg + q : in.qg, on);
    }
    cp_commit();
}

// A step's 16 x 32 products of a warp's rows with the tile's rows 32s..32s+31.
__device__ __forceinline__ void products(float (&c)[4][4], const uint32_t (&f)[8], uint32_t tile,
                                         int s, int lane)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t r[4];
        load_cols(r, tile, 4 * s + j, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[j][i] = 0.0f;
        mma(c[j], f, r[0], r[1]);
        mma(c[j], f + 4, r[2], r[3]);
    }
}

// acc += w (16 x 32, rounded to bf16: the matrix instruction's type) times the
// tile's rows 32s .. 32s + 31.
__device__ __forceinline__ void accumulate(float (&acc)[4][4], const float (&w)[4][4],
                                           uint32_t tile, int s, int lane)
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t f[4] = {pack_bf16(w[2 * k][0], w[2 * k][1]),
                               pack_bf16(w[2 * k][2], w[2 * k][3]),
                               pack_bf16(w[2 * k + 1][0], w[2 * k + 1][1]),
                               pack_bf16(w[2 * k + 1][2], w[2 * k + 1][3])};
#pragma unroll
        for (int d = 0; d < 4; d += 2) {
            uint32_t r[4];
            load_sum(r, tile, 2 * s + k, d, lane);
            mma(acc[d], f, r[0], r[1]);
            mma(acc[d + 1], f, r[2], r[3]);
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

__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <int HP, bool kBias>
__global__ void __launch_bounds__(kAttnThreads) attention_grad_queries_kernel(const BackwardArgs a)
{
    __shared__ BackwardSmem<HP> sm;
    const Inputs& in = a.in;
    int id = blockIdx.x;
    const int qt = id % a.q_tiles;
    id /= a.q_tiles;
    const int h = id % (in.H / HP) * HP, b = id / (in.H / HP);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int row = qt * kRows + warp * 16 + g;
    const bool on0 = row < in.Nq, on1 = row + 8 < in.Nq;
    const int64_t q0 = (int64_t)b * in.Nq + row;

    uint32_t qf[HP][8], of[HP][8];
    float e0[HP], e1[HP], tau0[HP] = {}, tau1[HP] = {};
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        const int64_t i = ((int64_t)b * in.H + h + hh) * in.Nq + row;
        e0[hh] = on0 ? __ldg(a.lse + i) : -INFINITY;
        e1[hh] = on1 ? __ldg(a.lse + i + 8) : -INFINITY;
        const bool live0 = e0[hh] != -INFINITY, live1 = e1[hh] != -INFINITY;
        load_rows(qf[hh], in.q + (int64_t)b * in.Nq * in.ldq + (h + hh) * kDim, in.ldq, row, live0,
                  live1, t);
        load_rows(of[hh], a.go + ((int64_t)b * in.Nq * in.H + h + hh) * kDim,
                  (int64_t)in.H * kDim, row, live0, live1, t);
        // a row that sees nothing: weight exp2(s - infinity) = 0 everywhere
        e0[hh] = live0 ? e0[hh] * kLog2e : INFINITY;
        e1[hh] = live1 ? e1[hh] * kLog2e : INFINITY;
        if constexpr (kBias) {
            if (live0) tau0[hh] = __ldg(in.tau + q0 * in.H + h + hh) * kLog2e;
            if (live1) tau1[hh] = __ldg(in.tau + (q0 + 8) * in.H + h + hh) * kLog2e;
        }
    }
    float2 p0{}, p1{};
    if constexpr (kBias) {  // (a row that sees nothing may have any point)
        if (e0[0] != INFINITY) p0 = __ldg(in.qp + q0);
        if (e1[0] != INFINITY) p1 = __ldg(in.qp + q0 + 8);
    }
    int g0 = 0, g1 = 0;
    GroupRange own{0, 0, true, true, true};
    if (in.qg != nullptr) {
        g0 = on0 ? __ldg(in.qg + q0) : -1;
        g1 = on1 ? __ldg(in.qg + q0 + 8) : -1;
        own = warp_range(in.qg, (int64_t)b * in.Nq + qt * kRows, min(kRows, in.Nq - qt * kRows));
    }
    const float scale = in.scale * kLog2e;
    float D0[HP] = {}, D1[HP] = {}, dt0[HP] = {}, dt1[HP] = {}, dq[HP][4][4] = {};

    const int tiles = a.k_tiles;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        for (int first = 0; first < tiles; first += kScan) {
            if (pass == 0 || tiles > kScan)
                scan_tiles<false>(sm.bits, own, true, in.kg, (int64_t)b * in.Nk, in.Nk, first,
                                  tiles);
            int tile = next_tile(sm.bits, first, first, tiles), stage = 0;
            if (tile < tiles) load_keys<HP, kBias>(sm, stage, in, b, h, tile);
            while (tile < tiles) {
                const int ahead = next_tile(sm.bits, tile + 1, first, tiles);
                if (ahead < tiles) {
                    load_keys<HP, kBias>(sm, stage ^ 1, in, b, h, ahead);
                    cp_wait<1>();
                } else {
                    cp_wait<0>();
                }
                __syncthreads();
                const bool clear =
                    (sm.bits.clear[(tile - first) >> 5] >> ((tile - first) & 31)) & 1;
#pragma unroll
                for (int st = 0; st < kTile / kHalf; ++st) {
                    float dist[4][4];
                    uint32_t hide = 0;
                    if constexpr (kBias) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 pk = *reinterpret_cast<const float4*>(
                                &sm.pos[stage][kHalf * st + 8 * j + 2 * t]);
                            dist[j][0] = distance(p0, pk.x, pk.y);
                            dist[j][1] = distance(p0, pk.z, pk.w);
                            dist[j][2] = distance(p1, pk.x, pk.y);
                            dist[j][3] = distance(p1, pk.z, pk.w);
                        }
                    }
                    if (!clear) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int at = kHalf * st + 8 * j + 2 * t + c;
                                const bool in_range = tile * kTile + at < in.Nk;
                                const int kg = in.kg != nullptr ? sm.group[stage][at] : 0;
                                hide |= (uint32_t)!(in_range && sees(g0, kg)) << (4 * j + c);
                                hide |= (uint32_t)!(in_range && sees(g1, kg)) << (4 * j + 2 + c);
                            }
                        }
                        if constexpr (kBias) {  // a masked point may be anything
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if ((hide >> (4 * j + c)) & 1) dist[j][c] = 0.0f;
                        }
                    }
#pragma unroll
                    for (int hh = 0; hh < HP; ++hh) {
                        const uint32_t sk = smem_addr(sm.a[stage]) + hh * kTileBytes;
                        const uint32_t sv = smem_addr(sm.b[stage]) + hh * kTileBytes;
                        float s[4][4], dp[4][4];
                        products(s, qf[hh], sk, st, lane);
                        products(dp, of[hh], sv, st, lane);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                float x = fmaf(s[j][c], scale, c < 2 ? -e0[hh] : -e1[hh]);
                                if constexpr (kBias)
                                    x = fmaf(c < 2 ? -tau0[hh] : -tau1[hh], dist[j][c], x);
                                if ((hide >> (4 * j + c)) & 1) x = -INFINITY;
                                s[j][c] = exp2_approx(x);
                            }
                        }
                        if (pass == 0) {
                            float a0 = 0.0f, a1 = 0.0f;  // a step's own sums, then the total
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                a0 = fmaf(s[j][0], dp[j][0], fmaf(s[j][1], dp[j][1], a0));
                                a1 = fmaf(s[j][2], dp[j][2], fmaf(s[j][3], dp[j][3], a1));
                            }
                            D0[hh] += a0;
                            D1[hh] += a1;
                        } else {
                            float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    s[j][c] *= dp[j][c] - (c < 2 ? D0[hh] : D1[hh]);
                                    if constexpr (kBias) {
                                        if (c < 2) a0 = fmaf(s[j][c], dist[j][c], a0);
                                        else a1 = fmaf(s[j][c], dist[j][c], a1);
                                    }
                                }
                            }
                            dt0[hh] += a0;
                            dt1[hh] += a1;
                            accumulate(dq[hh], s, sk, st, lane);
                        }
                    }
                }
                __syncthreads();
                tile = ahead;
                stage ^= 1;
            }
        }
        if (pass == 0) {
#pragma unroll
            for (int hh = 0; hh < HP; ++hh) {
                D0[hh] = quad_sum(D0[hh]);
                D1[hh] = quad_sum(D1[hh]);
                const int64_t i = ((int64_t)b * in.H + h + hh) * in.Nq + row;
                if (t == 0 && on0) a.rows[i] = make_float4(e0[hh], tau0[hh], D0[hh], 0.0f);
                if (t == 0 && on1) a.rows[i + 8] = make_float4(e1[hh], tau1[hh], D1[hh], 0.0f);
            }
        }
    }
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        store_rows(a.dq, q0, in.H, h + hh, dq[hh], in.scale, on0, on1, t);
        if constexpr (kBias) {
            dt0[hh] = quad_sum(dt0[hh]);
            dt1[hh] = quad_sum(dt1[hh]);
            if (t == 0 && on0) a.dtau[q0 * in.H + h + hh] = -dt0[hh];
            if (t == 0 && on1) a.dtau[(q0 + 8) * in.H + h + hh] = -dt1[hh];
        }
    }
}

template <int HP, bool kBias>
__global__ void __launch_bounds__(kAttnThreads) attention_grad_keys_kernel(const BackwardArgs a)
{
    __shared__ BackwardSmem<HP> sm;
    const Inputs& in = a.in;
    int id = blockIdx.x;
    const int kt = id % a.k_tiles;
    id /= a.k_tiles;
    const int h = id % (in.H / HP) * HP, b = id / (in.H / HP);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int row = kt * kRows + warp * 16 + g;
    const bool on0 = row < in.Nk, on1 = row + 8 < in.Nk;
    const int64_t k0 = (int64_t)b * in.Nk + row;
    int g0 = on0 ? 0 : -1, g1 = on1 ? 0 : -1;
    GroupRange own{0, 0, true, true, true};
    const int own_rows = min(kRows, in.Nk - kt * kRows);
    if (in.kg != nullptr) {
        if (on0) g0 = __ldg(in.kg + k0);
        if (on1) g1 = __ldg(in.kg + k0 + 8);
        own = warp_range(in.kg, (int64_t)b * in.Nk + kt * kRows, own_rows);
    }
    uint32_t kf[HP][8], vf[HP][8];
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
        load_rows(kf[hh], in.k + (int64_t)b * in.Nk * in.ldk + (h + hh) * kDim, in.ldk, row,
                  g0 >= 0, g1 >= 0, t);
        load_rows(vf[hh], in.v + (int64_t)b * in.Nk * in.ldv + (h + hh) * kDim, in.ldv, row,
                  g0 >= 0, g1 >= 0, t);
    }
    float2 p0{}, p1{};
    if constexpr (kBias) {
        if (g0 >= 0) p0 = __ldg(in.kp + k0);
        if (g1 >= 0) p1 = __ldg(in.kp + k0 + 8);
    }
    const float scale = in.scale * kLog2e;
    float dk[HP][4][4] = {}, dv[HP][4][4] = {};

    const int tiles = a.q_tiles;
    for (int first = 0; first < tiles; first += kScan) {
        scan_tiles<true>(sm.bits, own, own_rows == kRows, in.qg, (int64_t)b * in.Nq, in.Nq, first,
                         tiles);
        int tile = next_tile(sm.bits, first, first, tiles), stage = 0;
        if (tile < tiles) load_queries<HP, kBias>(sm, stage, a, b, h, tile);
        while (tile < tiles) {
            const int ahead = next_tile(sm.bits, tile + 1, first, tiles);
            if (ahead < tiles) {
                load_queries<HP, kBias>(sm, stage ^ 1, a, b, h, ahead);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
            const bool clear = (sm.bits.clear[(tile - first) >> 5] >> ((tile - first) & 31)) & 1;
#pragma unroll
            for (int st = 0; st < kTile / kHalf; ++st) {
                float dist[4][4];
                uint32_t hide = 0;
                if constexpr (kBias) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 pq = *reinterpret_cast<const float4*>(
                            &sm.pos[stage][kHalf * st + 8 * j + 2 * t]);
                        dist[j][0] = distance(p0, pq.x, pq.y);
                        dist[j][1] = distance(p0, pq.z, pq.w);
                        dist[j][2] = distance(p1, pq.x, pq.y);
                        dist[j][3] = distance(p1, pq.z, pq.w);
                    }
                }
                if (!clear) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int at = kHalf * st + 8 * j + 2 * t + c;
                            const bool in_range = tile * kTile + at < in.Nq;
                            const int qg = in.qg != nullptr ? sm.group[stage][at] : 0;
                            hide |= (uint32_t)!(in_range && sees(qg, g0)) << (4 * j + c);
                            hide |= (uint32_t)!(in_range && sees(qg, g1)) << (4 * j + 2 + c);
                        }
                    }
                }
#pragma unroll
                for (int hh = 0; hh < HP; ++hh) {
                    const uint32_t sq = smem_addr(sm.a[stage]) + hh * kTileBytes;
                    const uint32_t so = smem_addr(sm.b[stage]) + hh * kTileBytes;
                    float s[4][4], dp[4][4];
                    products(s, kf[hh], sq, st, lane);
                    products(dp, vf[hh], so, st, lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float4 r = sm.rows[stage][hh][kHalf * st + 8 * j + 2 * t + c];
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int i = 2 * half + c;
                                float x = fmaf(s[j][i], scale, -r.x);
                                if constexpr (kBias) x = fmaf(-r.y, dist[j][i], x);
                                if ((hide >> (4 * j + i)) & 1) x = -INFINITY;
                                s[j][i] = exp2_approx(x);
                                dp[j][i] = s[j][i] * (dp[j][i] - r.z);
                            }
                        }
                    }
                    accumulate(dv[hh], s, so, st, lane);
                    accumulate(dk[hh], dp, sq, st, lane);
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
}

template <int HP, bool kBias>
cudaError_t run(const BackwardArgs& a, cudaStream_t s)
{
    const int64_t per = (int64_t)a.in.B * (a.in.H / HP);
    if (a.in.Nq > 0) {
        attention_grad_queries_kernel<HP, kBias>
            <<<(unsigned)(per * a.q_tiles), kAttnThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.in.Nk > 0)
        attention_grad_keys_kernel<HP, kBias>
            <<<(unsigned)(per * a.k_tiles), kAttnThreads, 0, s>>>(a);
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
    return sizeof(float4) * (size_t)p->B * p->H * p->Nq;
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
    a.rows = static_cast<float4*>(workspace);
    a.q_tiles = (p->Nq + kTile - 1) / kTile;
    a.k_tiles = (p->Nk + kTile - 1) / kTile;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = p->tau != nullptr ? run<1, true>(a, s) : run<1, false>(a, s);
    return api_cuda(e, "msda_query_attention_backward");
}
