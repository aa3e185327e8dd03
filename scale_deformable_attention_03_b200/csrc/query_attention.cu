// msda_query_attention: attention among object queries with a distance bias
// and group masks (forward).
//   s_ij = scale q_i . k_j - tau_i |p_i - p_j|,  out_i = sum_j softmax(s)_ij v_j
// One pass over the keys with the running maximum and sum of the softmax, in
// the base-2 logarithm's units.  A CTA takes 64 queries of one or (with the
// bias) two heads, so that a distance serves both; its keys come in tiles of
// 64 through a double buffer of asynchronous copies.  Tiles that no query of
// the CTA sees are skipped, tiles without a masked pair take no comparison.
// Where the queries do not fill the GPU the keys are split over CTAs, whose
// sums a second kernel joins.
//
// Bound by the exponentials (one per score) and square roots (one per pair of
// points and two heads) at 16 per clock and SM, and by the issue of about 14
// instructions per score.
#include <algorithm>

#include "query_attention.cuh"

namespace msda {
namespace attn {
namespace {

constexpr int kSms = 148;
constexpr int kMaxSplits = 64;

struct ForwardArgs {
    Inputs in;
    __nv_bfloat16* out;
    float* lse;
    // split keys: per split [B, H, Nq, 32] sums and [B, H, Nq] (maximum, sum)
    float* part;
    float2* part_ml;
    int splits, split_tiles, q_tiles;
};

template <int HP>
struct ForwardSmem {
    alignas(128) unsigned char k[2][HP * kTileBytes];
    alignas(128) unsigned char v[2][HP * kTileBytes];
    float2 pos[2][kTile];
    int32_t group[2][kTile];
    TileBits bits;
};

template <int HP, bool kBias>
__device__ __forceinline__ void load_keys(ForwardSmem<HP>& sm, int stage, const Inputs& in, int b,
                                          int h, int tile)
{
    const int r0 = tile * kTile;
    const uint32_t sk = smem_addr(sm.k[stage]), sv = smem_addr(sm.v[stage]);
#pragma unroll
    for (int i = 0; i < 2 * HP; ++i) {
        const int id = i * kAttnThreads + (int)threadIdx.x;
        const int c = id % (4 * HP), row = id / (4 * HP);
        const int64_t key = (int64_t)b * in.Nk + r0 + row;
        bool on = r0 + row < in.Nk;
        // what padding rows hold must not meet a weight of zero
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

template <int HP, bool kBias>
__global__ void __launch_bounds__(kAttnThreads) attention_forward_kernel(const ForwardArgs a)
{
    __shared__ ForwardSmem<HP> sm;
    const Inputs& in = a.in;
    int id = blockIdx.x;
    const int qt = id % a.q_tiles;
    id /= a.q_tiles;
    const int hg = id % (in.H / HP);
    id /= in.H / HP;
    const int b = id % in.B, split = id / in.B;
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
    float2 p0{}, p1{};
    float tau0[HP] = {}, tau1[HP] = {};
    if constexpr (kBias) {
        if (on0) p0 = __ldg(in.qp + q0);
        if (on1) p1 = __ldg(in.qp + q0 + 8);
#pragma unroll
        for (int hh = 0; hh < HP; ++hh) {
            if (on0) tau0[hh] = __ldg(in.tau + q0 * in.H + h + hh) * kLog2e;
            if (on1) tau1[hh] = __ldg(in.tau + (q0 + 8) * in.H + h + hh) * kLog2e;
        }
    }
    int g0 = 0, g1 = 0;
    GroupRange own{0, 0, true, true, true};
    if (in.qg != nullptr) {
        g0 = on0 ? __ldg(in.qg + q0) : -1;
        g1 = on1 ? __ldg(in.qg + q0 + 8) : -1;
        own = warp_range(in.qg, (int64_t)b * in.Nq + qt * kRows, min(kRows, in.Nq - qt * kRows));
    }
    const float scale = in.scale * kLog2e;

    float o[HP][4][4] = {}, m0[HP], m1[HP], l0[HP] = {}, l1[HP] = {};
#pragma unroll
    for (int hh = 0; hh < HP; ++hh) m0[hh] = m1[hh] = -INFINITY;

    const int tiles = (in.Nk + kTile - 1) / kTile;
    const int begin = split * a.split_tiles, last = min(tiles, begin + a.split_tiles);
    for (int first = begin; first < last; first += kScan) {
        scan_tiles<false>(sm.bits, own, true, in.kg, (int64_t)b * in.Nk, in.Nk, first, last);
        int tile = next_tile(sm.bits, first, first, last), stage = 0;
        if (tile < last) load_keys<HP, kBias>(sm, stage, in, b, h, tile);
        while (tile < last) {
            const int ahead = next_tile(sm.bits, tile + 1, first, last);
            if (ahead < last) {
                load_keys<HP, kBias>(sm, stage ^ 1, in, b, h, ahead);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            __syncthreads();
            const bool clear = (sm.bits.clear[(tile - first) >> 5] >> ((tile - first) & 31)) & 1;
            float dist[8][4];
            if constexpr (kBias) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 pk =
                        *reinterpret_cast<const float4*>(&sm.pos[stage][8 * j + 2 * t]);
                    dist[j][0] = distance(p0, pk.x, pk.y);
                    dist[j][1] = distance(p0, pk.z, pk.w);
                    dist[j][2] = distance(p1, pk.x, pk.y);
                    dist[j][3] = distance(p1, pk.z, pk.w);
                }
            }
            uint32_t hide = 0;  // pairs of this thread that are masked
            if (!clear) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int at = 8 * j + 2 * t + c;
                        const bool in_range = tile * kTile + at < in.Nk;
                        const int kg = in.kg != nullptr ? sm.group[stage][at] : 0;
                        hide |= (uint32_t)!(in_range && sees(g0, kg)) << (4 * j + c);
                        hide |= (uint32_t)!(in_range && sees(g1, kg)) << (4 * j + 2 + c);
                    }
                }
            }
#pragma unroll
            for (int hh = 0; hh < HP; ++hh) {
                const uint32_t sk = smem_addr(sm.k[stage]) + hh * kTileBytes;
                const uint32_t sv = smem_addr(sm.v[stage]) + hh * kTileBytes;
                float s[8][4] = {};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t r[4];
                    load_cols(r, sk, j, lane);
                    mma(s[j], qf[hh], r[0], r[1]);
                    mma(s[j], qf[hh] + 4, r[2], r[3]);
                }
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        s[j][c] *= scale;
                        if constexpr (kBias)
                            s[j][c] = fmaf(c < 2 ? -tau0[hh] : -tau1[hh], dist[j][c], s[j][c]);
                    }
                }
                if (!clear) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if ((hide >> (4 * j + c)) & 1) s[j][c] = -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    t0 = fmaxf(t0, fmaxf(s[j][0], s[j][1]));
                    t1 = fmaxf(t1, fmaxf(s[j][2], s[j][3]));
                }
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
                const float n0 = fmaxf(m0[hh], t0), n1 = fmaxf(m1[hh], t1);
                // a row that has seen nothing yet stays at weight zero
                const float b0 = n0 == -INFINITY ? 0.0f : n0, b1 = n1 == -INFINITY ? 0.0f : n1;
                const float f0 = exp2_approx(m0[hh] - b0), f1 = exp2_approx(m1[hh] - b1);
                m0[hh] = n0;
                m1[hh] = n1;
                float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s[j][0] = exp2_approx(s[j][0] - b0);
                    s[j][1] = exp2_approx(s[j][1] - b0);
                    s[j][2] = exp2_approx(s[j][2] - b1);
                    s[j][3] = exp2_approx(s[j][3] - b1);
                    a0 += s[j][0] + s[j][1];
                    a1 += s[j][2] + s[j][3];
                }
                l0[hh] = fmaf(l0[hh], f0, a0);
                l1[hh] = fmaf(l1[hh], f1, a1);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    o[hh][d][0] *= f0;
                    o[hh][d][1] *= f0;
                    o[hh][d][2] *= f1;
                    o[hh][d][3] *= f1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the weights in bf16: the matrix instruction's type, v's own; 2^-8 of
                    // each at most, what out's own rounding may be
                    const uint32_t pf[4] = {pack_bf16(s[2 * k][0], s[2 * k][1]),
                                            pack_bf16(s[2 * k][2], s[2 * k][3]),
                                            pack_bf16(s[2 * k + 1][0], s[2 * k + 1][1]),
                                            pack_bf16(s[2 * k + 1][2], s[2 * k + 1][3])};
#pragma unroll
                    for (int d = 0; d < 4; d += 2) {
                        uint32_t r[4];
                        load_sum(r, sv, k, d, lane);
                        mma(o[hh][d], pf, r[0], r[1]);
                        mma(o[hh][d + 1], pf, r[2], r[3]);
                    }
                }
            }
            __syncthreads();
            tile = ahead;
            stage ^= 1;
        }
    }

#pragma unroll
    for (int hh = 0; hh < HP; ++hh) {
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            l0[hh] += __shfl_xor_sync(0xffffffffu, l0[hh], x);
            l1[hh] += __shfl_xor_sync(0xffffffffu, l1[hh], x);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (!(half ? on1 : on0)) continue;
            const int q = row + 8 * half;
            const float l = half ? l1[hh] : l0[hh], m = half ? m1[hh] : m0[hh];
            // a padding query saw the keys of group 0: it is left out here
            const bool dead = l == 0.0f || (half ? g1 : g0) < 0;
            const int64_t bhq = ((int64_t)b * in.H + h + hh) * in.Nq + q;
            if (a.splits == 1) {
                const float w = dead ? 0.0f : 1.0f / l;
                uint32_t* dst = reinterpret_cast<uint32_t*>(
                    a.out + (((int64_t)b * in.Nq + q) * in.H + h + hh) * kDim);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    dst[4 * d + t] = dead ? 0u : pack_bf16(o[hh][d][2 * half] * w,
                                                           o[hh][d][2 * half + 1] * w);
                if (a.lse != nullptr && t == 0)
                    a.lse[bhq] = dead ? -INFINITY : (m + log2f(l)) * kLn2;
            } else {
                const int64_t at = (int64_t)split * in.B * in.H * in.Nq + bhq;
                float2* dst = reinterpret_cast<float2*>(a.part + at * kDim);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    dst[4 * d + t] = make_float2(o[hh][d][2 * half], o[hh][d][2 * half + 1]);
                if (t == 0) a.part_ml[at] = dead ? make_float2(-INFINITY, 0.0f) : make_float2(m, l);
            }
        }
    }
}

// Eight threads per (item, head, query), four channels each, over the splits.
__global__ void __launch_bounds__(256) attention_join_kernel(const ForwardArgs a)
{
    const Inputs& in = a.in;
    const int64_t n = (int64_t)in.B * in.H * in.Nq;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3;
    const int c = threadIdx.x & 7;
    pdl_wait();
    if (i >= n) return;
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[s * n + i].x);
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < a.splits; ++s) {
        const float2 ml = a.part_ml[s * n + i];
        if (ml.y == 0.0f) continue;
        const float w = exp2_approx(ml.x - m);
        const float4 v = reinterpret_cast<const float4*>(a.part)[(s * n + i) * 8 + c];
        l = fmaf(w, ml.y, l);
        o.x = fmaf(w, v.x, o.x);
        o.y = fmaf(w, v.y, o.y);
        o.z = fmaf(w, v.z, o.z);
        o.w = fmaf(w, v.w, o.w);
    }
    const float w = l == 0.0f ? 0.0f : 1.0f / l;
    const int q = (int)(i % in.Nq);
    const int64_t bh = i / in.Nq;
    const int64_t at = ((bh / in.H * in.Nq + q) * in.H + bh % in.H) * kDim + c * 4;
    *reinterpret_cast<uint2*>(a.out + at) =
        make_uint2(pack_bf16(o.x * w, o.y * w), pack_bf16(o.z * w, o.w * w));
    if (a.lse != nullptr && c == 0) a.lse[i] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

struct Plan {
    int q_tiles, splits, split_tiles;
};

// Two CTAs per SM keep it busy; below that the keys are split, down to two
// tiles per CTA (a join costs about what two tiles do).
Plan plan_of(int B, int Nq, int Nk, int H)
{
    Plan p;
    p.q_tiles = (Nq + kRows - 1) / kRows;
    const int64_t ctas = (int64_t)p.q_tiles * B * H;
    const int tiles = (Nk + kTile - 1) / kTile;
    p.splits = 1;
    if (ctas < 2 * kSms)
        p.splits = (int)std::max<int64_t>(
            1, std::min<int64_t>({(2 * kSms + ctas - 1) / ctas, (tiles + 1) / 2, kMaxSplits}));
    p.split_tiles = std::max(1, (tiles + p.splits - 1) / p.splits);
    p.splits = std::max(1, (tiles + p.split_tiles - 1) / p.split_tiles);
    return p;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

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
    if (!std::isfinite(p->scale))
        return api_failf(MSDA_ERR_INVALID_ARG, "scale = %g must be finite", (double)p->scale);
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

extern "C" size_t msda_query_attention_workspace_size(const msda_attention_t* p)
{
    if (p == nullptr || p->B <= 0 || p->Nq <= 0 || p->Nk <= 0 || p->H < 1) return 0;
    const Plan plan = plan_of(p->B, p->Nq, p->Nk, p->H);
    if (plan.splits == 1) return 0;
    const size_t rows = (size_t)plan.splits * p->B * p->H * p->Nq;
    return up256(rows * kDim * sizeof(float)) + up256(rows * sizeof(float2));
}

extern "C" msda_status_t msda_query_attention(const msda_attention_t* p, void* out, float* lse,
                                              void* workspace, size_t workspace_bytes,
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
    const size_t need = msda_query_attention_workspace_size(p);
    const msda_status_t ws = check_workspace(workspace, workspace_bytes, need);
    if (ws != MSDA_OK) return ws;
    const cudaStream_t s = (cudaStream_t)stream;
    ForwardArgs a;
    a.in = inputs_of(*p);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    const Plan plan = plan_of(p->B, p->Nq, p->Nk, p->H);
    a.q_tiles = plan.q_tiles;
    a.splits = plan.splits;
    a.split_tiles = plan.split_tiles;
    const size_t rows = (size_t)plan.splits * p->B * p->H * p->Nq;
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                          up256(rows * kDim * sizeof(float)));
    const bool bias = p->tau != nullptr;
    const int64_t ctas = (int64_t)plan.q_tiles * p->B * p->H * plan.splits;
    // two heads per CTA share the distances, where that still fills the GPU
    const bool pair = bias && p->H % 2 == 0 && ctas >= 8 * kSms;
    cudaError_t e;
    if (pair)
        attention_forward_kernel<2, true><<<(unsigned)(ctas / 2), kAttnThreads, 0, s>>>(a);
    else if (bias)
        attention_forward_kernel<1, true><<<(unsigned)ctas, kAttnThreads, 0, s>>>(a);
    else
        attention_forward_kernel<1, false><<<(unsigned)ctas, kAttnThreads, 0, s>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess && plan.splits > 1) {
        const int64_t n = (int64_t)p->B * p->H * p->Nq;
        e = launch_pdl(attention_join_kernel, dim3((unsigned)((n * 8 + 255) / 256)), dim3(256), 0,
                       s, a);
    }
    return api_cuda(e, "msda_query_attention");
}
