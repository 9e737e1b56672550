// gn_common.cuh -- the activations, the elementwise halves and the launch geometry that the
// group norm's forward and backward share.
#pragma once
#include <algorithm>
#include <type_traits>

#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

// 2^x and 1/x in one instruction each (2 and 1 units in the last place; results below 2^-126
// are 0).  The general-range forms of exp and of the quotient take about four times the
// instructions, and the activations are most of what these kernels compute.  An exponential's argument
// is a rounded product here, so exp(-z) is also off by up to |z| 2^-24 of itself: below 2e-6 as far as
// the sigmoid has 2^-40 of its value left.
__device__ __forceinline__ float fast_exp2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float fast_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// The kernels compute on pairs of values: one instruction adds or multiplies both.
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

__device__ __forceinline__ float2 sigmoid2(float2 z)
{
    const float2 u = mul2(z, both(-kLog2e));
    const float2 w = add2(make_float2(fast_exp2(u.x), fast_exp2(u.y)), both(1.f));
    return make_float2(fast_rcp(w.x), fast_rcp(w.y));
}

// Phi(z) and e = exp(-z^2 / 2).  Phi from Abramowitz & Stegun 7.1.26, Handbook of Mathematical
// Functions: erf(x) = 1 - (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + 0.3275911 x), x >= 0,
// to 1.5e-7 (so Phi to 0.75e-7); its exponential is the density's.  With its roundings in fp32 Phi is
// off by up to 3.1e-7, and over z ~ N(0, 1) GELU by 8.5e-8 and its slope by 1.0e-7 of their norms, twice
// what a correctly rounded erf leaves (3.8e-8 and 4.1e-8; for z in [-4, 0] at most 2.1e-7 against
// 0.6e-7): a choice for fewer instructions.  A bf16 result shows nothing of it.
__device__ __forceinline__ float2 normal_cdf2(float2 z, float2& e)
{
    constexpr float c = 0.3275911f * 0.70710678118654752f;
    const float2 t = make_float2(fast_rcp(fmaf(fabsf(z.x), c, 1.f)), fast_rcp(fmaf(fabsf(z.y), c, 1.f)));
    const float2 u = mul2(mul2(z, both(-0.5f * kLog2e)), z);
    e = make_float2(fast_exp2(u.x), fast_exp2(u.y));
    // half of the polynomial: Phi(-|z|) = 0.5 (a1 t + ...) e
    float2 w = fma2(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
    w = fma2(w, t, both(0.5f * 1.421413741f));
    w = fma2(w, t, both(0.5f * -0.284496736f));
    w = fma2(w, t, both(0.5f * 0.254829592f));
    const float2 tail = mul2(mul2(w, t), e);
    return make_float2(z.x < 0.f ? tail.x : 1.f - tail.x, z.y < 0.f ? tail.y : 1.f - tail.y);
}

template <int ACT> __device__ __forceinline__ float2 act_value(float2 z)
{
    if constexpr (ACT == CONV_ACT_RELU)  // NaN stays
        return make_float2(z.x < 0.f ? 0.f : z.x + 0.f, z.y < 0.f ? 0.f : z.y + 0.f);
    if constexpr (ACT == CONV_ACT_SILU) return mul2(z, sigmoid2(z));
    if constexpr (ACT == CONV_ACT_GELU) {
        float2 e;
        return mul2(z, normal_cdf2(z, e));
    }
    return z;
}
template <int ACT> __device__ __forceinline__ float act_value(float z) { return act_value<ACT>(both(z)).x; }

// dz = dy * act'(z); a ReLU that is off passes nothing, whatever dy holds there.
template <int ACT> __device__ __forceinline__ float2 gn_dz(float2 dy, float2 z)
{
    if constexpr (ACT == CONV_ACT_RELU) return make_float2(z.x > 0.f ? dy.x : 0.f, z.y > 0.f ? dy.y : 0.f);
    if constexpr (ACT == CONV_ACT_SILU) {  // p + z p (1 - p)
        const float2 p = sigmoid2(z);
        return mul2(dy, fma2(mul2(p, z), add2(both(1.f), mul2(p, both(-1.f))), p));
    }
    if constexpr (ACT == CONV_ACT_GELU) {
        float2 e;
        const float2 cdf = normal_cdf2(z, e);
        return mul2(dy, fma2(mul2(z, both(0.39894228040143268f)), e, cdf));
    }
    return dy;
}
template <int ACT> __device__ __forceinline__ float gn_dz(float dy, float z) { return gn_dz<ACT>(both(dy), both(z)).x; }

// xhat and z by individually rounded operations (no contraction): the forward and the backward
// then agree on every bit of z, so the backward's ReLU mask is the forward's.
__device__ __forceinline__ float gn_xhat(float x, float mean, float rstd)
{
    return __fmul_rn(__fsub_rn(x, mean), rstd);
}
__device__ __forceinline__ float gn_z(float xhat, float gamma, float beta)
{
    return __fadd_rn(__fmul_rn(xhat, gamma), beta);
}

// a + b that no compiler merges with the product that a is (the pair's addition may be).
__device__ __forceinline__ float2 add2_apart(float2 a, float2 b)
{
    return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// y from d = x - mean, rounded.  The ReLU's forward and backward round z alike, operation by
// operation, so that their masks agree; the smooth activations take rstd * gamma in one.
template <int ACT> __device__ __forceinline__ float2 gn_out(float2 d, float2 rstd, float2 gamma_or_scale, float2 beta)
{
    if constexpr (ACT == CONV_ACT_RELU) return act_value<ACT>(add2_apart(mul2(mul2(d, rstd), gamma_or_scale), beta));
    return act_value<ACT>(fma2(d, gamma_or_scale, beta));
}
// dz from xhat.
template <int ACT> __device__ __forceinline__ float2 gn_grad(float2 dy, float2 xhat, float2 gamma, float2 beta)
{
    if constexpr (ACT == CONV_ACT_RELU) return gn_dz<ACT>(dy, add2_apart(mul2(xhat, gamma), beta));
    return gn_dz<ACT>(dy, fma2(xhat, gamma, beta));
}

// dz from d = x - mean like gn_out.
template <int ACT>
__device__ __forceinline__ float2 gn_dz_at(float2 dy, float2 d, float2 rstd, float2 gamma_or_scale, float2 beta)
{
    if constexpr (ACT == CONV_ACT_RELU) return gn_dz<ACT>(dy, add2_apart(mul2(mul2(d, rstd), gamma_or_scale), beta));
    return gn_dz<ACT>(dy, fma2(d, gamma_or_scale, beta));
}

// Calls f(integral_constant<ACT>) for the runtime activation.
template <class F> __device__ __forceinline__ void with_act(int act, F&& f)
{
    switch (act) {
        case CONV_ACT_RELU: f(std::integral_constant<int, CONV_ACT_RELU>()); break;
        case CONV_ACT_SILU: f(std::integral_constant<int, CONV_ACT_SILU>()); break;
        case CONV_ACT_GELU: f(std::integral_constant<int, CONV_ACT_GELU>()); break;
        default: f(std::integral_constant<int, CONV_ACT_NONE>()); break;
    }
}

// The backward's channel sums: a thread adds its place's values over the samples it walks one after
// another, at most GN_CHAIN of them, so that the chain's roundings stay below 4e-6 of the sum of
// magnitudes (2105 samples of equal values, which one block walked, lost 2.3e-5).  So many blocks for
// `samples` samples (whole waves of `chunks`; never more than there are samples):
constexpr int GN_CHAIN = 256;
inline int gn_bounded_chunks(int chunks, int samples)
{
    return chunks * (((samples - 1) / GN_CHAIN + chunks) / chunks);
}

// ---- small groups: a team of lanes holds a group in registers --------------------------------
// A team is L lanes of a warp (a power of two); lane l holds the group's vectors l, l + L, ...
// (K of V values, E = K*V).  A block has gpc teams side by side on consecutive groups, spc such
// rows on consecutive samples, and walks the samples with its groups fixed, so that a lane's
// offsets in the sample and (backward) its channel sums stay in registers.  Gamma and beta lie
// in shared memory by position, in the order the lanes read them.
constexpr int GN_THREADS = 256;
// Values a lane holds at most; larger groups go to a cluster.  The backward also keeps two sums a
// value.  M = 512, forward, us, team / cluster: bf16 2048 x 512 x 16 21.7 / 24.4 (channels last
// 22.5 / 32.8), fp32 32.2 / 27.5.
constexpr int gn_team_values(int dt, bool bwd) { return bwd || dt == DT_F32 ? 12 : 16; }

struct GnTeam {
    int V, K, L;
    int gpc, spc, gsets, chunks;      // grid = gsets * chunks
    int threads;
    bool ok;
    FastDivmod dm_cgv, dm_p, dm_cg, dm_m;
};
GnTeam gn_team(const GnParams& p, int dt, const DevInfo& d, bool bwd);

// Vectors a lane (K) that are compiled for each width.
inline bool gn_team_k(int V, int K)
{
    switch (V) {
        case 8: return K == 1 || K == 2;
        case 4: return K >= 1 && K <= 4;
        case 2: return K == 2 || K == 4 || K == 8;
        default: return K == 2 || K == 4 || K == 8;
    }
}

// Offset of the group's vector j in the sample.
__device__ __forceinline__ int gn_offset(const GnParams& p, const GnTeam& q, int g, int j)
{
    if (p.layout == CONV_LAYOUT_NCHW) return int(g * p.M) + j * q.V;
    uint32_t row, cv;
    q.dm_cgv.divmod(uint32_t(j), row, cv);
    return int(row) * p.C + g * p.Cg + int(cv) * q.V;
}
// Channel (within the group) of the group's value e, counted in the order of the vectors.
__device__ __forceinline__ int gn_channel(const GnParams& p, const GnTeam& q, int e)
{
    uint32_t a, b;
    if (p.layout == CONV_LAYOUT_NCHW) return int(q.dm_p.div(uint32_t(e)));
    q.dm_cg.divmod(uint32_t(e), a, b);
    return int(b);
}
// Gamma and beta of the block's groups by position: gam[gpc * M], bet[gpc * M].
template <typename T>
__device__ __forceinline__ void gn_team_tables(const GnParams& p, const GnTeam& q, int g0, const T* gamma,
                                               const T* beta, float* gam, float* bet)
{
    const int m = int(p.M), n = min(q.gpc, p.G - g0) * m;
#pragma unroll 1
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        uint32_t gi, e;
        q.dm_m.divmod(uint32_t(i), gi, e);
        const int c = (g0 + int(gi)) * p.Cg + gn_channel(p, q, int(e));
        gam[i] = gamma ? Elem<T>::ldg(gamma + c) : 1.f;
        bet[i] = beta ? Elem<T>::ldg(beta + c) : 0.f;
    }
}

// Value pair h of K vectors of V values.
template <typename T, int V, int K> __device__ __forceinline__ float2 pair_of(const Vec<T, V> (&v)[K], int h)
{
    return make_float2(v[2 * h / V].get(2 * h % V), v[(2 * h + 1) / V].get((2 * h + 1) % V));
}
// A lane's table entries as pairs; toff[k]: where vector k's V floats begin.  Read 16 bytes at a
// time where V allows: consecutive lanes then read consecutive 16 bytes and no bank twice.
template <int V, int K>
__device__ __forceinline__ void table_pairs(const float* tab, const int (&toff)[K], float2 (&f)[K * V / 2])
{
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if constexpr (V >= 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 r = *reinterpret_cast<const float4*>(tab + toff[k] + i);
                f[(k * V + i) / 2] = make_float2(r.x, r.y);
                f[(k * V + i) / 2 + 1] = make_float2(r.z, r.w);
            }
        } else if constexpr (V == 2) {
            f[k] = *reinterpret_cast<const float2*>(tab + toff[k]);
        } else if (k % 2 == 0) {
            f[k / 2] = make_float2(tab[toff[k]], tab[toff[k + 1]]);
        }
    }
}

// s / m for m = p.m with the correctly rounded quotient's bits (one Newton step on s * inv_m), so
// that the mean of equal values is that value.
__device__ __forceinline__ float div_m(const GnParams& p, float s)
{
    const float q = s * p.inv_m;
    return fmaf(fmaf(-q, p.m, s), p.inv_m, q);
}

// Sums s of n values less a pivot (c is minus the pivot) and sq of their squares, moved to another
// pivot: the values' mean, rounded.  With D the step that the rounded pivot took, sum (x - p - D) is
// s - n D and sum (x - p - D)^2 is sq - D (s + (s - n D)), so nothing depends on how D was rounded.
template <int H> __device__ __forceinline__ void recentre(float2 (&c)[H], float2 (&s)[H], float2 (&sq)[H], float n)
{
    const float w = -fast_rcp(n);
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const float2 to = fma2(s[h], both(w), c[h]);
        const float2 step = add2(to, mul2(c[h], both(-1.f)));  // -D
        const float2 left = fma2(step, both(n), s[h]);
        sq[h] = fma2(step, add2(s[h], left), sq[h]);
        s[h] = left;
        c[h] = to;
    }
}

// Sum over the block, the same value in every thread.  `sm` holds 64 floats; `turn` alternates
// its halves so that one barrier a call is enough.
__device__ __forceinline__ float block_total(float v, float* sm, int& turn)
{
    v = warp_sum(v);
    float* half = sm + (turn & 1) * 32;
    ++turn;
    if ((threadIdx.x & 31) == 0) half[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = int(blockDim.x) >> 5;
    float t = 0.f;
    for (int w = 0; w < nw; ++w) t += half[w];
    return t;
}

// A thread's part of n numbers, n < 2^31 - 2^20: f(i, some) adds number i to `some`, which is added to
// `sum` after every 64, so that no chain of additions is long (2048 of equal numbers in one lost 2.6e-5).
template <class S, class F> __device__ __forceinline__ void gn_stretches(int n, S& sum, F&& f)
{
    const int hop = int(blockDim.x);
    for (int i = threadIdx.x; i < n;) {
        S some = {};
        for (const int stop = min(n, i + 64 * hop); i < stop; i += hop) f(i, some);
        if constexpr (sizeof(S) == 8) sum = add2(sum, some);
        else sum += some;
    }
}

// ---- large groups kept on chip by a cluster (kernels_gn_cluster.cu) --------------------------
struct GnCluster {
    int V, S, log_s, threads, K; // vector width, blocks a cluster (and its log2), threads, slots a thread
    int chunks;                  // clusters that share a unit's samples
    int W, cols, lanes, groups;  // NHWC: channels, vectors and groups of a window, rows side by side
    int wins;                    // units a sample
    int vecs;                    // NCHW: vectors of a unit
    int Cg, smem;
    bool nhwc, one, ok;          // one: NHWC, a vector lies in one group
    FastDivmod dm_cols, dm_cg, dm_p, dm_wins;
};
GnCluster gn_cluster(const GnParams& p, int dt, const DevInfo& d, bool bwd);
cudaError_t run_gn_cluster_fwd(const GnParams& p, const GnCluster& q, int dt, const void* x, const void* gamma,
                               const void* beta, void* y, float* mean, float* rstd, cudaStream_t s);
// part: (chunks * S, 2, C) channel sums (dgamma's, dbeta's), or NULL.
cudaError_t run_gn_cluster_bwd(const GnParams& p, const GnCluster& q, int dt, const void* x, const void* dy,
                               const void* gamma, const void* beta, const float* mean, const float* rstd, void* dx,
                               float* part, cudaStream_t s);

// ---- channels last, large groups: two passes over row tiles (kernels_gn_nhwc.cu) --------------
struct GnRows {
    int V, W, cols, wins;        // vector width; channels and vectors of a window, windows a sample
    int per;                     // windows a group (1: a window holds whole groups)
    int lanes, threads;          // rows side by side in a block
    int len, pieces, parts;      // rows a tile, tiles of the sample's rows, partial results of a group
    int64_t blocks;
    FastDivmod dm_cols, dm_cg, dm_wins, dm_pieces, dm_per;
};
GnRows gn_rows(const GnParams& p, int dt, const DevInfo& d, bool bwd);
// one position: both layouts are the same
inline bool gn_by_rows(const GnParams& p) { return p.layout == CONV_LAYOUT_NHWC || p.P == 1; }
// ws: B * G * parts float2
cudaError_t run_gn_rows_fwd(const GnParams& p, const GnRows& q, int dt, const void* x, const void* gamma,
                            const void* beta, void* y, float* mean, float* rstd, void* ws, cudaStream_t s);
// part: (B * pieces, 2, C) channel sums (dgamma's, dbeta's), or NULL.
cudaError_t run_gn_rows_bwd(const GnParams& p, const GnRows& q, int dt, const void* x, const void* dy,
                            const void* gamma, const void* beta, const float* mean, const float* rstd, void* dx,
                            float* part, void* ws, cudaStream_t s);

// ---- NCHW groups that no cluster holds: pieces of rows (one channel's positions) -------------
struct GnPieces {
    int V;
    int pieces, len;     // pieces a row, positions each
    int row_lanes;       // threads a row: the whole block, or a warp for short rows
    int threads;
    int64_t blocks;      // grid of the passes over x
};
GnPieces gn_pieces(const GnParams& p, int dt, const DevInfo& d);

// A block's rows: `sub` is the row within the block, `lane` the thread within the row.
struct GnRow {
    int64_t row;  // sample * C + channel
    int pc, lane, e0, e1, hop;
    bool in;
    __device__ __forceinline__ GnRow(const GnParams& p, const GnPieces& q, int V, int64_t at)
    {
        const int rows = int(blockDim.x) / q.row_lanes, sub = int(threadIdx.x) / q.row_lanes;
        lane = int(threadIdx.x) - sub * q.row_lanes;
        const int64_t i = at * rows + sub;
        row = i / q.pieces;
        pc = int(i - row * q.pieces);
        in = row < int64_t(p.B) * p.C;
        e0 = pc * q.len + lane * V;
        e1 = in ? min(p.P, pc * q.len + q.len) : 0;
        hop = q.row_lanes * V;
    }
};

// Index of the partial of (sample, piece, channel).
__device__ __forceinline__ int64_t gn_part(const GnParams& p, int pieces, int64_t b, int c, int pc)
{
    return (b * pieces + pc) * p.C + c;
}

// The compiled (V, K); MORE: those of the bf16 forward only.
#define GN_DISPATCH_TEAM(T, FWD, CALL)                                 \
    do {                                                               \
        constexpr bool MORE = (FWD) && sizeof(T) == 2;                 \
        if constexpr (sizeof(T) == 2)                                  \
            if (q.V == 8) {                                            \
                if constexpr (MORE)                                    \
                    if (q.K == 2) { CALL(T, 8, 2); break; }            \
                CALL(T, 8, 1);                                         \
                break;                                                 \
            }                                                          \
        if (q.V == 4) {                                                \
            if constexpr (MORE)                                        \
                if (q.K == 4) { CALL(T, 4, 4); break; }                \
            if (q.K == 1) { CALL(T, 4, 1); }                           \
            else if (q.K == 2) { CALL(T, 4, 2); }                      \
            else { CALL(T, 4, 3); }                                    \
        } else if (q.V == 2) {                                         \
            if constexpr (MORE)                                        \
                if (q.K == 8) { CALL(T, 2, 8); break; }                \
            if (q.K == 2) { CALL(T, 2, 2); }                           \
            else { CALL(T, 2, 4); }                                    \
        } else {                                                       \
            if (q.K == 2) { CALL(T, 1, 2); }                           \
            else if (q.K == 4) { CALL(T, 1, 4); }                      \
            else { CALL(T, 1, 8); }                                    \
        }                                                              \
    } while (0)

#define GN_DISPATCH_V(T, V_, CALL)                                     \
    do {                                                               \
        if constexpr (sizeof(T) == 2)                                  \
            if (V_ == 8) { CALL(T, 8); break; }                        \
        if (V_ == 4) { CALL(T, 4); }                                   \
        else if (V_ == 2) { CALL(T, 2); }                              \
        else { CALL(T, 1); }                                           \
    } while (0)

}  // namespace igc
