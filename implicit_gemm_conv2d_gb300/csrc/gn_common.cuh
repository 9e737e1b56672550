// gn_common.cuh -- the activations, the elementwise halves and the launch geometry that the
// group norm's forward and backward share.
#pragma once
#include <algorithm>
#include <type_traits>

#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

template <int ACT> __device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == CONV_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    if constexpr (ACT == CONV_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    if constexpr (ACT == CONV_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    return z;
}

template <int ACT> __device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == CONV_ACT_SILU) {
        const float p = __fdividef(1.f, 1.f + __expf(-z));
        return p * (1.f + z * (1.f - p));
    }
    if constexpr (ACT == CONV_ACT_GELU)
        return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.39894228040143268f * __expf(-0.5f * z * z);
    return 1.f;
}

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

// dz = dy * act'(z); a ReLU that is off passes nothing, whatever dy holds there.
template <int ACT> __device__ __forceinline__ float gn_dz(float dy, float xhat, float gamma, float beta)
{
    if constexpr (ACT == CONV_ACT_NONE) return dy;
    const float z = gn_z(xhat, gamma, beta);
    if constexpr (ACT == CONV_ACT_RELU) return z > 0.f ? dy : 0.f;
    return dy * act_slope<ACT>(z);
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

// ---- small groups: a team of threads holds a group in registers ------------------------------
// A team is L lanes (a power of two within a warp, or a whole block of 32*W threads); lane l
// holds the group's vectors l, l + L, ... (K of V values).  A block has gpc teams side by side
// on consecutive groups, spc such rows on consecutive samples, and walks the samples with its
// groups fixed: a lane's offsets in the sample, its gamma and beta and (backward) its channel
// sums stay in registers.
constexpr int GN_THREADS = 256;       // block of sub-warp teams
constexpr int GN_TEAM_MAX = 512;      // lanes of a block-wide team
constexpr int GN_LANE_VALUES = 16;    // values a lane holds at most

struct GnTeam {
    int V, K, L;
    int gpc, spc, gsets, chunks;      // grid = gsets * chunks
    int threads;
    bool ok;
};

inline int gn_vector_width(const GnParams& p, int es)
{
    // the widest vector (16 bytes at most) that keeps every group's vectors aligned and whole
    const int64_t n = p.layout == CONV_LAYOUT_NCHW ? p.M : p.Cg;
    int v = 16 / es;
    while (v > 1 && n % v != 0) v /= 2;
    return v;
}

// K variants that are compiled for each V.
inline bool gn_team_k(int V, int K)
{
    switch (V) {
        case 8: return K == 1 || K == 2;
        case 4: return K >= 1 && K <= 4;
        case 2: return K == 2 || K == 4 || K == 8;
        default: return K == 2 || K == 4 || K == 8 || K == 16;
    }
}

GnTeam gn_team(const GnParams& p, int dt, const DevInfo& d, bool bwd);

// Sum over a block-wide team (or a sub-warp one), the same value in every lane.  `sm` holds 64
// floats; `turn` alternates its halves so that one barrier a call is enough.
template <bool WIDE> __device__ __forceinline__ float team_total(float v, int L, float* sm, int& turn)
{
    if constexpr (!WIDE) return team_sum(v, L);
    v = warp_sum(v);
    float* half = sm + (turn & 1) * 32;
    ++turn;
    if ((threadIdx.x & 31) == 0) half[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = L >> 5;
    float t = 0.f;
    for (int w = 0; w < nw; ++w) t += half[w];
    return t;
}

// ---- large groups: pieces of rows ------------------------------------------------------------
// NHWC: a piece is a range of a sample's positions, all channels of a column window; NCHW: a
// range of one channel's positions.  `pieces` a sample (a channel), `len` positions each.
struct GnPieces {
    int V;
    int pieces, len;
    int cols, wins;      // NHWC: column vectors a window, windows
    int row_lanes;       // NCHW: threads a row (channel): the whole block, or a warp for short rows
    int threads;
    int64_t blocks;      // grid of the passes over x
};
GnPieces gn_pieces(const GnParams& p, int dt, const DevInfo& d);

// The NHWC passes' block: window fastest, then piece, then sample.
struct GnTile {
    int b, pc, cv0, cols, lanes, col, lane, r0, r1;
    __device__ __forceinline__ GnTile(const GnParams& p, const GnPieces& q, int V, int64_t at)
    {
        const int per = q.pieces * q.wins;
        b = int(at / per);
        const int rest = int(at - int64_t(b) * per);
        pc = rest / q.wins;
        cv0 = (rest - pc * q.wins) * q.cols;
        cols = min(q.cols, p.C / V - cv0);
        lanes = max(1, int(blockDim.x) / q.cols);
        lane = int(threadIdx.x) / q.cols;
        col = int(threadIdx.x) - lane * q.cols;
        r0 = pc * q.len;
        r1 = min(p.P, r0 + q.len);
    }
    __device__ __forceinline__ bool in() const { return lane < lanes && col < cols; }
};
// The NCHW passes' rows: `sub` is the row within the block, `lane` the thread within the row.
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

// Index of the partial of (sample, channel, piece).
__device__ __forceinline__ int64_t gn_part(const GnParams& p, int pieces, int b, int c, int pc)
{
    return p.layout == CONV_LAYOUT_NHWC ? (int64_t(b) * pieces + pc) * p.C + c
                                        : (int64_t(b) * p.C + c) * pieces + pc;
}

#define GN_DISPATCH_TEAM(T, CALL)                                      \
    do {                                                               \
        if constexpr (sizeof(T) == 2)                                  \
            if (q.V == 8) {                                            \
                if (q.K == 1) { CALL(T, 8, 1); }                       \
                else { CALL(T, 8, 2); }                                \
                break;                                                 \
            }                                                          \
        if (q.V == 4) {                                                \
            if (q.K == 1) { CALL(T, 4, 1); }                           \
            else if (q.K == 2) { CALL(T, 4, 2); }                      \
            else if (q.K == 3) { CALL(T, 4, 3); }                      \
            else { CALL(T, 4, 4); }                                    \
        } else if (q.V == 2) {                                         \
            if (q.K == 2) { CALL(T, 2, 2); }                           \
            else if (q.K == 4) { CALL(T, 2, 4); }                      \
            else { CALL(T, 2, 8); }                                    \
        } else {                                                       \
            if (q.K == 2) { CALL(T, 1, 2); }                           \
            else if (q.K == 4) { CALL(T, 1, 4); }                      \
            else if (q.K == 8) { CALL(T, 1, 8); }                      \
            else { CALL(T, 1, 16); }                                   \
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
