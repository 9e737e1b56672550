// train_internal.h -- what the training-step operators' translation units share: vector access
// in either storage type, warp reductions, and the launchers behind the C ABI (train_api.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/conv_train.h"
#include "internal.h"

namespace igc {

// V consecutive elements of T in registers, as loaded (bf16 stays packed until it is used).
template <int BYTES> struct RawBits;
template <> struct RawBits<2> { uint16_t w[1]; };
template <> struct __align__(4) RawBits<4> { uint32_t w[1]; };
template <> struct __align__(8) RawBits<8> { uint32_t w[2]; };
template <> struct __align__(16) RawBits<16> { uint32_t w[4]; };

template <typename T, int V> struct Vec {
    RawBits<int(sizeof(T)) * V> r;

    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (sizeof(T) * V == 16) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
        } else if constexpr (sizeof(T) * V == 8) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            r.w[0] = u.x; r.w[1] = u.y;
        } else if constexpr (sizeof(T) * V == 4) {
            r.w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            r.w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const
    {
        if constexpr (sizeof(T) * V == 16)
            *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        else if constexpr (sizeof(T) * V == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
        else if constexpr (sizeof(T) * V == 4)
            *reinterpret_cast<uint32_t*>(p) = r.w[0];
        else
            *reinterpret_cast<uint16_t*>(p) = r.w[0];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < int(sizeof(r.w) / sizeof(r.w[0])); ++i) r.w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i]);
        else if constexpr (V == 1) return __uint_as_float(uint32_t(r.w[0]) << 16);
        else return __uint_as_float((i & 1) ? (r.w[i >> 1] & 0xFFFF0000u) : (r.w[i >> 1] << 16));
    }
    // All V values at once: bf16 rounds each to nearest even.
    __device__ __forceinline__ void set(const float (&v)[V])
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(v[i]);
        } else if constexpr (V == 1) {
            r.w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
};

// Sum over the `width` lanes of a team (a power of two; teams are aligned in the warp), in a
// fixed butterfly order; every lane of the warp takes part.
__device__ __forceinline__ float team_sum(float v, int width)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < width) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// ---- group norm (kernels_gn_fwd.cu, kernels_gn_bwd.cu) --------------------------------------
struct GnParams {
    int B, C, P, G, Cg;
    int act, layout;
    int64_t M;        // values of a group: Cg * P
    int64_t N;        // values of a sample: C * P
    float eps, m, inv_m;  // M and 1 / M
};
size_t gn_fwd_workspace(const GnParams& p, int dt, const DevInfo& d);
cudaError_t run_gn_fwd(const GnParams& p, int dt, const DevInfo& d, const void* x, const void* gamma,
                       const void* beta, void* y, float* mean, float* rstd, void* ws, cudaStream_t s);
size_t gn_bwd_workspace(const GnParams& p, int dt, const DevInfo& d);
cudaError_t run_gn_bwd(const GnParams& p, int dt, const DevInfo& d, const void* x, const void* dy, const void* gamma,
                       const void* beta, const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                       void* ws, cudaStream_t s);

// ---- embedding (kernels_embed.cu) -----------------------------------------------------------
cudaError_t run_embed_fwd(const conv_embed_desc_t& e, const DevInfo& d, const void* idx, const void* table, void* y,
                          cudaStream_t s);
size_t embed_bwd_workspace(const conv_embed_desc_t& e, const DevInfo& d);
cudaError_t run_embed_bwd(const conv_embed_desc_t& e, const DevInfo& d, const void* idx, const void* dy, void* dtable,
                          void* ws, cudaStream_t s);

// ---- gradient norm (kernels_grad.cu) --------------------------------------------------------
size_t grad_workspace(const conv_grad_t* g, int count, const DevInfo& d);
cudaError_t run_grad_norm(const conv_grad_t* g, int count, bool clip, float max_norm, const DevInfo& d, float* norm,
                          void* ws, cudaStream_t s);

}  // namespace igc
