// kernels_grad.cu -- the global gradient norm over a list of tensors and clipping by it:
//   norm = sqrt(sum g^2),   out = g * min(1, max_norm / (norm + 1e-6)).
//
// One pass for the squares, one to scale: bound by memory.  The list travels in the kernel's
// parameters (no copy of pointers, no host wait).  The tensors are cut into tiles that the
// blocks take round robin, so each block's sum, and the order in which the scaling pass adds
// the blocks' sums, depend only on the list's sizes: the norm has the same bits every run.  The
// scaling pass walks the tiles backwards, so that what the first pass read last is still in L2.
#include <algorithm>

#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int GRAD_THREADS = 512;
constexpr int GRAD_TILE = 16384;   // elements
constexpr int GRAD_BLOCKS_SM = 4;
constexpr int GRAD_LIST = 512;     // entries a launch

struct GradList {
    int count;
    int tiles;
    int first[GRAD_LIST + 1];      // first tile of each entry
    const void* grad[GRAD_LIST];
    void* out[GRAD_LIST];
    int64_t n[GRAD_LIST];          // elements; negative: bf16, -n of them
};

__device__ __forceinline__ int find_entry(const GradList& l, int tile)
{
    int lo = 0, hi = l.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (l.first[mid] <= tile) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// V elements at p: one load where p is aligned for it, else element by element.  Which thread
// takes which elements does not depend on the alignment, so neither do the sum's bits.
template <typename T, int V> __device__ __forceinline__ void load_any(Vec<T, V>& v, const T* p, bool aligned)
{
    if (aligned) {
        v.load(p);
    } else {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = Elem<T>::ld(p + i);
        v.set(f);
    }
}

template <typename T> __device__ __forceinline__ bool aligned_vec(const T* p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

template <typename T> __device__ __forceinline__ float tile_squares(const T* g, int cnt)
{
    constexpr int V = 16 / int(sizeof(T)), U = 4;
    const bool al = aligned_vec(g);
    const int done = cnt / V * V;
    float s = 0.f;
    for (int e = int(threadIdx.x) * V; e < done; e += GRAD_THREADS * V * U) {
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = e + u * GRAD_THREADS * V;
            if (at < done) load_any(v[u], g + at, al);
            else v[u].zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) s += v[u].get(i) * v[u].get(i);
    }
    if (done + int(threadIdx.x) < cnt) {
        const float f = Elem<T>::ld(g + done + threadIdx.x);
        s += f * f;
    }
    return s;
}

template <typename T> __device__ __forceinline__ void tile_scale(const T* g, T* o, int cnt, float coef)
{
    constexpr int V = 16 / int(sizeof(T)), U = 4;
    const bool al = aligned_vec(g), al_out = aligned_vec(o);
    const int done = cnt / V * V;
    for (int e = int(threadIdx.x) * V; e < done; e += GRAD_THREADS * V * U) {
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = e + u * GRAD_THREADS * V;
            if (at < done) load_any(v[u], g + at, al);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = e + u * GRAD_THREADS * V;
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = v[u].get(i) * coef;
            if (at < done) {
                if (al_out) {
                    v[u].set(f);
                    v[u].store(o + at);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) Elem<T>::st(o + at + i, f[i]);
                }
            }
        }
    }
    const int e = done + int(threadIdx.x);
    if (e < cnt) Elem<T>::st(o + e, Elem<T>::ld(g + e) * coef);
}

__device__ __forceinline__ float block_total(float s, float* sm)
{
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
    for (int w = 0; w < int(blockDim.x) / 32; ++w) s += sm[w];
    return s;
}

__global__ void __launch_bounds__(GRAD_THREADS) grad_squares(const __grid_constant__ GradList l, float* part)
{
    __shared__ float sm[GRAD_THREADS / 32];
    float s = 0.f;
    tc::grid_dep_wait();
    for (int t = blockIdx.x; t < l.tiles; t += gridDim.x) {
        const int k = find_entry(l, t);
        const int64_t n = l.n[k] < 0 ? -l.n[k] : l.n[k], at = int64_t(t - l.first[k]) * GRAD_TILE;
        const int cnt = int(n - at < GRAD_TILE ? n - at : GRAD_TILE);
        s += l.n[k] < 0 ? tile_squares(static_cast<const __nv_bfloat16*>(l.grad[k]) + at, cnt)
                        : tile_squares(static_cast<const float*>(l.grad[k]) + at, cnt);
    }
    s = block_total(s, sm);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ float norm_of(const float* part, int parts, float* sm)
{
    float s = 0.f;
    for (int i = threadIdx.x; i < parts; i += blockDim.x) s += part[i];
    return sqrtf(block_total(s, sm));
}

__global__ void __launch_bounds__(GRAD_THREADS) grad_norm_kernel(const float* part, int parts, float* norm)
{
    __shared__ float sm[GRAD_THREADS / 32];
    tc::grid_dep_wait();
    const float v = norm_of(part, parts, sm);
    if (threadIdx.x == 0) *norm = v;
}

__global__ void __launch_bounds__(GRAD_THREADS) grad_scale(const __grid_constant__ GradList l, const float* part,
                                                           int parts, float max_norm, float* norm)
{
    __shared__ float sm[GRAD_THREADS / 32];
    tc::grid_dep_wait();
    const float v = norm_of(part, parts, sm);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    float coef = __fdiv_rn(max_norm, v + 1e-6f);
    coef = coef > 1.f ? 1.f : coef;  // NaN stays
    for (int t = l.tiles - 1 - int(blockIdx.x); t >= 0; t -= int(gridDim.x)) {
        const int k = find_entry(l, t);
        const int64_t n = l.n[k] < 0 ? -l.n[k] : l.n[k], at = int64_t(t - l.first[k]) * GRAD_TILE;
        const int cnt = int(n - at < GRAD_TILE ? n - at : GRAD_TILE);
        if (l.n[k] < 0)
            tile_scale(static_cast<const __nv_bfloat16*>(l.grad[k]) + at, static_cast<__nv_bfloat16*>(l.out[k]) + at,
                       cnt, coef);
        else
            tile_scale(static_cast<const float*>(l.grad[k]) + at, static_cast<float*>(l.out[k]) + at, cnt, coef);
    }
}

// Entries [i0, ...) that fit a launch; returns the next one.
int fill_list(const conv_grad_t* g, int count, int i0, GradList& l)
{
    l.count = 0;
    int64_t tiles = 0;
    int i = i0;
    for (; i < count && l.count < GRAD_LIST; ++i) {
        if (g[i].n == 0) continue;
        const int64_t t = (g[i].n + GRAD_TILE - 1) / GRAD_TILE;
        if (tiles + t > (int64_t(1) << 30)) break;
        l.first[l.count] = int(tiles);
        l.grad[l.count] = g[i].grad;
        l.out[l.count] = g[i].out;
        l.n[l.count] = g[i].dtype == CONV_BF16 ? -g[i].n : g[i].n;
        tiles += t;
        ++l.count;
    }
    l.first[l.count] = int(tiles);
    l.tiles = int(tiles);
    return i;
}

int list_grid(const GradList& l, const DevInfo& d) { return std::max(1, std::min(l.tiles, d.sms * GRAD_BLOCKS_SM)); }

}  // namespace

// One float a block of each launch.
size_t grad_workspace(const conv_grad_t* g, int count, const DevInfo& d)
{
    GradList l;
    size_t floats = 0;
    for (int i = 0; i < count;) {
        i = fill_list(g, count, i, l);
        if (l.tiles > 0) floats += size_t(list_grid(l, d));
    }
    return floats * 4;
}

cudaError_t run_grad_norm(const conv_grad_t* g, int count, bool clip, float max_norm, const DevInfo& d, float* norm,
                          void* ws, cudaStream_t s)
{
    float* part = static_cast<float*>(ws);
    GradList l;
    int parts = 0;
    for (int i = 0; i < count;) {
        i = fill_list(g, count, i, l);
        if (l.tiles == 0) continue;
        const int grid = list_grid(l, d);
        const cudaError_t e = launch_ex(grad_squares, dim3(grid), dim3(GRAD_THREADS), 0, s, 1, true, l, part + parts);
        if (e != cudaSuccess) return e;
        parts += grid;
    }
    const float* cpart = part;
    if (!clip || parts == 0) {
        const cudaError_t e = launch_ex(grad_norm_kernel, dim3(1), dim3(GRAD_THREADS), 0, s, 1, true, cpart, parts, norm);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    for (int i = 0, first = 1; i < count;) {
        i = fill_list(g, count, i, l);
        if (l.tiles == 0) continue;
        const cudaError_t e = launch_ex(grad_scale, dim3(list_grid(l, d)), dim3(GRAD_THREADS), 0, s, 1, true, l, cpart,
                                        parts, max_norm, first ? norm : static_cast<float*>(nullptr));
        if (e != cudaSuccess) return e;
        first = 0;
    }
    return cudaGetLastError();
}

}  // namespace igc
