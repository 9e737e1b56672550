// kernels_grad.cu -- the global gradient norm over a list of tensors and clipping by it:
//   norm = sqrt(sum g^2),   out = g * min(1, max_norm / (norm + 1e-6)).
//
// One pass for the squares, one to scale: bound by memory.  The list travels in the kernel's
// parameters (no copy of pointers, no host wait).  The tensors are cut into tiles that the
// blocks take round robin, so each block's sum, and the order in which the scaling pass adds
// the blocks' sums, depend only on the list's sizes: the norm has the same bits every run.  The
// scaling pass walks the tiles backwards, so that what the first pass read last is still in L2.
//
// Measured: 48 tensors, 400 M bf16 values, clipped: 376 us; two reads and a write of 800 MB are 359
// us at the measured copy's rate, so 95% of that (L2 keeps an eighth of the second read at best).
// 300 tensors of either type, 60 M values, the norm: 30 us, 6.0 TB/s, 90%.  The encoder's nine
// tensors, 341 k fp32 values, clipped: 8 us, two launches.
#include <algorithm>

#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int GRAD_THREADS = 512;
constexpr int GRAD_TILE = 16384, GRAD_TILE_MIN = 2048;  // elements
constexpr int GRAD_BLOCKS_SM = 4;
constexpr int GRAD_LIST = 512, GRAD_SHORT = 32;         // entries a launch; of a short list's kernel

// N entries: a launch copies its parameters, so a short list has a short type, 1 KB and not 14: a clip of
// 9 tensors, the GPU waited for, takes 19.1 to 20.8 us with it and 19.7 to 21.0 without; among other
// calls, and with 48 tensors, the two do not differ.
template <int N> struct GradListOf {
    int count;
    int tiles;
    int tile;                      // elements
    int first[N + 1];              // first tile of each entry
    const void* grad[N];
    void* out[N];
    int64_t n[N];                  // elements; negative: bf16, -n of them
};
using GradList = GradListOf<GRAD_LIST>;
using GradShort = GradListOf<GRAD_SHORT>;

template <class L> __device__ __forceinline__ int find_entry(const L& l, int tile)
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

template <class L>
__global__ void __launch_bounds__(GRAD_THREADS) grad_squares(const __grid_constant__ L l, float* part)
{
    __shared__ float sm[GRAD_THREADS / 32];
    float s = 0.f;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    for (int t = blockIdx.x; t < l.tiles; t += gridDim.x) {
        const int k = find_entry(l, t);
        const int64_t n = l.n[k] < 0 ? -l.n[k] : l.n[k], at = int64_t(t - l.first[k]) * l.tile;
        const int cnt = int(n - at < l.tile ? n - at : l.tile);
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

template <class L>
__global__ void __launch_bounds__(GRAD_THREADS) grad_scale(const __grid_constant__ L l, const float* part, int parts,
                                                           float max_norm, float* norm)
{
    __shared__ float sm[GRAD_THREADS / 32];
    tc::grid_dep_wait();
    const float v = norm_of(part, parts, sm);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    float coef = __fdiv_rn(max_norm, v + 1e-6f);
    coef = coef > 1.f ? 1.f : coef;  // NaN stays
    for (int t = l.tiles - 1 - int(blockIdx.x); t >= 0; t -= int(gridDim.x)) {
        const int k = find_entry(l, t);
        const int64_t n = l.n[k] < 0 ? -l.n[k] : l.n[k], at = int64_t(t - l.first[k]) * l.tile;
        const int cnt = int(n - at < l.tile ? n - at : l.tile);
        if (l.n[k] < 0)
            tile_scale(static_cast<const __nv_bfloat16*>(l.grad[k]) + at, static_cast<__nv_bfloat16*>(l.out[k]) + at,
                       cnt, coef);
        else
            tile_scale(static_cast<const float*>(l.grad[k]) + at, static_cast<float*>(l.out[k]) + at, cnt, coef);
    }
}

// Elements a tile: GRAD_TILE where that gives every SM a few tiles, else down to GRAD_TILE_MIN
// (four elements a thread).
int tile_of(const conv_grad_t* g, int count, const DevInfo& d)
{
    int64_t total = 0;
    for (int i = 0; i < count; ++i) total += g[i].n;
    int tile = GRAD_TILE;
    while (tile > GRAD_TILE_MIN && total < int64_t(tile) * d.sms * GRAD_BLOCKS_SM) tile /= 2;
    return tile;
}

// Entries [i0, ...) that fit a launch; returns the next one.
int fill_list(const conv_grad_t* g, int count, int i0, int tile, GradList& l)
{
    l.count = 0;
    l.tile = tile;
    int64_t tiles = 0;
    int i = i0;
    for (; i < count && l.count < GRAD_LIST; ++i) {
        if (g[i].n == 0) continue;
        const int64_t t = (g[i].n + tile - 1) / tile;
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

void shorten(const GradList& l, GradShort& q)
{
    q.count = l.count;
    q.tiles = l.tiles;
    q.tile = l.tile;
    for (int i = 0; i < l.count; ++i) {
        q.first[i] = l.first[i];
        q.grad[i] = l.grad[i];
        q.out[i] = l.out[i];
        q.n[i] = l.n[i];
    }
    q.first[l.count] = l.tiles;
}

int list_grid(const GradList& l, const DevInfo& d) { return std::max(1, std::min(l.tiles, d.sms * GRAD_BLOCKS_SM)); }

cudaError_t launch_squares(const GradList& l, int grid, float* part, cudaStream_t s)
{
    if (l.count > GRAD_SHORT)
        return launch_ex(grad_squares<GradList>, dim3(grid), dim3(GRAD_THREADS), 0, s, 1, true, l, part);
    GradShort q;
    shorten(l, q);
    return launch_ex(grad_squares<GradShort>, dim3(grid), dim3(GRAD_THREADS), 0, s, 1, true, q, part);
}

cudaError_t launch_scale(const GradList& l, int grid, const float* part, int parts, float max_norm, float* norm,
                         cudaStream_t s)
{
    if (l.count > GRAD_SHORT)
        return launch_ex(grad_scale<GradList>, dim3(grid), dim3(GRAD_THREADS), 0, s, 1, true, l, part, parts, max_norm,
                         norm);
    GradShort q;
    shorten(l, q);
    return launch_ex(grad_scale<GradShort>, dim3(grid), dim3(GRAD_THREADS), 0, s, 1, true, q, part, parts, max_norm,
                     norm);
}

}  // namespace

// One float a block of each launch.
size_t grad_workspace(const conv_grad_t* g, int count, const DevInfo& d)
{
    GradList l;
    size_t floats = 0;
    const int tile = tile_of(g, count, d);
    for (int i = 0; i < count;) {
        i = fill_list(g, count, i, tile, l);
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
    const int tile = tile_of(g, count, d);
    for (int i = 0; i < count;) {
        i = fill_list(g, count, i, tile, l);
        if (l.tiles == 0) continue;
        const int grid = list_grid(l, d);
        const cudaError_t e = launch_squares(l, grid, part + parts, s);
        if (e != cudaSuccess) return e;
        parts += grid;
    }
    const float* cpart = part;
    if (!clip || parts == 0) {
        const cudaError_t e = launch_ex(grad_norm_kernel, dim3(1), dim3(GRAD_THREADS), 0, s, 1, true, cpart, parts, norm);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    for (int i = 0, first = 1; i < count;) {
        i = fill_list(g, count, i, tile, l);
        if (l.tiles == 0) continue;
        const cudaError_t e = launch_scale(l, list_grid(l, d), cpart, parts, max_norm, first ? norm : nullptr, s);
        if (e != cudaSuccess) return e;
        first = 0;
    }
    return cudaGetLastError();
}

}  // namespace igc
