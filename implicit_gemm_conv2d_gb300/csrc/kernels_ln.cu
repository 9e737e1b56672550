// kernels_ln.cu -- layer norm of rows, of a residual sum where one is given:
//   s = x + residual (kept as T)      y = (s - mean) rstd gamma + beta
//   dx = rstd (e - m1 - xhat m2) + dtotal,  e = dy gamma,  m1 = mean of e,  m2 = mean of e xhat
//   dgamma = sum over the rows of dy xhat      dbeta = sum over the rows of dy
// (the form without a mean: mean, m1 and beta are 0).
//
// Bound by memory: a row is read once and held in the registers of a team, from a few lanes to 32
// warps; mean and squared deviations are two passes over the registers.  Blocks stay and take rows in turn.  In
// the backward a thread keeps its columns' sums of dgamma and dbeta over all rows of its team, the
// block's go to the workspace and a second kernel adds those: an order that the sizes fix.
// Rows that no team holds are read again for each pass.
#include <algorithm>

#include "gn_common.cuh"
#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int LN_MOST = 1024;    // threads of a team, forward
constexpr int LN_MOST_BWD = 512; // backward: 128 registers a thread
constexpr int LN_FLUSH = 256;    // rows that are added to each other in one chain

// Rows a team of the backward takes at once: what a thread's registers hold of x, dy and dtotal, 48 of them, beside
// its columns' sums.
constexpr int ln_rows(int es, int V, int NV)
{
    const int regs = 3 * NV * (es == 2 && V > 1 ? V / 2 : V);
    return regs <= 12 ? 4 : NV * V <= 8 ? 2 : 1;
}

// A thread's place: teams of TL threads, each a row at a time.
struct LnAt {
    int lane, team, TL, teams, warps;  // warps of a team of more than one, else 1
    __device__ __forceinline__ explicit LnAt(const LnParams& p)
    {
        TL = p.TL;
        teams = p.teams;
        lane = teams > 1 ? int(threadIdx.x) & (TL - 1) : int(threadIdx.x);
        team = teams > 1 ? int(threadIdx.x) / TL : 0;
        warps = TL > 32 ? TL / 32 : 1;
    }
};

// Sums of K values over the team; every thread of the block takes part.  sm: 32 * K floats that nobody reads any
// more.
template <int K> __device__ __forceinline__ void ln_sum(const LnAt& q, float (&v)[K], float* sm)
{
    const int width = q.TL < 32 ? q.TL : 32;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < width) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
        }
    if (q.warps == 1) return;
    const int warp = int(threadIdx.x) >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) sm[warp * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.f;
    for (int w = 0; w < q.warps; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += sm[w * K + k];
}

template <typename T, int V, int NV>
__global__ void __launch_bounds__(LN_MOST)
ln_fwd_kernel(const __grid_constant__ LnParams p, const T* x, const T* residual, const T* gamma, const T* beta, T* y,
              T* total, float* mean, float* rstd)
{
    __shared__ float sm[2][32];
    const LnAt q(p);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    for (int64_t row0 = int64_t(blockIdx.x) * q.teams; row0 < p.N; row0 += int64_t(gridDim.x) * q.teams) {
        const int64_t row = row0 + q.team, at = row * p.D;
        const bool on = row < p.N;
        Vec<T, V> a[NV];
        float f[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = q.lane + i * q.TL;
            a[i].zero();
            if (on && j < p.vecs) a[i].load(x + at + int64_t(j) * V);
        }
        if (residual) {
            Vec<T, V> r[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = q.lane + i * q.TL;
                r[i].zero();
                if (on && j < p.vecs) r[i].load(residual + at + int64_t(j) * V);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = q.lane + i * q.TL;
                float s[V];
#pragma unroll
                for (int v = 0; v < V; ++v) s[v] = a[i].get(v) + r[i].get(v);
                a[i].set(s);
                if (on && j < p.vecs) a[i].store(total + at + int64_t(j) * V);
            }
        }
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[i][v] = a[i].get(v);
                sum[0] += f[i][v];
            }
        float m = 0.f;
        if (!p.rms) {
            ln_sum(q, sum, sm[0]);
            m = sum[0] * p.inv_d;
        }
        float sq[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = q.lane + i * q.TL < p.vecs;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                f[i][v] -= m;
                if (in) sq[0] += f[i][v] * f[i][v];
            }
        }
        if (p.rms && q.warps > 1) __syncthreads();  // the sums of the row before have been read
        ln_sum(q, sq, sm[1]);
        const float r = __frsqrt_rn(sq[0] * p.inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int j = q.lane + i * q.TL;
            if (!on || j >= p.vecs) continue;
            Vec<T, V> g, b, o;
            if (gamma) g.load(gamma + j * V);
            if (beta) b.load(beta + j * V);
            float out[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float h = f[i][v] * r;
                out[v] = fmaf(h, gamma ? g.get(v) : 1.f, beta ? b.get(v) : 0.f);
            }
            o.set(out);
            o.store(y + at + int64_t(j) * V);
        }
        if (on && q.lane == 0) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = r;
        }
    }
}

// A block a row, of any length: the row is read again for each pass.
template <typename T, int V>
__global__ void __launch_bounds__(LN_MOST)
ln_fwd_long(const __grid_constant__ LnParams p, const T* x, const T* residual, const T* gamma, const T* beta, T* y,
            T* total, float* mean, float* rstd)
{
    __shared__ float sm[2][32];
    const LnAt q(p);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
        const int64_t at = row * p.D;
        const T* s = residual ? total : x;
        float sum[1] = {0.f};
        for (int j = q.lane; j < p.vecs; j += q.TL) {
            Vec<T, V> a;
            a.load(x + at + int64_t(j) * V);
            float f[V], t = 0.f;
            if (residual) {
                Vec<T, V> r;
                r.load(residual + at + int64_t(j) * V);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = a.get(v) + r.get(v);
                a.set(f);
                a.store(total + at + int64_t(j) * V);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) t += a.get(v);
            sum[0] += t;
        }
        float m = 0.f;
        if (!p.rms) {
            ln_sum(q, sum, sm[0]);
            m = sum[0] * p.inv_d;
        }
        float sq[1] = {0.f};
        for (int j = q.lane; j < p.vecs; j += q.TL) {
            Vec<T, V> a;
            a.load(s + at + int64_t(j) * V);
            float t = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) t += (a.get(v) - m) * (a.get(v) - m);
            sq[0] += t;
        }
        if (p.rms) __syncthreads();
        ln_sum(q, sq, sm[1]);
        const float r = __frsqrt_rn(sq[0] * p.inv_d + p.eps);
        for (int j = q.lane; j < p.vecs; j += q.TL) {
            Vec<T, V> a, g, b;
            a.load(s + at + int64_t(j) * V);
            if (gamma) g.load(gamma + int64_t(j) * V);
            if (beta) b.load(beta + int64_t(j) * V);
            float out[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                out[v] = fmaf((a.get(v) - m) * r, gamma ? g.get(v) : 1.f, beta ? b.get(v) : 0.f);
            a.set(out);
            a.store(y + at + int64_t(j) * V);
        }
        if (threadIdx.x == 0) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = r;
        }
    }
}

// Columns c and c + 1 of a thread's NV vectors; a single column has a second one of 0.
template <typename T, int V, int NV> __device__ __forceinline__ float2 pick(const Vec<T, V> (&a)[NV], int c)
{
    if constexpr (V * NV == 1) return make_float2(a[0].get(0), 0.f);
    else return make_float2(a[c / V].get(c % V), a[(c + 1) / V].get((c + 1) % V));
}

// R rows a team at a time.  part: [block][dgamma, dbeta][D], or NULL.
template <typename T, int V, int NV, int R>
__global__ void __launch_bounds__(LN_MOST_BWD)
ln_bwd_kernel(const __grid_constant__ LnParams p, const T* x, const T* dy, const T* gamma, const float* mean,
              const float* rstd, const T* dtotal, T* dx, float* part)
{
    extern __shared__ __align__(16) float dyn[];  // [2 NV V][threads]: what the chains of additions have left so far
    __shared__ float sm[2][32 * 2 * R];
    constexpr int CPT = NV * V, P = (CPT + 1) / 2;
    const LnAt q(p);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float2 dg[P], db[P];
    Vec<T, V> g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = q.lane + i * q.TL;
        float one[V];
#pragma unroll
        for (int v = 0; v < V; ++v) one[v] = 1.f;
        g[i].set(one);
        if (gamma && j < p.vecs) g[i].load(gamma + j * V);
    }
#pragma unroll
    for (int c = 0; c < P; ++c) dg[c] = db[c] = both(0.f);
    const int slot = 2 * int(blockDim.x);
    if (p.flush)
        for (int k = 0; k < 2 * P; ++k) reinterpret_cast<float2*>(dyn)[k * int(blockDim.x) + int(threadIdx.x)] = both(0.f);
    auto flush = [&] {
#pragma unroll
        for (int c = 0; c < P; ++c) {
            float2* a = reinterpret_cast<float2*>(dyn) + c * slot + threadIdx.x;
            a[0] = add2(a[0], dg[c]);
            a[blockDim.x] = add2(a[blockDim.x], db[c]);
            dg[c] = db[c] = both(0.f);
        }
    };
    const int64_t stride = int64_t(gridDim.x) * q.teams * R;
    int turn = 0, chain = 0;
    for (int64_t row0 = int64_t(blockIdx.x) * q.teams * R; row0 < p.N; row0 += stride, turn ^= 1) {
        const int64_t row = row0 + q.team * R;
        Vec<T, V> a[R][NV], d[R][NV], t[R][NV];
        float m[R], r[R], sums[2 * R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const bool on = row + k < p.N;
            m[k] = on && mean ? mean[row + k] : 0.f;
            r[k] = on ? rstd[row + k] : 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = q.lane + i * q.TL;
                const int64_t at = (row + k) * p.D + int64_t(j) * V;
                a[k][i].zero();
                d[k][i].zero();  // (dy of 0: a place that is not there adds nothing)
                t[k][i].zero();
                if (on && j < p.vecs) {
                    a[k][i].load(x + at);
                    d[k][i].load(dy + at);
                    if (dtotal) t[k][i].load(dtotal + at);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int c = 0; c < P; ++c) {
                const float2 xh = mul2(add2(pick(a[k], 2 * c), both(-m[k])), both(r[k])), y = pick(d[k], 2 * c);
                const float2 e = mul2(y, pick(g, 2 * c));
                s1 = add2(s1, e);
                s2 = fma2(e, xh, s2);
                dg[c] = fma2(y, xh, dg[c]);
                db[c] = add2(db[c], y);
            }
            sums[2 * k] = s1.x + s1.y;
            sums[2 * k + 1] = s2.x + s2.y;
        }
        ln_sum(q, sums, sm[turn]);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (row + k >= p.N) continue;
            const float m1 = p.rms ? 0.f : sums[2 * k] * p.inv_d, m2 = sums[2 * k + 1] * p.inv_d;
            float o[2 * P];
#pragma unroll
            for (int c = 0; c < P; ++c) {
                const float2 xh = mul2(add2(pick(a[k], 2 * c), both(-m[k])), both(r[k]));
                const float2 e = mul2(pick(d[k], 2 * c), pick(g, 2 * c));
                const float2 v = fma2(both(r[k]), fma2(xh, both(-m2), add2(e, both(-m1))), pick(t[k], 2 * c));
                o[2 * c] = v.x;
                o[2 * c + 1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int j = q.lane + i * q.TL;
                float f[V];
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = o[i * V + v];
                a[k][i].set(f);
                if (j < p.vecs) a[k][i].store(dx + (row + k) * p.D + int64_t(j) * V);
            }
        }
        chain += R;
        if (p.flush && chain >= LN_FLUSH) {
            flush();
            chain = 0;
        }
    }
    if (!part) return;
    if (p.flush) {
        flush();
#pragma unroll
        for (int c = 0; c < P; ++c) {
            const float2* a = reinterpret_cast<const float2*>(dyn) + c * slot + threadIdx.x;
            dg[c] = a[0];
            db[c] = a[blockDim.x];
        }
        __syncthreads();
    }
    float* to = part + int64_t(blockIdx.x) * 2 * p.D;
    const int warp = int(threadIdx.x) >> 5, warps = int(blockDim.x) >> 5;
    // Teams of a warp and less: over the warp's teams by shuffles, over the warps in shared memory.
    float* at = q.teams > 1 ? dyn + warp * 2 * p.D : to;
    const bool writes = q.teams == 1 || (threadIdx.x & 31) < unsigned(q.TL);
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
        float u = c & 1 ? dg[c / 2].y : dg[c / 2].x, w = c & 1 ? db[c / 2].y : db[c / 2].x;
        const int j = q.lane + c / V * q.TL;
        for (int o = q.TL; o < 32; o *= 2) {
            u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
            w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
        }
        if (writes && j < p.vecs) {
            at[j * V + c % V] = u;
            at[p.D + j * V + c % V] = w;
        }
    }
    if (q.teams == 1) return;
    __syncthreads();
    for (int c = int(threadIdx.x); c < 2 * p.D; c += int(blockDim.x)) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += dyn[w * 2 * p.D + c];
        to[c] = s;
    }
}

// ---- rows that no team holds: the rows' sums, then columns of all rows -------------------------
template <typename T, int V>
__global__ void __launch_bounds__(LN_MOST)
ln_bwd_rows(const __grid_constant__ LnParams p, const T* x, const T* dy, const T* gamma, const float* mean,
            const float* rstd, float2* sums)
{
    __shared__ float sm[2][64];
    const LnAt q(p);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, turn ^= 1) {
        const float m = mean ? mean[row] : 0.f, r = rstd[row];
        float s[2] = {0.f, 0.f};
        for (int j = q.lane; j < p.vecs; j += q.TL) {
            const int64_t at = row * p.D + int64_t(j) * V;
            Vec<T, V> a, d, g;
            a.load(x + at);
            d.load(dy + at);
            if (gamma) g.load(gamma + int64_t(j) * V);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float e = gamma ? d.get(v) * g.get(v) : d.get(v);
                s1 += e;
                s2 += e * ((a.get(v) - m) * r);
            }
            s[0] += s1;
            s[1] += s2;
        }
        ln_sum(q, s, sm[turn]);
        if (threadIdx.x == 0) sums[row] = make_float2(p.rms ? 0.f : s[0] * p.inv_d, s[1] * p.inv_d);
    }
}

// Block (x, y): LN_COLUMNS vectors of columns, every gridDim.y-th row; a thread a vector.
constexpr int LN_COLUMNS = 128;
template <typename T, int V>
__global__ void __launch_bounds__(LN_COLUMNS)
ln_bwd_columns(const __grid_constant__ LnParams p, const T* x, const T* dy, const T* gamma, const float* mean,
               const float* rstd, const T* dtotal, const float2* sums, T* dx, float* part)
{
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int64_t j = int64_t(blockIdx.x) * LN_COLUMNS + threadIdx.x;
    if (j >= p.vecs) return;
    Vec<T, V> g;
    if (gamma) g.load(gamma + j * V);
    float dg[V], db[V], dg2[V], db2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dg[v] = db[v] = dg2[v] = db2[v] = 0.f;
    int chain = 0;
    for (int64_t row = blockIdx.y; row < p.N; row += gridDim.y) {
        const int64_t at = row * p.D + j * V;
        const float m = mean ? mean[row] : 0.f, r = rstd[row];
        const float2 s = sums[row];
        Vec<T, V> a, d, t;
        a.load(x + at);
        d.load(dy + at);
        t.zero();
        if (dtotal) t.load(dtotal + at);
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float xh = (a.get(v) - m) * r, y = d.get(v), e = gamma ? y * g.get(v) : y;
            dg[v] += y * xh;
            db[v] += y;
            o[v] = fmaf(r, e - s.x - xh * s.y, t.get(v));
        }
        a.set(o);
        a.store(dx + at);
        if (++chain == LN_FLUSH) {
            chain = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dg2[v] += dg[v];
                db2[v] += db[v];
                dg[v] = db[v] = 0.f;
            }
        }
    }
    if (!part) return;
    float* to = part + int64_t(blockIdx.y) * 2 * p.D;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        to[j * V + v] = dg2[v] + dg[v];
        to[p.D + j * V + v] = db2[v] + db[v];
    }
}

// dgamma, dbeta from the blocks' sums: 32 columns a block, its 32 warps take every 32nd partial.
template <typename T>
__global__ void __launch_bounds__(1024)
ln_params_kernel(const float* part, int parts, int D, T* dgamma, T* dbeta)
{
    __shared__ float sm[32][33];
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5, columns = dbeta ? 2 * D : D;
    const int64_t c = int64_t(blockIdx.x) * 32 + lane;
    float s = 0.f;
    if (c < columns) {
#pragma unroll 8
        for (int k = warp; k < parts; k += 32) s += part[int64_t(k) * 2 * D + c];
    }
    sm[warp][lane] = s;
    __syncthreads();
    const float v = warp_sum(sm[lane][warp]);
    const int64_t o = int64_t(blockIdx.x) * 32 + warp;
    if (lane == 0 && o < columns) Elem<T>::st(o < D ? dgamma + o : dbeta + (o - D), v);
}

template <int N> using Int = std::integral_constant<int, N>;

// Calls f(T(), V) for the plan.
template <class F> cudaError_t ln_types(const LnParams& p, int dt, F&& f)
{
    if (dt == DT_F32) return p.V == 4 ? f(float(), Int<4>()) : p.V == 2 ? f(float(), Int<2>()) : f(float(), Int<1>());
    return p.V == 8   ? f(__nv_bfloat16(), Int<8>())
           : p.V == 2 ? f(__nv_bfloat16(), Int<2>())
                      : f(__nv_bfloat16(), Int<1>());
}

}  // namespace

LnParams ln_plan(const conv_ln_desc_t& e, const DevInfo& d, bool bwd)
{
    LnParams p = {};
    const int es = e.dtype == CONV_F32 ? 4 : 2, ve = 16 / es;
    p.N = e.N;
    p.D = e.D;
    p.eps = e.eps;
    p.inv_d = float(1.0 / e.D);
    p.rms = e.rms != 0;
    p.V = e.D % ve == 0 ? ve : e.D % 2 == 0 ? 2 : 1;
    p.vecs = e.D / p.V;
    const int64_t room = int64_t(d.sms) * 2048;  // threads
    const int most_nv = bwd ? 16 / p.V : 8;
    // Vectors of a thread: in the backward as few as a team of 256 can do with (a thread keeps two sums a column), in
    // the forward as many as 4, by which a row of a warp needs no barrier.
    int nv = 1;
    while (nv < most_nv && (bwd ? p.vecs > nv * 256 : nv < 4 ? p.vecs > nv * 32 : p.vecs > nv * 256)) nv *= 2;
    p.NV = nv;
    const int need = (p.vecs + nv - 1) / nv;
    if (need > (bwd ? LN_MOST_BWD : LN_MOST)) {
        p.NV = 0;
        p.TL = LN_MOST;
        p.teams = 1;
        p.blocks = int(std::min<int64_t>(e.N, d.sms * 2));
        return p;
    }
    if (need <= 32) {
        p.TL = 1;
        while (p.TL < need) p.TL *= 2;
        p.teams = 256 / p.TL;
    } else {
        p.TL = (need + 31) / 32 * 32;
        p.teams = 1;
    }
    p.R = bwd ? ln_rows(es, p.V, p.NV) : 1;
    const int threads = p.TL * p.teams;
    const int64_t blocks = (e.N + int64_t(p.teams) * p.R - 1) / (int64_t(p.teams) * p.R);
    // The forward: as many blocks as the SMs hold threads for.  The backward: as its registers allow, 128 a thread or 64.
    const int per_sm = std::max(1, (p.NV * p.V * p.R <= 8 ? 1024 : 512) / threads);
    p.blocks = int(std::max<int64_t>(1, std::min(blocks, bwd ? int64_t(d.sms) * per_sm : room / threads)));
    if (bwd) p.flush = e.N > int64_t(p.blocks) * p.teams * LN_FLUSH;
    return p;
}

namespace {

int ln_smem(const LnParams& p)
{
    const int threads = p.TL * p.teams;
    return std::max(p.flush ? 2 * (p.NV * p.V + 1) / 2 * 2 * threads * 4 : 0, p.teams > 1 ? threads / 32 * 2 * p.D * 4 : 0);
}

// The blocks of columns and rows of a long row's second kernel.
dim3 ln_columns_grid(const LnParams& p, const DevInfo& d)
{
    const int64_t x = (int64_t(p.vecs) + LN_COLUMNS - 1) / LN_COLUMNS;
    const int64_t y = std::max<int64_t>(1, std::min<int64_t>(p.N, (d.sms * 8 + x - 1) / x));
    return dim3(unsigned(x), unsigned(y));
}

}  // namespace

cudaError_t run_ln_fwd(const conv_ln_desc_t& e, const DevInfo& d, const void* x, const void* residual, const void* gamma,
                       const void* beta, void* y, void* total, float* mean, float* rstd, cudaStream_t s)
{
    const LnParams p = ln_plan(e, d, false);
    return ln_types(p, e.dtype, [&](auto t, auto v) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value;
        auto go = [&](auto kern) {
            return launch_ex(kern, dim3(p.blocks), dim3(p.TL * p.teams), 0, s, 1, true, p, static_cast<const T*>(x),
                             static_cast<const T*>(residual), static_cast<const T*>(gamma), static_cast<const T*>(beta),
                             static_cast<T*>(y), static_cast<T*>(total), mean, rstd);
        };
        switch (p.NV) {
            case 1: return go(ln_fwd_kernel<T, V, 1>);
            case 2: return go(ln_fwd_kernel<T, V, 2>);
            case 4: return go(ln_fwd_kernel<T, V, 4>);
            case 8: return go(ln_fwd_kernel<T, V, 8>);
            default: return go(ln_fwd_long<T, V>);
        }
    });
}

size_t ln_bwd_workspace(const conv_ln_desc_t& e, const DevInfo& d)
{
    if (e.N == 0) return 0;
    const LnParams p = ln_plan(e, d, true);
    if (p.NV > 0) return size_t(p.blocks) * 2 * size_t(e.D) * 4;
    return (size_t(e.N) * 8 + 15) / 16 * 16 + size_t(ln_columns_grid(p, d).y) * 2 * size_t(e.D) * 4;
}

cudaError_t run_ln_bwd(const conv_ln_desc_t& e, const DevInfo& d, const void* x, const void* dy, const void* gamma,
                       const float* mean, const float* rstd, const void* dtotal, void* dx, void* dgamma, void* dbeta,
                       void* ws, cudaStream_t s)
{
    const LnParams p = ln_plan(e, d, true);
    return ln_types(p, e.dtype, [&](auto t, auto v) {
        using T = decltype(t);
        constexpr int V = decltype(v)::value;
        const T *px = static_cast<const T*>(x), *pdy = static_cast<const T*>(dy), *pg = static_cast<const T*>(gamma);
        const T* pt = static_cast<const T*>(dtotal);
        T* pdx = static_cast<T*>(dx);
        float* part = static_cast<float*>(ws);
        int parts = e.N > 0 ? p.blocks : 0;
        cudaError_t err = cudaSuccess;
        if (e.N > 0 && p.NV > 0) {
            auto go = [&](auto nv) {
                constexpr int NV = decltype(nv)::value;
                if constexpr (NV * V <= 16) {
                    constexpr auto kern = ln_bwd_kernel<T, V, NV, ln_rows(sizeof(T), V, NV)>;
                    const int smem = ln_smem(p);
                    if (const cudaError_t bad = ensure_smem<kern>(smem); bad != cudaSuccess) return bad;
                    return launch_ex(kern, dim3(p.blocks), dim3(p.TL * p.teams), smem, s, 1, true, p, px, pdy, pg, mean,
                                     rstd, pt, pdx, dgamma ? part : static_cast<float*>(nullptr));
                } else {
                    return cudaErrorInvalidValue;
                }
            };
            err = p.NV == 1   ? go(Int<1>())
                  : p.NV == 2 ? go(Int<2>())
                  : p.NV == 4 ? go(Int<4>())
                  : p.NV == 8 ? go(Int<8>())
                              : go(Int<16>());
        } else if (e.N > 0) {
            float2* sums = static_cast<float2*>(ws);
            part += (size_t(e.N) * 8 + 15) / 16 * 4;
            const dim3 grid = ln_columns_grid(p, d);
            parts = int(grid.y);
            err = launch_ex(ln_bwd_rows<T, V>, dim3(p.blocks), dim3(p.TL), 0, s, 1, true, p, px, pdy, pg, mean, rstd, sums);
            if (err != cudaSuccess) return err;
            err = launch_ex(ln_bwd_columns<T, V>, grid, dim3(LN_COLUMNS), 0, s, 1, true, p, px, pdy, pg, mean, rstd, pt,
                            static_cast<const float2*>(sums), pdx, dgamma ? part : static_cast<float*>(nullptr));
        }
        if (err != cudaSuccess || !dgamma) return err;
        const int64_t columns = int64_t(e.D) * (dbeta ? 2 : 1);
        return launch_ex(ln_params_kernel<T>, dim3(unsigned((columns + 31) / 32)), dim3(1024), 0, s, 1, true,
                         static_cast<const float*>(part), parts, e.D, static_cast<T*>(dgamma), static_cast<T*>(dbeta));
    });
}

}  // namespace igc
