// kernels_ln.cu -- layer norm of rows, of a residual sum where one is given:
//   s = x + residual (kept as T)      y = (s - mean) rstd gamma + beta
//   dx = rstd (e - m1 - xhat m2) + dtotal,  e = dy gamma,  m1 = mean of e,  m2 = mean of e xhat
//   dgamma = sum over the rows of dy xhat      dbeta = sum over the rows of dy
// (the form without a mean: mean, m1 and beta are 0).
//
// Bound by memory: a row is read once and held in the registers of a team, from one thread to 16
// warps; mean and squared deviations are two passes over the registers.  Blocks stay and take rows in turn.  In
// the backward a thread keeps its columns' sums of dgamma and dbeta over all rows of its team, the
// block's go to the workspace and a second kernel adds those: an order that the sizes fix.
// Where D is no multiple of 16 bytes, rows begin anywhere, but every VE-th row (VE values are 16 bytes)
// alike: a team's rows are a multiple of VE apart, so that it reads them all by the same whole vectors of memory
// and a thread's columns stay its own.  The first and the last vector hold values of the rows beside it,
// which are cut off as they come in and never written.
// Rows that no team holds are read again for each pass.  Forward rows that take eight vectors a thread (above
// 8192 fp32 or 16384 bf16 values) are held in part by local memory: 64 registers spill 280 to 810 bytes a thread.
//
// Measured, with the share of the floor (each array once) at the measured copy's bandwidth: 32768 x 1024 bf16
// forward 46.6 us (85 %), backward 48.3 (82 %, of it 7 the columns' sums), 6001 x 1430 fp32 backward without a mean
// 25.0 (61 %: 304 blocks of one team of 192 threads, 12 warps an SM at 0.57 issued a slot, then the columns' sums), 2000 x 16384
// bf16 backward 93 (42 %: read twice), 2000 x 12288 fp32 forward 109 (53 %) and 2000 x 24576 bf16 143 (40 %: both spill), 2000 x
// 40000 bf16 114 (83 %: read three times, mostly from L2).
#include <algorithm>

#include "gn_common.cuh"
#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int LN_MOST = 512;     // threads of a team
constexpr int LN_LONG = 1024;    // threads a row that no team holds
constexpr int LN_SUMS = 128;     // floats: two sums of four rows of each warp
constexpr int LN_FLUSH = 256;    // rows that are added to each other in one chain

template <typename T> constexpr int ln_ve() { return 16 / int(sizeof(T)); }

// Rows a team of the backward takes at once: 192 bytes a thread of x, dy and dtotal.
constexpr int ln_rows(int NV) { return 4 / NV; }

// A thread's place: teams of TL threads, each a row at a time, `rows` apart.
struct LnAt {
    int lane, team, TL, teams, warps;  // warps of a team of more than one, else 1
    int64_t first, rows;               // the team's first row; rows to its next
    __device__ __forceinline__ explicit LnAt(const LnParams& p)
    {
        TL = p.TL;
        teams = p.teams;
        lane = teams > 1 ? int(threadIdx.x) & (TL - 1) : int(threadIdx.x);
        team = teams > 1 ? int(threadIdx.x) / TL : 0;
        warps = TL > 32 ? TL / 32 : 1;
        first = int64_t(blockIdx.x) * teams + team;
        rows = int64_t(gridDim.x) * teams;
    }
};

// A thread's NV vectors of its team's rows.  EDGE: rows do not all begin at 16 bytes; a vector's values that
// belong to the row are the bits of `have`.
template <typename T, int NV, bool EDGE> struct LnRow {
    static constexpr int VE = ln_ve<T>(), FULL = (1 << VE) - 1;
    using Vector = Vec<T, VE>;
    int off;         // elements of vector 0 that belong to the row before
    uint32_t have[EDGE ? NV : 1];
    int lane, TL, vecs;
    int64_t end;     // elements of the array
    __device__ __forceinline__ LnRow(const LnParams& p, const LnAt& q) : lane(q.lane), TL(q.TL), end(p.N * p.D)
    {
        off = EDGE ? int(uint64_t(q.first) * uint64_t(p.D) % VE) : 0;
        vecs = (off + p.D + VE - 1) / VE;
        if constexpr (EDGE) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = (lane + i * TL) * VE - off;  // the vector's first column
                const int lo = max(0, -at), hi = min(VE, p.D - at);
                have[i] = hi > lo ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
            }
        }
    }
    __device__ __forceinline__ bool in(int i) const { return EDGE ? have[EDGE ? i : 0] != 0 : lane + i * TL < vecs; }
    __device__ __forceinline__ bool whole(int i) const { return !EDGE || have[EDGE ? i : 0] == FULL; }
    __device__ __forceinline__ bool has(int i, int v) const { return !EDGE || (have[EDGE ? i : 0] >> v & 1u); }
    __device__ __forceinline__ int column(int i) const { return (lane + i * TL) * VE - off; }
    // Element of the array that vector i of a row begins with.
    __device__ __forceinline__ int64_t at(int64_t row, int D, int i) const
    {
        return row * D - off + int64_t(lane + i * TL) * VE;
    }
    // Vector i with what lies beside the row in it; cut() makes that 0, once all loads are on their way.
    __device__ __forceinline__ void load(Vector& r, const T* a, int64_t at, int i) const
    {
        if (whole(i) || at + VE <= end) {
            r.load(a + at);
        } else {  // the array's last vector
            float f[VE];
#pragma unroll
            for (int v = 0; v < VE; ++v) f[v] = has(i, v) ? Elem<T>::ld(a + at + v) : 0.f;
            r.set(f);
        }
    }
    __device__ __forceinline__ void cut(Vector& r, int i) const
    {
        if (whole(i)) return;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) r.r.w[k] = has(i, k) ? r.r.w[k] : 0u;
            else r.r.w[k] &= (has(i, 2 * k) ? 0xFFFFu : 0u) | (has(i, 2 * k + 1) ? 0xFFFF0000u : 0u);
        }
    }
    __device__ __forceinline__ void cut(Vector (&a)[NV]) const
    {
        if constexpr (EDGE)
#pragma unroll
            for (int i = 0; i < NV; ++i) cut(a[i], i);
    }
    // The same vector on its way to shared memory; what lies behind the array is not read.
    __device__ __forceinline__ void copy(uint32_t to, const T* a, int64_t at, int i) const
    {
        int bytes = 16;
        if (EDGE && !whole(i) && at + VE > end) bytes = int(end - at) * int(sizeof(T));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(a + at), "r"(bytes) : "memory");
    }
    __device__ __forceinline__ void store(T* a, int64_t at, int i, const Vector& r) const
    {
        if (whole(i)) {
            r.store(a + at);
        } else {
#pragma unroll
            for (int v = 0; v < VE; ++v)
                if (has(i, v)) Elem<T>::st(a + at + v, r.get(v));
        }
    }
    // A parameter of the thread's columns, `other` where there is none.
    __device__ __forceinline__ void params(Vector& r, const T* a, int i, float other) const
    {
        float f[VE];
#pragma unroll
        for (int v = 0; v < VE; ++v) f[v] = other;
        r.set(f);
        if (!a || !in(i)) return;
        if constexpr (!EDGE) {
            r.load(a + column(i));
        } else {
#pragma unroll
            for (int v = 0; v < VE; ++v)
                if (has(i, v)) f[v] = Elem<T>::ld(a + column(i) + v);
            r.set(f);
        }
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

template <typename T, int NV, bool EDGE>
__global__ void __launch_bounds__(LN_MOST, 2)
ln_fwd_kernel(const __grid_constant__ LnParams p, const T* x, const T* residual, const T* gamma, const T* beta, T* y,
              T* total, float* mean, float* rstd)
{
    __shared__ float sm[2][32];
    constexpr int VE = ln_ve<T>();
    using Vector = Vec<T, VE>;
    const LnAt q(p);
    const LnRow<T, NV, EDGE> w(p, q);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    // Whole vectors of gamma and beta are read again for each row, from L1; where rows begin anywhere, from copies in
    // shared memory that begin as the rows of the block's team, or of its VE-th team each, do.
    extern __shared__ __align__(16) uint8_t columns[];
    const int wide = (p.D + 2 * VE - 1) / VE * VE, copies = EDGE ? min(q.teams, VE) : 0;
    T* const mine = reinterpret_cast<T*>(columns) + (q.team % VE) * 2 * wide;
    if constexpr (EDGE) {
        for (int k = int(threadIdx.x); k < copies * wide; k += int(blockDim.x)) {
            const int copy = k / wide, e = k % wide;
            const int c = e - int(uint64_t(int64_t(blockIdx.x) * q.teams + copy) * uint64_t(p.D) % VE);
            T* to = reinterpret_cast<T*>(columns) + copy * 2 * wide + e;
            const bool there = c >= 0 && c < p.D;
            Elem<T>::st(to, there ? (gamma ? Elem<T>::ld(gamma + c) : 1.f) : 0.f);
            Elem<T>::st(to + wide, there && beta ? Elem<T>::ld(beta + c) : 0.f);
        }
        __syncthreads();
    }
    for (int64_t row = q.first; row - q.team < p.N; row += q.rows) {
        const bool on = row < p.N;
        Vector a[NV];
        float f[NV][VE];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            a[i].zero();
            if (on && w.in(i)) w.load(a[i], x, w.at(row, p.D, i), i);
        }
        if (residual) {
            Vector r[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                r[i].zero();
                if (on && w.in(i)) w.load(r[i], residual, w.at(row, p.D, i), i);
            }
            w.cut(a);
            w.cut(r);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float s[VE];
#pragma unroll
                for (int v = 0; v < VE; ++v) s[v] = a[i].get(v) + r[i].get(v);
                a[i].set(s);
                if (on && w.in(i)) w.store(total, w.at(row, p.D, i), i, a[i]);
            }
        } else {
            w.cut(a);
        }
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < VE; ++v) {
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
#pragma unroll
            for (int v = 0; v < VE; ++v) f[i][v] -= m;
            if (!w.in(i)) continue;
            if (w.whole(i)) {
#pragma unroll
                for (int v = 0; v < VE; ++v) sq[0] += f[i][v] * f[i][v];
            } else {
#pragma unroll
                for (int v = 0; v < VE; ++v)
                    if (w.has(i, v)) sq[0] += f[i][v] * f[i][v];
            }
        }
        if (p.rms && q.warps > 1) __syncthreads();  // the sums of the row before have been read
        ln_sum(q, sq, sm[1]);
        const float r = __frsqrt_rn(sq[0] * p.inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on || !w.in(i)) continue;
            Vector gi, bi, o;
            if constexpr (EDGE) {
                gi.load(mine + (q.lane + i * q.TL) * VE);
                bi.load(mine + wide + (q.lane + i * q.TL) * VE);
            } else {
                if (gamma) gi.load(gamma + w.column(i));
                if (beta) bi.load(beta + w.column(i));
            }
            float out[VE];
#pragma unroll
            for (int v = 0; v < VE; ++v)
                out[v] = fmaf(f[i][v] * r, EDGE || gamma ? gi.get(v) : 1.f, EDGE || beta ? bi.get(v) : 0.f);
            o.set(out);
            w.store(y, w.at(row, p.D, i), i, o);
        }
        if (on && q.lane == 0) {
            if (mean) mean[row] = m;
            if (rstd) rstd[row] = r;
        }
    }
}

// A thread's sums over the vectors of a row that no team holds: f(j, part) adds vector j's.  An addition may be off by
// half a step, each the same way, so a chain has 256 vectors at most; CHAINS: where a thread has more, its chains
// are added to each other in 64 bits.  (A row of 2^29 - 1 values alike was one of 524288, off by 0.4 %.  In one
// kernel for both the registers of the longer form cost rows of any length: 2000 x 40000 bf16 forward 114 us, 160 so.)
constexpr int LN_CHAIN = 256;
template <bool CHAINS, int K, class F>
__device__ __forceinline__ void ln_long_sums(const LnAt& q, int vecs, float (&sum)[K], F&& f)
{
#pragma unroll
    for (int k = 0; k < K; ++k) sum[k] = 0.f;
    if constexpr (!CHAINS) {
        for (int j = q.lane; j < vecs; j += q.TL) f(j, sum);
    } else {
        double all[K] = {};
        const int chain = LN_CHAIN * q.TL;
        for (int from = q.lane; from < vecs; from += chain) {
            float part[K] = {};
            const int to = min(vecs, from + chain);
            for (int j = from; j < to; j += q.TL) f(j, part);
#pragma unroll
            for (int k = 0; k < K; ++k) all[k] += double(part[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) sum[k] = float(all[k]);
    }
}

// A block a row, of any length: the row is read again for each pass.
template <typename T, int V, bool CHAINS>
__global__ void __launch_bounds__(LN_LONG)
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
        float sum[1];
        ln_long_sums<CHAINS>(q, p.vecs, sum, [&](int j, float (&part)[1]) {
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
            part[0] += t;
        });
        float m = 0.f;
        if (!p.rms) {
            ln_sum(q, sum, sm[0]);
            m = sum[0] * p.inv_d;
        }
        float sq[1];
        ln_long_sums<CHAINS>(q, p.vecs, sq, [&](int j, float (&part)[1]) {
            Vec<T, V> a;
            a.load(s + at + int64_t(j) * V);
            float t = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) t += (a.get(v) - m) * (a.get(v) - m);
            part[0] += t;
        });
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

// Columns v and v + 1 of a vector.
template <typename T, int VE> __device__ __forceinline__ float2 pick(const Vec<T, VE>& a, int v)
{
    return make_float2(a.get(v), a.get(v + 1));
}

// R rows of a team at a time: neighbours, where rows begin at 16 bytes.  A thread's own vectors of the next rows are on
// their way to its own places in shared memory while these are worked on: no barrier, and few registers.  What
// both passes need is read there twice.  part: [block][dgamma, dbeta][D], or NULL.
template <typename T, int NV, bool EDGE>
__global__ void __launch_bounds__(LN_MOST)
ln_bwd_kernel(const __grid_constant__ LnParams p, const T* x, const T* dy, const T* gamma, const float* mean,
              const float* rstd, const T* dtotal, T* dx, float* part)
{
    // the rows' sums, twice in turn; [stage][row][x, dy, dtotal][NV][thread] vectors; what the chains of additions have
    // left so far, where a block has several teams (one team's goes to the workspace)
    extern __shared__ __align__(16) float dyn[];
    constexpr int VE = ln_ve<T>(), CPT = NV * VE, P = CPT / 2, R = ln_rows(NV);
    float* const tiles = dyn + 2 * LN_SUMS;
    using Vector = Vec<T, VE>;
    const LnAt q(p);
    const LnRow<T, NV, EDGE> w(p, q);
    const uint32_t stages = tc::smem_u32(tiles) + threadIdx.x * 16;
    const int step = int(blockDim.x) * 16, stage_bytes = R * 3 * NV * step;
    float2* const left = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(tiles) + 2 * stage_bytes);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float2 dg[P], db[P];
    Vector g[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) w.params(g[i], gamma, i, 1.f);
#pragma unroll
    for (int c = 0; c < P; ++c) dg[c] = db[c] = both(0.f);
    float* const to = part + int64_t(blockIdx.x) * 2 * p.D;
    if (p.flush && q.teams > 1)
        for (int k = 0; k < 2 * P; ++k) left[k * int(blockDim.x) + int(threadIdx.x)] = both(0.f);
    bool begun = false;  // there are sums in the workspace
    auto hand_over = [&] {
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            if (!w.in(c / VE) || !w.has(c / VE, c % VE)) continue;
            float *a = to + w.column(c / VE) + c % VE, *b = a + p.D;
            const float u = c & 1 ? dg[c / 2].y : dg[c / 2].x, v = c & 1 ? db[c / 2].y : db[c / 2].x;
            *a = begun ? *a + u : u;
            *b = begun ? *b + v : v;
        }
        begun = true;
    };
    auto flush = [&] {
        if (q.teams == 1) {
            hand_over();
#pragma unroll
            for (int c = 0; c < P; ++c) dg[c] = db[c] = both(0.f);
            return;
        }
#pragma unroll
        for (int c = 0; c < P; ++c) {
            float2* a = left + 2 * c * int(blockDim.x) + int(threadIdx.x);
            a[0] = add2(a[0], dg[c]);
            a[blockDim.x] = add2(a[blockDim.x], db[c]);
            dg[c] = db[c] = both(0.f);
        }
    };
    const int64_t next = EDGE ? q.rows : 1, hop = next * p.D;  // from one of the R rows to the next
    float m_next[R], r_next[R];
    auto fetch = [&](int64_t row0, uint32_t to) {
        const int64_t at0 = w.at(row0, p.D, 0);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            m_next[k] = r_next[k] = 0.f;
            if (row0 + k * next >= p.N) continue;
            if (mean) m_next[k] = mean[row0 + k * next];
            r_next[k] = rstd[row0 + k * next];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!w.in(i)) continue;
                const int64_t at = at0 + k * hop + i * q.TL * VE;
                const uint32_t slot = to + uint32_t((k * 3 * NV + i) * step);
                w.copy(slot, x, at, i);
                w.copy(slot + uint32_t(NV * step), dy, at, i);
                if (dtotal) w.copy(slot + uint32_t(2 * NV * step), dtotal, at, i);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto read = [&](Vector& r, uint32_t slot, int i) {
        const int4 u = tc::lds128(slot);
        r.r.w[0] = uint32_t(u.x); r.r.w[1] = uint32_t(u.y); r.r.w[2] = uint32_t(u.z); r.r.w[3] = uint32_t(u.w);
        if (EDGE) w.cut(r, i);
    };
    const int64_t first = EDGE ? q.first : q.first * R, ahead = R * q.rows;
    fetch(first, stages);
    int turn = 0, chain = 0;
    for (int64_t row0 = first; row0 - (EDGE ? 1 : R) * q.team < p.N; row0 += ahead, turn ^= 1) {
        const uint32_t now = stages + uint32_t(turn * stage_bytes);
        float m[R], r[R], sums[2 * R];
        uint32_t on = 0;  // rows that are there
#pragma unroll
        for (int k = 0; k < R; ++k) {
            m[k] = m_next[k];
            r[k] = r_next[k];
            if (row0 + k * next < p.N) on |= 1u << k;
        }
        fetch(row0 + ahead, stages + uint32_t((turn ^ 1) * stage_bytes));
        asm volatile("cp.async.wait_group 1;" ::: "memory");
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!(on >> k & 1u) || !w.in(i)) continue;
                Vector a, d;
                read(a, now + uint32_t((k * 3 * NV + i) * step), i);
                read(d, now + uint32_t((k * 3 * NV + NV + i) * step), i);  // (0 where the row is not)
#pragma unroll
                for (int v = 0; v < VE; v += 2) {
                    const int c = (i * VE + v) / 2;
                    const float2 xh = mul2(add2(pick(a, v), both(-m[k])), both(r[k])), y = pick(d, v);
                    const float2 e = mul2(y, pick(g[i], v));
                    s1 = add2(s1, e);
                    s2 = fma2(e, xh, s2);
                    dg[c] = fma2(y, xh, dg[c]);
                    db[c] = add2(db[c], y);
                }
            }
            sums[2 * k] = s1.x + s1.y;
            sums[2 * k + 1] = s2.x + s2.y;
        }
        ln_sum(q, sums, dyn + turn * LN_SUMS);
        const int64_t at0 = w.at(row0, p.D, 0);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const float m1 = p.rms ? 0.f : sums[2 * k] * p.inv_d, m2 = sums[2 * k + 1] * p.inv_d;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!(on >> k & 1u) || !w.in(i)) continue;
                Vector a, d, t;
                read(a, now + uint32_t((k * 3 * NV + i) * step), i);
                read(d, now + uint32_t((k * 3 * NV + NV + i) * step), i);
                t.zero();
                if (dtotal) read(t, now + uint32_t((k * 3 * NV + 2 * NV + i) * step), i);
                float o[VE];
#pragma unroll
                for (int v = 0; v < VE; v += 2) {
                    const float2 xh = mul2(add2(pick(a, v), both(-m[k])), both(r[k]));
                    const float2 e = mul2(pick(d, v), pick(g[i], v));
                    const float2 u = fma2(both(r[k]), fma2(xh, both(-m2), add2(e, both(-m1))), pick(t, v));
                    o[v] = u.x;
                    o[v + 1] = u.y;
                }
                a.set(o);
                w.store(dx, at0 + k * hop + i * q.TL * VE, i, a);
            }
        }
        chain += R;
        if (p.flush && part && chain >= LN_FLUSH) {
            flush();
            chain = 0;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!part) return;
    if (q.teams == 1) {
        hand_over();
        return;
    }
    if (p.flush) {
        flush();
#pragma unroll
        for (int c = 0; c < P; ++c) {
            const float2* a = left + 2 * c * int(blockDim.x) + int(threadIdx.x);
            dg[c] = a[0];
            db[c] = a[blockDim.x];
        }
    }
    // Teams of a warp and less: one team of each warp after the other into the warp's columns (teams begin their
    // vectors at other columns, where rows do), then over the warps.
    const int warp = int(threadIdx.x) >> 5, warps = int(blockDim.x) >> 5, of_warp = (int(threadIdx.x) & 31) / q.TL;
    float* at = tiles + warp * 2 * p.D;  // over the stages
    __syncthreads();
    for (int c = int(threadIdx.x) & 31; c < 2 * p.D; c += 32) at[c] = 0.f;
    for (int k = 0; k < 32 / q.TL; ++k) {
        __syncwarp();
        if (k != of_warp) continue;
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const int col = w.column(c / VE) + c % VE;
            if (w.in(c / VE) && w.has(c / VE, c % VE)) {
                at[col] += c & 1 ? dg[c / 2].y : dg[c / 2].x;
                at[p.D + col] += c & 1 ? db[c / 2].y : db[c / 2].x;
            }
        }
    }
    __syncthreads();
    for (int c = int(threadIdx.x); c < 2 * p.D; c += int(blockDim.x)) {
        float s = 0.f;
        for (int k = 0; k < warps; ++k) s += tiles[k * 2 * p.D + c];
        to[c] = s;
    }
}

// ---- rows that no team holds: the rows' sums, then columns of all rows -------------------------
template <typename T, int V, bool CHAINS>
__global__ void __launch_bounds__(LN_LONG)
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
        float s[2];
        ln_long_sums<CHAINS>(q, p.vecs, s, [&](int j, float (&part)[2]) {
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
            part[0] += s1;
            part[1] += s2;
        });
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

// Calls f(T(), EDGE) for a plan with teams.
template <class F> cudaError_t ln_edge(const LnParams& p, int dt, F&& f)
{
    if (dt == DT_F32) return p.edge ? f(float(), std::true_type()) : f(float(), std::false_type());
    return p.edge ? f(__nv_bfloat16(), std::true_type()) : f(__nv_bfloat16(), std::false_type());
}
// Calls f(CHAINS) for a plan without.
template <class F> cudaError_t ln_chains(const LnParams& p, F&& f)
{
    return p.vecs > LN_CHAIN * LN_LONG ? f(std::true_type()) : f(std::false_type());
}
// Calls f(T(), V) for such a plan.
template <class F> cudaError_t ln_long(const LnParams& p, int dt, F&& f)
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
    p.edge = e.D % ve != 0;
    const int vecs = int((int64_t(e.D) + ve - 1) / ve) + (p.edge ? 1 : 0);
    // Vectors of a thread.  Forward: four, where a row has as many, and eight for the longest.  Backward, where a thread
    // keeps two sums a column: eight columns, sixteen for the longest rows.
    int nv = 1;
    if (!bwd) {
        while (nv < 4 && nv * 2 <= vecs) nv *= 2;
        if (vecs > 4 * LN_MOST) nv = 8;
        // Teams of several warps that begin anywhere: two spill nothing in bf16, and more threads share a block's copies of
        // gamma and beta (8001 x 1431 30.4 us with four, 26.4 with two; 4001 x 5001 46.0 and 42.7; one warp, 20000 x 770, 36.3 and
        // 38.5; fp32 3001 x 2750 29.3 and 35.4).
        if (p.edge && es == 2 && vecs > 4 * 32 && vecs <= 2 * LN_MOST) nv = 2;
    } else {
        nv = es == 2 || vecs < 2 ? 1 : 2;
        if (vecs > nv * LN_MOST) nv *= 2;
    }
    const int need = (vecs + nv - 1) / nv;
    if (need > LN_MOST) {
        p.V = e.D % ve == 0 ? ve : e.D % 2 == 0 ? 2 : 1;
        p.vecs = e.D / p.V;
        p.TL = LN_LONG;
        p.teams = 1;
        p.blocks = int(std::max<int64_t>(1, std::min<int64_t>(e.N, d.sms * 2)));
        return p;
    }
    p.NV = nv;
    if (need <= 32) {
        p.TL = 1;
        while (p.TL < need) p.TL *= 2;
        p.teams = 256 / p.TL;
    } else {
        p.TL = (need + 31) / 32 * 32;
        p.teams = 1;
    }
    p.R = bwd ? ln_rows(nv) : 1;
    const int threads = p.TL * p.teams;
    const int64_t rows = int64_t(p.teams) * p.R, blocks = (e.N + rows - 1) / rows;
    // Twice as many blocks as the SMs hold at once with 64 registers a thread; in the backward as many as they do with 128.
    // Where rows begin anywhere, each makes its copies of gamma and beta first: as many as the SMs hold (6001 x 1430 fp32
    // 32.6 us with twice as many, 29.5 with these, 37.8 with half of them).  A multiple of what makes a team's rows begin alike.
    const int per_sm = std::max(1, (bwd ? 512 : p.edge ? 1024 : 2048) / threads);
    p.blocks = int(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t(d.sms) * per_sm)));
    if (p.edge && p.teams % ve != 0) p.blocks = (p.blocks + ve - 1) / ve * ve;
    if (bwd) p.flush = e.N > int64_t(p.blocks) * p.teams * LN_FLUSH;
    return p;
}

namespace {

int ln_smem(const LnParams& p, int ve)
{
    const int threads = p.TL * p.teams, stages = 2 * p.R * 3 * p.NV * threads * 16;
    return 8 * LN_SUMS + std::max(stages + (p.flush && p.teams > 1 ? 2 * p.NV * ve * threads * 4 : 0), p.teams > 1 ? threads / 32 * 2 * p.D * 4 : 0);
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
    const int ve = e.dtype == CONV_F32 ? 4 : 8;
    const int smem = p.edge && p.NV > 0 ? std::min(p.teams, ve) * 2 * ((e.D + 2 * ve - 1) / ve * ve) * (16 / ve) : 0;
    auto go = [&](auto kern, auto t) {
        using T = decltype(t);
        return launch_ex(kern, dim3(p.blocks), dim3(p.TL * p.teams), smem, s, 1, true, p, static_cast<const T*>(x),
                         static_cast<const T*>(residual), static_cast<const T*>(gamma), static_cast<const T*>(beta),
                         static_cast<T*>(y), static_cast<T*>(total), mean, rstd);
    };
    if (p.NV == 0)
        return ln_long(p, e.dtype, [&](auto t, auto v) {
            return ln_chains(p, [&](auto chains) {
                return go(ln_fwd_long<decltype(t), decltype(v)::value, decltype(chains)::value>, t);
            });
        });
    return ln_edge(p, e.dtype, [&](auto t, auto edge) {
        using T = decltype(t);
        constexpr bool EDGE = decltype(edge)::value;
        auto team = [&](auto nv) {
            constexpr auto kern = ln_fwd_kernel<T, decltype(nv)::value, EDGE>;
            const cudaError_t bad = ensure_smem<kern>(smem > 0 ? smem + 1024 : 0);  // (and the static part)
            return bad != cudaSuccess ? bad : go(kern, t);
        };
        if constexpr (!EDGE)  // (rows that begin anywhere have two vectors at least)
            if (p.NV == 1) return team(Int<1>());
        return p.NV == 2 ? team(Int<2>()) : p.NV == 4 ? team(Int<4>()) : team(Int<8>());
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
    float* part = static_cast<float*>(ws);
    int parts = e.N > 0 ? p.blocks : 0;
    cudaError_t err = cudaSuccess;
    if (e.N > 0 && p.NV > 0) {
        err = ln_edge(p, e.dtype, [&](auto t, auto edge) {
            using T = decltype(t);
            auto go = [&](auto nv) {
                constexpr int NV = decltype(nv)::value, ES = int(sizeof(T));
                constexpr auto kern = ln_bwd_kernel<T, NV, decltype(edge)::value>;
                const int smem = ln_smem(p, 16 / ES);
                if (const cudaError_t bad = ensure_smem<kern>(smem); bad != cudaSuccess) return bad;
                return launch_ex(kern, dim3(p.blocks), dim3(p.TL * p.teams), smem, s, 1, true, p,
                                 static_cast<const T*>(x), static_cast<const T*>(dy), static_cast<const T*>(gamma), mean,
                                 rstd, static_cast<const T*>(dtotal), static_cast<T*>(dx),
                                 dgamma ? part : static_cast<float*>(nullptr));
            };
            if constexpr (sizeof(T) == 4)
                if (p.NV == 4) return go(Int<4>());
            if constexpr (sizeof(T) == 2 || !decltype(edge)::value)  // (as in the forward)
                if (p.NV == 1) return go(Int<1>());
            return go(Int<2>());
        });
    } else if (e.N > 0) {
        float2* sums = static_cast<float2*>(ws);
        part += (size_t(e.N) * 8 + 15) / 16 * 4;
        const dim3 grid = ln_columns_grid(p, d);
        parts = int(grid.y);
        err = ln_long(p, e.dtype, [&](auto t, auto v) {
            using T = decltype(t);
            constexpr int V = decltype(v)::value;
            const T *px = static_cast<const T*>(x), *pdy = static_cast<const T*>(dy), *pg = static_cast<const T*>(gamma);
            const cudaError_t bad = ln_chains(p, [&](auto chains) {
                return launch_ex(ln_bwd_rows<T, V, decltype(chains)::value>, dim3(p.blocks), dim3(p.TL), 0, s, 1, true, p, px,
                                 pdy, pg, mean, rstd, sums);
            });
            if (bad != cudaSuccess) return bad;
            return launch_ex(ln_bwd_columns<T, V>, grid, dim3(LN_COLUMNS), 0, s, 1, true, p, px, pdy, pg, mean, rstd,
                             static_cast<const T*>(dtotal), static_cast<const float2*>(sums), static_cast<T*>(dx),
                             dgamma ? part : static_cast<float*>(nullptr));
        });
    }
    if (err != cudaSuccess || !dgamma) return err;
    const dim3 grid(unsigned((int64_t(e.D) * (dbeta ? 2 : 1) + 31) / 32));
    auto add = [&](auto t) {
        using T = decltype(t);
        return launch_ex(ln_params_kernel<T>, grid, dim3(1024), 0, s, 1, true, static_cast<const float*>(part), parts, e.D,
                         static_cast<T*>(dgamma), static_cast<T*>(dbeta));
    };
    return e.dtype == CONV_F32 ? add(float()) : add(__nv_bfloat16());
}

}  // namespace igc
