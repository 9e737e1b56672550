// kernels_gn_cluster.cu -- group norm of groups too large for a team of lanes, kept on chip: a
// thread-block cluster of S blocks holds a unit (NCHW: one group of a sample; NHWC: a sample's
// positions of a window of whole groups) in its shared memory, so x (and dy) are read from
// memory once.  A thread copies its own vectors asynchronously into its own slots and is the
// only one to read them: the tile is an extension of its registers and needs no barrier.  The
// blocks exchange their groups' partial results through distributed shared memory, once.
//
// Bound by memory: the tile is written once and read three times (forward: sum, squares, result)
// or twice (backward: sums, result) at shared-memory speed, about a third of its rate when HBM
// is saturated; two blocks an SM (where the unit allows) let one load while the other computes.
#include "gn_common.cuh"

namespace igc {

namespace {

constexpr int GC_MAX_CG = 2048;            // channels of a group (NCHW: their gammas sit in shared memory)
constexpr int GC_TWO = 110 * 1024;         // shared memory of a block when two share an SM
constexpr int GC_ONE = 220 * 1024;
constexpr int GC_VECS = 16;                // vectors a thread, about
constexpr int GC_THREADS = 512;

}  // namespace

// Bytes of shared memory beside the tile.
static int gc_extra(const GnCluster& q, bool bwd)
{
    if (q.nhwc && bwd) return 8 * (q.threads * q.V + q.threads + q.W + 1) + 16 * q.W + 16 * q.groups;
    if (q.nhwc) return 16 * q.threads + 8 * q.W + 16 * q.groups;
    return 4 * (2 * q.Cg + 64) + (bwd ? 8 * (q.K * q.threads + 2 * q.Cg) : 0);
}

GnCluster gn_cluster(const GnParams& p, int dt, const DevInfo& d, bool bwd)
{
    GnCluster q = {};
    const int es = dt == DT_F32 ? 4 : 2;
    // one position: both layouts are the same, and channels last reads it in wide vectors
    const bool nhwc = p.layout == CONV_LAYOUT_NHWC || p.P == 1;
    q.nhwc = nhwc;
    q.Cg = p.Cg;
    q.V = 16 / es;
    // a vector lies in two groups (NHWC) or two channels (NCHW) at most
    if (nhwc) while (p.C % q.V != 0 || q.V > p.Cg) q.V /= 2;
    else while (p.M % q.V != 0 || q.V > p.P) q.V /= 2;
    const int tiles = bwd ? 2 : 1, vb = q.V * es;
    if (p.Cg > GC_MAX_CG) return q;
    int lcm = p.Cg;
    while (lcm % q.V != 0) lcm += p.Cg;
    // NHWC: windows of whole vectors and whole groups, 64 bytes of a row (two sectors) or less.
    // Two blocks an SM come before wide rows and small clusters: a block alone on its SM waits
    // with it.
    const int widest = nhwc ? std::max(1, std::min(ceil_div(64, lcm * es), ceil_div(p.C, lcm))) : 1;
    for (const int limit : {GC_TWO, std::min(GC_ONE, d.smem_optin - 1024)})
        for (int m = widest; m >= 1; --m) {
            int64_t vecs;  // of the unit
            if (nhwc) {
                q.W = std::min(m * lcm, p.C);
                q.cols = q.W / q.V;
                q.groups = q.W / p.Cg;
                q.wins = ceil_div(p.C, q.W);
                if (q.cols > GC_THREADS) continue;
                vecs = int64_t(p.P) * q.cols;
            } else {
                q.wins = p.G;
                vecs = p.M / q.V;
                q.vecs = int(vecs);
            }
            const int64_t units = int64_t(p.B) * q.wins;
            if (units * kMaxCluster > 0x7FFFFFFF) return q;
            const int most = int(std::min<int64_t>(kMaxCluster, nhwc ? p.P : vecs / 32 + 1));
            for (int S = 1, log = 0; S <= most; S *= 2, ++log) {
                const int64_t per = (vecs + S - 1) / S;
                int T = 32;
                while (T < (bwd && limit == GC_TWO ? 256 : GC_THREADS) && per > int64_t(T) * GC_VECS) T *= 2;
                if (nhwc) while (T < q.cols) T *= 2;
                q.S = S;
                q.log_s = log;
                q.threads = T;
                q.lanes = nhwc ? T / q.cols : 1;
                const int64_t K = nhwc ? (ceil_div(p.P, S) + q.lanes - 1) / q.lanes : (per + T - 1) / T;
                if (K * T * vb * tiles > limit) continue;
                q.K = int(K);
                q.smem = q.K * T * vb * tiles + gc_extra(q, bwd);
                if (q.smem > limit) continue;
                // larger clusters while the SMs are not filled and the blocks still have a few
                // kilobytes each
                if (S * 2 <= most && units * S < 2 * d.sms && per * vb > 4096) continue;
                q.ok = true;
                return q;
            }
        }
    return q;
}

namespace {

template <int BYTES> __device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, int V> __device__ __forceinline__ void fetch_vec(unsigned char* slot, const T* src)
{
    if constexpr (sizeof(T) * V >= 4) {
        copy_async<int(sizeof(T)) * V>(tc::smem_u32(slot), src);
    } else {
        Vec<T, V> v;
        v.load(src);
        v.store(reinterpret_cast<T*>(slot));
    }
}

// The cluster barrier in two halves (the warp has to be converged for each).
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Where block r's part of n items begins (S is a power of two).
__device__ __forceinline__ int gc_cut(int n, const GnCluster& q, int r) { return int((int64_t(n) * r) >> q.log_s); }

// The unit of an NHWC block: rows [r0, r1) of its window; thread (lane, col) holds the vector
// `col` of the rows r0 + lane, r0 + lane + lanes, ...
struct GcTile {
    int b, rank, c0, W, groups, g0, lane, col, r0, r1, mine;
    int g, split;  // the group (in the window) of the vector's first channel, its channels in that group
    bool in;
    __device__ __forceinline__ GcTile(const GnParams& p, const GnCluster& q, int V)
    {
        rank = q.S > 1 ? int(tc::cluster_rank()) : 0;
        const int unit = int(blockIdx.x) / q.S;
        b = unit / q.wins;
        c0 = (unit - b * q.wins) * q.W;
        W = min(q.W, p.C - c0);
        groups = W / p.Cg;
        g0 = c0 / p.Cg;
        lane = int(threadIdx.x) / q.cols;
        col = int(threadIdx.x) - lane * q.cols;
        in = lane < q.lanes && col * V < W;
        r0 = gc_cut(p.P, q, rank);
        r1 = gc_cut(p.P, q, rank + 1);
        mine = in ? max(0, (r1 - r0 - lane + q.lanes - 1) / q.lanes) : 0;
        g = in ? col * V / p.Cg : 0;
        split = in ? min(V, (g + 1) * p.Cg - col * V) : V;
    }
};
__device__ __forceinline__ float gc_rows(const GnParams& p, const GnCluster& q, int r)
{
    return float(gc_cut(p.P, q, r + 1) - gc_cut(p.P, q, r));
}
// A vector's values as pairs; one value: (value, 0).
template <int V> constexpr int gc_pairs() { return (V + 1) / 2; }
template <typename T, int V> __device__ __forceinline__ void gc_unpack(const Vec<T, V>& v, float2 (&f)[gc_pairs<V>()])
{
#pragma unroll
    for (int h = 0; h < gc_pairs<V>(); ++h) f[h] = make_float2(v.get(2 * h), 2 * h + 1 < V ? v.get(2 * h + 1) : 0.f);
}
template <typename T, int V> __device__ __forceinline__ void gc_pack(Vec<T, V>& v, const float2 (&f)[gc_pairs<V>()])
{
    float r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
    v.set(r);
}

// ---- channels last ---------------------------------------------------------------------------
template <typename T, int V>
__global__ void __launch_bounds__(GC_THREADS, 2)
gn_cluster_fwd_nhwc(const GnParams p, const GnCluster q, const T* x, const T* gamma, const T* beta, T* y,
                    float* mean_out, float* rstd_out)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T)), H = gc_pairs<V>();
    const GcTile t(p, q, V);
    const int nt = int(blockDim.x), hop = nt * VB;
    unsigned char* slot = dyn + threadIdx.x * VB;
    float4* rec = reinterpret_cast<float4*>(dyn + size_t(q.K) * hop);  // threads x (mean, M2) of either group
    float* gs = reinterpret_cast<float*>(rec + nt);   // groups x (mean, M2) of the block, read by the others
    float* stat = gs + 2 * q.groups;                  // groups x (mean, rstd) of the unit
    float* gb = stat + 2 * q.groups;                  // W gammas, W betas
    const int64_t at = int64_t(t.b) * p.N + t.c0 + t.col * V;
    tc::grid_dep_wait();
    for (int k = 0, r = t.r0 + t.lane; k < t.mine; ++k, r += q.lanes)
        fetch_vec<T, V>(slot + k * hop, x + at + int64_t(r) * p.C);
    for (int c = threadIdx.x; c < t.W; c += nt) {
        gb[c] = gamma ? Elem<T>::ldg(gamma + t.c0 + c) : 1.f;
        gb[q.W + c] = beta ? Elem<T>::ldg(beta + t.c0 + c) : 0.f;
    }
    copy_wait();
    // The thread's mean of its values of either group, then the squares about it.
    {
        float2 s[H], mu[H];
        float m0 = 0.f, m1 = 0.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                s[h] = both(0.f);
                mu[h] = make_float2(2 * h < t.split ? -m0 : -m1, 2 * h + 1 < t.split ? -m0 : -m1);
                if (V == 1) mu[h].y = 0.f;
            }
#pragma unroll 2
            for (int k = 0; k < t.mine; ++k) {
                Vec<T, V> v;
                float2 f[H];
                v.load(reinterpret_cast<const T*>(slot + k * hop));
                gc_unpack<T, V>(v, f);
                if (pass == 0) {
#pragma unroll
                    for (int h = 0; h < H; ++h) s[h] = add2(s[h], f[h]);
                } else {
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        f[h] = add2(f[h], mu[h]);
                        s[h] = fma2(f[h], f[h], s[h]);
                    }
                }
            }
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = i % 2 ? s[i / 2].y : s[i / 2].x;
                a += i < t.split ? e : 0.f;
                b += i < t.split ? 0.f : e;
            }
            if (pass == 0) {
                m0 = t.mine ? __fdiv_rn(a, float(t.mine * t.split)) : 0.f;
                m1 = t.mine && t.split < V ? __fdiv_rn(b, float(t.mine * (V - t.split))) : 0.f;
            } else {
                rec[threadIdx.x] = make_float4(m0, a, m1, b);
            }
        }
    }
    __syncthreads();
    // A warp a group: the mean over its threads' means, then the squares about it.
    const int full = (t.r1 - t.r0) / q.lanes, extra = (t.r1 - t.r0) - full * q.lanes;
    for (int g = int(threadIdx.x >> 5); g < t.groups; g += nt >> 5) {
        const int ca = g * p.Cg, va = ca / V, vb = (ca + p.Cg - 1) / V;
        float mean = 0.f, m2 = 0.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            float s = 0.f;
            for (int cv = va; cv <= vb; ++cv) {
                const bool later = cv * V < ca;  // the vector begins in the group before
                const int width = min(ca + p.Cg, cv * V + V) - max(ca, cv * V);
#pragma unroll 2
                for (int l = int(threadIdx.x & 31); l < q.lanes; l += 32) {
                    const float4 r = rec[l * q.cols + cv];
                    const float n = float((full + (l < extra)) * width);
                    const float mu = later ? r.z : r.x, dlt = mu - mean;
                    s += pass == 0 ? n * mu : (later ? r.w : r.y) + n * dlt * dlt;
                }
            }
            s = warp_sum(s);
            if (pass == 0) mean = __fdiv_rn(s, gc_rows(p, q, t.rank) * float(p.Cg));
            else m2 = s;
        }
        if ((threadIdx.x & 31) == 0) {
            gs[2 * g] = mean;
            gs[2 * g + 1] = m2;
            if (q.S == 1) {
                stat[2 * g] = mean;
                stat[2 * g + 1] = rsqrtf(m2 * p.inv_m + p.eps);
            }
        }
    }
    if (q.S > 1) {
        cluster_arrive(), cluster_wait();
        const uint32_t base = tc::smem_u32(gs);
        for (int g = threadIdx.x; g < t.groups; g += nt) {
            float mu[8], m2[8], sum = 0.f, sq = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S) {
                    mu[r] = tc::ld_dsmem_f32(tc::dsmem_addr(base + 8 * g, r));
                    m2[r] = tc::ld_dsmem_f32(tc::dsmem_addr(base + 8 * g + 4, r));
                }
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S) sum += mu[r] * (gc_rows(p, q, r) * float(p.Cg));
            const float m = __fdiv_rn(sum, p.m);
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S) {
                    const float dlt = mu[r] - m;
                    sq += m2[r] + dlt * dlt * (gc_rows(p, q, r) * float(p.Cg));
                }
            stat[2 * g] = m;
            stat[2 * g + 1] = rsqrtf(sq * p.inv_m + p.eps);
        }
        cluster_arrive();  // this block has read what it needs from the others
    }
    __syncthreads();
    if (mean_out && t.rank == 0)
        for (int g = threadIdx.x; g < t.groups; g += nt) {
            mean_out[int64_t(t.b) * p.G + t.g0 + g] = stat[2 * g];
            rstd_out[int64_t(t.b) * p.G + t.g0 + g] = stat[2 * g + 1];
        }
    if (t.mine) {
        float2 mu[H], rs[H], ga[H], be[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int ca = t.col * V + 2 * h, cb = min(ca + 1, t.col * V + V - 1);
            const int ka = t.g + (2 * h >= t.split), kb = t.g + (cb - t.col * V >= t.split);
            mu[h] = make_float2(-stat[2 * ka], -stat[2 * kb]);
            rs[h] = make_float2(stat[2 * ka + 1], stat[2 * kb + 1]);
            ga[h] = make_float2(gb[ca], gb[cb]);
            be[h] = make_float2(gb[q.W + ca], gb[q.W + cb]);
        }
        T* py = y + at + int64_t(t.r0 + t.lane) * p.C;
        const int64_t row_hop = int64_t(q.lanes) * p.C;
        with_act(p.act, [&](auto act) {
#pragma unroll 2
            for (int k = 0; k < t.mine; ++k) {
                Vec<T, V> v;
                float2 f[H];
                v.load(reinterpret_cast<const T*>(slot + k * hop));
                gc_unpack<T, V>(v, f);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    f[h] = add2(mul2(mul2(add2(f[h], mu[h]), rs[h]), ga[h]), be[h]);
                    f[h] = make_float2(act_value<act.value>(f[h].x), act_value<act.value>(f[h].y));
                }
                gc_pack<T, V>(v, f);
                v.store(py + k * row_hop);
            }
        });
    }
    if (q.S > 1) cluster_wait();  // no block leaves while another still reads its shared memory
}

template <typename T, int V>
__global__ void __launch_bounds__(GC_THREADS, 1)
gn_cluster_bwd_nhwc(const GnParams p, const GnCluster q, const T* x, const T* dy, const T* gamma, const T* beta,
                    const float* mean, const float* rstd, T* dx, float* part)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T)), H = gc_pairs<V>();
    const GcTile t(p, q, V);
    const int nt = int(blockDim.x), hop = nt * VB, tile = q.K * hop;
    unsigned char* slot = dyn + threadIdx.x * VB;
    float2* red = reinterpret_cast<float2*>(dyn + 2 * size_t(tile));  // lanes x W (sum dz*xhat, sum dz)
    float2* red2 = red + nt * V;
    float2* col = red2 + nt;                          // W: the block's channel sums, read by the others
    float2* gs = col + q.W;                           // groups x (sum dz*gamma*xhat, sum dz*gamma), read by the others
    float2* gt = gs + q.groups;                       // groups x (m2, m1) of the unit
    float4* cp = reinterpret_cast<float4*>(gt + q.groups + (q.W & 1));  // W x (-mean, rstd, gamma, beta)
    const int64_t at = int64_t(t.b) * p.N + t.c0 + t.col * V;
    tc::grid_dep_wait();
    for (int k = 0, r = t.r0 + t.lane; k < t.mine; ++k, r += q.lanes) {
        fetch_vec<T, V>(slot + k * hop, x + at + int64_t(r) * p.C);
        fetch_vec<T, V>(slot + tile + k * hop, dy + at + int64_t(r) * p.C);
    }
    for (int c = threadIdx.x; c < t.W; c += nt) {
        const int64_t g = int64_t(t.b) * p.G + t.g0 + c / p.Cg;
        cp[c] = make_float4(-mean[g], rstd[g], gamma ? Elem<T>::ldg(gamma + t.c0 + c) : 1.f,
                            beta ? Elem<T>::ldg(beta + t.c0 + c) : 0.f);
    }
    copy_wait();
    __syncthreads();
    float2 mu[H], rs[H], ga[H], be[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int c = t.in ? t.col * V + 2 * h : 0;
        const float4 a = cp[c], b = cp[2 * h + 1 < V ? c + 1 : c];
        mu[h] = make_float2(a.x, b.x);
        rs[h] = make_float2(a.y, b.y);
        ga[h] = make_float2(a.z, b.z);
        be[h] = make_float2(a.w, b.w);
    }
    {
        float2 sg[H], sb[H];
#pragma unroll
        for (int h = 0; h < H; ++h) sg[h] = sb[h] = both(0.f);
        with_act(p.act, [&](auto act) {
#pragma unroll 2
            for (int k = 0; k < t.mine; ++k) {
                Vec<T, V> v;
                float2 xh[H], dz[H];
                v.load(reinterpret_cast<const T*>(slot + k * hop));
                gc_unpack<T, V>(v, xh);
                v.load(reinterpret_cast<const T*>(slot + tile + k * hop));
                gc_unpack<T, V>(v, dz);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    xh[h] = mul2(add2(xh[h], mu[h]), rs[h]);
                    const float2 z = add2(mul2(xh[h], ga[h]), be[h]);
                    dz[h] = make_float2(gn_dz<act.value>(dz[h].x, z.x), gn_dz<act.value>(dz[h].y, z.y));
                    sb[h] = add2(sb[h], dz[h]);
                    sg[h] = fma2(dz[h], xh[h], sg[h]);
                }
            }
        });
        if (t.in)
#pragma unroll
            for (int i = 0; i < V; ++i)
                red[t.lane * t.W + t.col * V + i] = i % 2 ? make_float2(sg[i / 2].y, sb[i / 2].y)
                                                          : make_float2(sg[i / 2].x, sb[i / 2].x);
    }
    __syncthreads();
    {  // the lanes' sums of each channel: `parts` subsets of the lanes side by side, then those
        const int parts = max(1, min(nt / t.W, 16));
        float2* first = parts > 1 ? red2 : col;
        for (int i = threadIdx.x; i < t.W * parts; i += nt) {
            const int pt = i / t.W, c = i - pt * t.W;
            float2 s = both(0.f);
            for (int l = pt; l < q.lanes; l += parts) s = add2(s, red[l * t.W + c]);
            first[i] = s;
        }
        __syncthreads();
        if (parts > 1) {
            for (int c = threadIdx.x; c < t.W; c += nt) {
                float2 s = both(0.f);
                for (int pt = 0; pt < parts; ++pt) s = add2(s, red2[pt * t.W + c]);
                col[c] = s;
            }
            __syncthreads();
        }
    }
    for (int g = int(threadIdx.x >> 5); g < t.groups; g += nt >> 5) {
        float2 s = both(0.f);
        for (int c = g * p.Cg + int(threadIdx.x & 31); c < (g + 1) * p.Cg; c += 32) s = fma2(both(cp[c].z), col[c], s);
        s = make_float2(warp_sum(s.x), warp_sum(s.y));
        if ((threadIdx.x & 31) == 0) {
            gs[g] = s;
            if (q.S == 1) gt[g] = mul2(s, both(p.inv_m));
        }
    }
    if (q.S > 1) {
        cluster_arrive(), cluster_wait();
        const uint32_t gbase = tc::smem_u32(gs);
        for (int g = threadIdx.x; g < 2 * t.groups; g += nt) {
            float v[8], s = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S) v[r] = tc::ld_dsmem_f32(tc::dsmem_addr(gbase + 4 * g, r));
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S) s += v[r];
            reinterpret_cast<float*>(gt)[g] = s * p.inv_m;
        }
    }
    if (part) {  // the unit's channel sums: block r of the cluster writes every S-th
        const uint32_t cbase = tc::smem_u32(col);
        for (int i = int(threadIdx.x) * q.S + t.rank; i < 2 * t.W; i += nt * q.S) {
            const int kind = i >= t.W, c = i - kind * t.W;
            float s = 0.f;
            if (q.S > 1) {
                float v[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < q.S) v[r] = tc::ld_dsmem_f32(tc::dsmem_addr(cbase + 8 * c + 4 * kind, r));
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < q.S) s += v[r];
            } else {
                s = kind ? col[c].y : col[c].x;
            }
            part[(int64_t(t.b) * 2 + kind) * p.C + t.c0 + c] = s;
        }
    }
    if (q.S > 1) cluster_arrive();
    __syncthreads();
    if (t.mine) {
        float2 m1[H], m2[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int i1 = min(2 * h + 1, V - 1);
            const float2 a = gt[t.g + (2 * h >= t.split)], b = gt[t.g + (i1 >= t.split)];
            m2[h] = make_float2(-a.x, -b.x);
            m1[h] = make_float2(-a.y, -b.y);
        }
        T* po = dx + at + int64_t(t.r0 + t.lane) * p.C;
        const int64_t row_hop = int64_t(q.lanes) * p.C;
        with_act(p.act, [&](auto act) {
#pragma unroll 1
            for (int k = 0; k < t.mine; ++k) {
                Vec<T, V> v;
                float2 xh[H], dz[H];
                v.load(reinterpret_cast<const T*>(slot + tile + k * hop));
                gc_unpack<T, V>(v, dz);
                v.load(reinterpret_cast<const T*>(slot + k * hop));
                gc_unpack<T, V>(v, xh);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    xh[h] = mul2(add2(xh[h], mu[h]), rs[h]);
                    const float2 z = add2(mul2(xh[h], ga[h]), be[h]);
                    dz[h] = make_float2(gn_dz<act.value>(dz[h].x, z.x), gn_dz<act.value>(dz[h].y, z.y));
                    xh[h] = mul2(rs[h], fma2(xh[h], m2[h], fma2(dz[h], ga[h], m1[h])));
                }
                gc_pack<T, V>(v, xh);
                v.store(po + k * row_hop);
            }
        });
    }
    if (q.S > 1) cluster_wait();
}

// ---- NCHW ------------------------------------------------------------------------------------
// A unit is a group's M consecutive values; block r holds the vectors [r*n/S, (r+1)*n/S), thread
// t the vectors t, t + T, ... of them.  A vector lies in one channel or spans two (V <= P).
struct GcRange {
    int b, g, rank, v0, v1;
    int64_t base;
    __device__ __forceinline__ GcRange(const GnParams& p, const GnCluster& q, int V)
    {
        rank = q.S > 1 ? int(tc::cluster_rank()) : 0;
        const int unit = int(blockIdx.x) / q.S;
        b = unit / p.G;
        g = unit - b * p.G;
        v0 = gc_cut(q.vecs, q, rank);
        v1 = gc_cut(q.vecs, q, rank + 1);
        base = int64_t(b) * p.N + int64_t(g) * p.M;
    }
};
__device__ __forceinline__ int gc_count(const GnCluster& q, int V, int r)
{
    return (gc_cut(q.vecs, q, r + 1) - gc_cut(q.vecs, q, r)) * V;
}

// Gamma and beta of a vector's values: channel c up to value `split`, channel c + 1 from there.
struct GcChan {
    int c, split;
    __device__ __forceinline__ GcChan(const GnParams& p, const FastDivmod& dmP, int v, int V)
    {
        uint32_t cc, r;
        dmP.divmod(uint32_t(v) * uint32_t(V), cc, r);
        c = int(cc);
        split = p.P - int(r);
    }
};

__device__ __forceinline__ float block_sum(float v, float* sm)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < int(blockDim.x) / 32; ++w) v += sm[w];
    return v;
}

template <typename T, int V>
__global__ void __launch_bounds__(GC_THREADS, 2)
gn_cluster_fwd_nchw(const GnParams p, const GnCluster q, const FastDivmod dmP, const T* x, const T* gamma,
                    const T* beta, T* y, float* mean_out, float* rstd_out)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T));
    const GcRange t(p, q, V);
    const int nt = int(blockDim.x);
    unsigned char* slot = dyn + threadIdx.x * VB;
    float* gb = reinterpret_cast<float*>(dyn + size_t(q.K) * nt * VB);  // Cg x (gamma, beta)
    float* sm = gb + 2 * p.Cg;
    float* ex = sm + 32;  // the block's mean and M2, read by the others
    const T* px = x + t.base;
    tc::grid_dep_wait();
    for (int v = t.v0 + int(threadIdx.x), k = 0; v < t.v1; v += nt, ++k)
        fetch_vec<T, V>(slot + size_t(k) * nt * VB, px + int64_t(v) * V);
    for (int c = threadIdx.x; c < p.Cg; c += nt) {
        gb[2 * c] = gamma ? Elem<T>::ldg(gamma + t.g * p.Cg + c) : 1.f;
        gb[2 * c + 1] = beta ? Elem<T>::ldg(beta + t.g * p.Cg + c) : 0.f;
    }
    copy_wait();
    const int left = t.v1 - t.v0 - int(threadIdx.x), mine = left > 0 ? (left + nt - 1) / nt : 0;
    float s = 0.f;
#pragma unroll 2
    for (int k = 0; k < mine; ++k) {
        Vec<T, V> v;
        v.load(reinterpret_cast<const T*>(slot + size_t(k) * nt * VB));
#pragma unroll
        for (int i = 0; i < V; ++i) s += v.get(i);
    }
    float mu = __fdiv_rn(block_sum(s, sm), float((t.v1 - t.v0) * V));
    s = 0.f;
#pragma unroll 2
    for (int k = 0; k < mine; ++k) {
        Vec<T, V> v;
        v.load(reinterpret_cast<const T*>(slot + size_t(k) * nt * VB));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float dlt = v.get(i) - mu;
            s += dlt * dlt;
        }
    }
    float sq = block_sum(s, sm);
    if (q.S > 1) {
        if (threadIdx.x == 0) {
            ex[0] = mu;
            ex[1] = sq;
        }
        cluster_arrive(), cluster_wait();
        const uint32_t base = tc::smem_u32(ex);
        float m[8], m2[8], sum = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < q.S) {
                m[r] = tc::ld_dsmem_f32(tc::dsmem_addr(base, r));
                m2[r] = tc::ld_dsmem_f32(tc::dsmem_addr(base + 4, r));
            }
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < q.S) sum += m[r] * float(gc_count(q, V, r));
        mu = __fdiv_rn(sum, p.m);
        sq = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < q.S) {
                const float dlt = m[r] - mu;
                sq += m2[r] + dlt * dlt * float(gc_count(q, V, r));
            }
        cluster_arrive();
    }
    const float rs = rsqrtf(sq * p.inv_m + p.eps);
    if (mean_out && t.rank == 0 && threadIdx.x == 0) {
        mean_out[int64_t(t.b) * p.G + t.g] = mu;
        rstd_out[int64_t(t.b) * p.G + t.g] = rs;
    }
    T* py = y + t.base;
    with_act(p.act, [&](auto act) {
#pragma unroll 2
        for (int k = 0; k < mine; ++k) {
            const int at = t.v0 + int(threadIdx.x) + k * nt;
            const GcChan ch(p, dmP, at, V);
            const float2 a = *reinterpret_cast<const float2*>(gb + 2 * ch.c);
            const float2 b = *reinterpret_cast<const float2*>(gb + 2 * min(ch.c + 1, p.Cg - 1));
            Vec<T, V> v;
            v.load(reinterpret_cast<const T*>(slot + size_t(k) * nt * VB));
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool first = i < ch.split;
                o[i] = act_value<act.value>(gn_z(gn_xhat(v.get(i), mu, rs), first ? a.x : b.x, first ? a.y : b.y));
            }
            v.set(o);
            v.store(py + int64_t(at) * V);
        }
    });
    if (q.S > 1) cluster_wait();
}

template <typename T, int V>
__global__ void __launch_bounds__(GC_THREADS, 1)
gn_cluster_bwd_nchw(const GnParams p, const GnCluster q, const FastDivmod dmP, const T* x, const T* dy,
                    const T* gamma, const T* beta, const float* mean, const float* rstd, T* dx, float* part)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T));
    const GcRange t(p, q, V);
    const int nt = int(blockDim.x);
    const size_t tile = size_t(q.K) * nt * VB;
    unsigned char* slot = dyn + threadIdx.x * VB;
    float2* vs = reinterpret_cast<float2*>(dyn + 2 * tile);  // each vector's sums (its first channel's)
    float2* over = vs + q.K * nt;                            // channel c: sums of the vector that enters c from c - 1
    float2* chs = over + p.Cg;                               // channel sums of the block, read by the others
    float* gb = reinterpret_cast<float*>(chs + p.Cg);
    float* sm = gb + 2 * p.Cg;
    float* ex = sm + 32;
    const int64_t grp = int64_t(t.b) * p.G + t.g;
    tc::grid_dep_wait();
    for (int v = t.v0 + int(threadIdx.x), k = 0; v < t.v1; v += nt, ++k) {
        fetch_vec<T, V>(slot + size_t(k) * nt * VB, x + t.base + int64_t(v) * V);
        fetch_vec<T, V>(slot + tile + size_t(k) * nt * VB, dy + t.base + int64_t(v) * V);
    }
    for (int c = threadIdx.x; c < p.Cg; c += nt) {
        gb[2 * c] = gamma ? Elem<T>::ldg(gamma + t.g * p.Cg + c) : 1.f;
        gb[2 * c + 1] = beta ? Elem<T>::ldg(beta + t.g * p.Cg + c) : 0.f;
        over[c] = make_float2(0.f, 0.f);
    }
    const float mu = mean[grp], rs = rstd[grp];
    copy_wait();
    __syncthreads();
    const int left = t.v1 - t.v0 - int(threadIdx.x), mine = left > 0 ? (left + nt - 1) / nt : 0;
    float s1 = 0.f, s2 = 0.f;
    with_act(p.act, [&](auto act) {
#pragma unroll 1
        for (int k = 0; k < mine; ++k) {
            const GcChan ch(p, dmP, t.v0 + int(threadIdx.x) + k * nt, V);
            const float2 a = *reinterpret_cast<const float2*>(gb + 2 * ch.c);
            const float2 b = *reinterpret_cast<const float2*>(gb + 2 * min(ch.c + 1, p.Cg - 1));
            Vec<T, V> vx, vd;
            vx.load(reinterpret_cast<const T*>(slot + size_t(k) * nt * VB));
            vd.load(reinterpret_cast<const T*>(slot + tile + size_t(k) * nt * VB));
            float2 f = make_float2(0.f, 0.f), o = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool first = i < ch.split;
                const float xh = gn_xhat(vx.get(i), mu, rs);
                const float dz = gn_dz<act.value>(vd.get(i), gn_z(xh, first ? a.x : b.x, first ? a.y : b.y));
                const float dg = dz * xh;
                f.x += first ? dg : 0.f;
                f.y += first ? dz : 0.f;
                o.x += first ? 0.f : dg;
                o.y += first ? 0.f : dz;
            }
            s1 += f.y * a.x + o.y * b.x;
            s2 += f.x * a.x + o.x * b.x;
            vs[k * nt + threadIdx.x] = f;
            if (ch.split < V) over[ch.c + 1] = o;
        }
    });
    s1 = block_sum(s1, sm);
    s2 = block_sum(s2, sm);
    if (q.S > 1 && threadIdx.x == 0) {
        ex[0] = s1;
        ex[1] = s2;
    }
    if (part) {
        // channel c's vectors are those that start in it: [ceil(c*P/V), ceil((c+1)*P/V)), of
        // which this block holds some; few vectors a channel: a thread a channel, else a warp
        const bool thin = p.P < 8 * V;
        const int lane = thin ? 0 : int(threadIdx.x & 31), hop = thin ? 1 : 32;
        for (int c = thin ? int(threadIdx.x) : int(threadIdx.x >> 5); c < p.Cg; c += thin ? nt : nt >> 5) {
            const int lo = max(t.v0, int(unsigned(c * p.P + V - 1) / V));
            const int hi = min(t.v1, int(unsigned((c + 1) * p.P + V - 1) / V));
            float2 s = make_float2(0.f, 0.f);
            for (int v = lo + lane; v < hi; v += hop) {
                const float2 e = vs[v - t.v0];
                s.x += e.x;
                s.y += e.y;
            }
            if (!thin) {
                s.x = warp_sum(s.x);
                s.y = warp_sum(s.y);
            }
            if (lane == 0) chs[c] = make_float2(s.x + over[c].x, s.y + over[c].y);
        }
    }
    if (q.S > 1) cluster_arrive(), cluster_wait();
    else __syncthreads();
    if (q.S > 1) {
        const uint32_t base = tc::smem_u32(ex);
        float a[8], b[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < q.S) {
                a[r] = tc::ld_dsmem_f32(tc::dsmem_addr(base, r));
                b[r] = tc::ld_dsmem_f32(tc::dsmem_addr(base + 4, r));
            }
        s1 = s2 = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < q.S) {
                s1 += a[r];
                s2 += b[r];
            }
    }
    if (part) {
        const uint32_t cbase = tc::smem_u32(chs);
        for (int i = int(threadIdx.x) * q.S + t.rank; i < 2 * p.Cg; i += nt * q.S) {
            const int c = i >> 1, kind = i & 1;
            float v[8], s = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S)
                    v[r] = q.S > 1 ? tc::ld_dsmem_f32(tc::dsmem_addr(cbase + 4 * i, r))
                                   : reinterpret_cast<const float*>(chs)[i];
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < q.S) s += v[r];
            part[(int64_t(t.b) * 2 + kind) * p.C + t.g * p.Cg + c] = s;
        }
    }
    if (q.S > 1) cluster_arrive();
    const float m1 = s1 * p.inv_m, m2 = s2 * p.inv_m;
    T* po = dx + t.base;
    with_act(p.act, [&](auto act) {
#pragma unroll 1
        for (int k = 0; k < mine; ++k) {
            const int at = t.v0 + int(threadIdx.x) + k * nt;
            const GcChan ch(p, dmP, at, V);
            const float2 a = *reinterpret_cast<const float2*>(gb + 2 * ch.c);
            const float2 b = *reinterpret_cast<const float2*>(gb + 2 * min(ch.c + 1, p.Cg - 1));
            Vec<T, V> vx, vd;
            vx.load(reinterpret_cast<const T*>(slot + size_t(k) * nt * VB));
            vd.load(reinterpret_cast<const T*>(slot + tile + size_t(k) * nt * VB));
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool first = i < ch.split;
                const float xh = gn_xhat(vx.get(i), mu, rs);
                const float dz = gn_dz<act.value>(vd.get(i), gn_z(xh, first ? a.x : b.x, first ? a.y : b.y));
                o[i] = rs * (dz * (first ? a.x : b.x) - m1 - xh * m2);
            }
            vx.set(o);
            vx.store(po + int64_t(at) * V);
        }
    });
    if (q.S > 1) cluster_wait();
}

template <typename T>
cudaError_t cluster_fwd_t(const GnParams& p, const GnCluster& q, const T* x, const T* gamma, const T* beta, T* y,
                          float* mean, float* rstd, cudaStream_t s)
{
    const dim3 grid(unsigned(p.B) * unsigned(q.wins) * unsigned(q.S)), block(q.threads);
    const FastDivmod dm{uint32_t(p.P)};
    cudaError_t e = cudaSuccess;
#define GN_CALL(T_, V_)                                                                                               \
    do {                                                                                                              \
        if (q.nhwc) {                                                                                                 \
            e = ensure_smem<gn_cluster_fwd_nhwc<T_, V_>>(q.smem);                                                     \
            if (e == cudaSuccess)                                                                                     \
                e = launch_ex(gn_cluster_fwd_nhwc<T_, V_>, grid, block, q.smem, s, q.S, true, p, q, x, gamma, beta,   \
                              y, mean, rstd);                                                                         \
        } else {                                                                                                      \
            e = ensure_smem<gn_cluster_fwd_nchw<T_, V_>>(q.smem);                                                     \
            if (e == cudaSuccess)                                                                                     \
                e = launch_ex(gn_cluster_fwd_nchw<T_, V_>, grid, block, q.smem, s, q.S, true, p, q, dm, x, gamma,     \
                              beta, y, mean, rstd);                                                                   \
        }                                                                                                             \
    } while (0)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t cluster_bwd_t(const GnParams& p, const GnCluster& q, const T* x, const T* dy, const T* gamma,
                          const T* beta, const float* mean, const float* rstd, T* dx, float* part, cudaStream_t s)
{
    const dim3 grid(unsigned(p.B) * unsigned(q.wins) * unsigned(q.S)), block(q.threads);
    const FastDivmod dm{uint32_t(p.P)};
    cudaError_t e = cudaSuccess;
#define GN_CALL(T_, V_)                                                                                               \
    do {                                                                                                              \
        if (q.nhwc) {                                                                                                 \
            e = ensure_smem<gn_cluster_bwd_nhwc<T_, V_>>(q.smem);                                                     \
            if (e == cudaSuccess)                                                                                     \
                e = launch_ex(gn_cluster_bwd_nhwc<T_, V_>, grid, block, q.smem, s, q.S, true, p, q, x, dy, gamma,     \
                              beta, mean, rstd, dx, part);                                                            \
        } else {                                                                                                      \
            e = ensure_smem<gn_cluster_bwd_nchw<T_, V_>>(q.smem);                                                     \
            if (e == cudaSuccess)                                                                                     \
                e = launch_ex(gn_cluster_bwd_nchw<T_, V_>, grid, block, q.smem, s, q.S, true, p, q, dm, x, dy, gamma, \
                              beta, mean, rstd, dx, part);                                                            \
        }                                                                                                             \
    } while (0)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t run_gn_cluster_fwd(const GnParams& p, const GnCluster& q, int dt, const void* x, const void* gamma,
                               const void* beta, void* y, float* mean, float* rstd, cudaStream_t s)
{
    if (dt == DT_F32)
        return cluster_fwd_t<float>(p, q, (const float*)x, (const float*)gamma, (const float*)beta, (float*)y, mean,
                                    rstd, s);
    using H = __nv_bfloat16;
    return cluster_fwd_t<H>(p, q, (const H*)x, (const H*)gamma, (const H*)beta, (H*)y, mean, rstd, s);
}

cudaError_t run_gn_cluster_bwd(const GnParams& p, const GnCluster& q, int dt, const void* x, const void* dy,
                               const void* gamma, const void* beta, const float* mean, const float* rstd, void* dx,
                               float* part, cudaStream_t s)
{
    if (dt == DT_F32)
        return cluster_bwd_t<float>(p, q, (const float*)x, (const float*)dy, (const float*)gamma, (const float*)beta,
                                    mean, rstd, (float*)dx, part, s);
    using H = __nv_bfloat16;
    return cluster_bwd_t<H>(p, q, (const H*)x, (const H*)dy, (const H*)gamma, (const H*)beta, mean, rstd, (H*)dx, part,
                            s);
}

}  // namespace igc
