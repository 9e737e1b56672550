// kernels_gn_cluster.cu -- group norm of groups too large for a team of lanes, kept on chip: a
// thread-block cluster of S blocks holds a unit (NCHW: one group of a sample; NHWC: a sample's
// positions of a window of whole groups) in its shared memory, so x (and dy) are read from
// memory once.  A thread copies its own vectors asynchronously into its own slots and is the
// only one to read them: the tile is an extension of its registers and needs no barrier.
//
// A cluster walks the samples with its groups fixed.  A slot is refilled with the next sample's
// vector as soon as its result has been stored, so the next sample is on its way while this one
// is finished, without a second tile.  What is set up once -- indices, gamma and beta, the
// backward's channel sums, kept per value's place and added up when the cluster ends -- is most
// of the instructions of a small unit.  Per sample the blocks exchange their groups' partial
// results through distributed shared memory, with one cluster barrier.
//
// Measured (us; of the rate of the measured copy for one read of each input and one write):
//   24 x 320 x 72x72 bf16, 32 groups of 10, SiLU, channels last, forward: 48, 49%; NCHW 41, 58%;
//     fp32 84 and 60.
//   12 x 192 x 95x101 bf16, 24 groups of 8, GELU, channels last, backward: 63, 32% (ReLU 12 less).
// Bound by latency: an instruction is issued in 0.51 (forward) or 0.47 slots, from 20 warps an SM.
// They wait for the activation's steps (its 2^x and 1/x), for shared memory and, a fifth of the
// backward's time, at the barriers around a sample's sums.  In bf16 the backward's 48 instructions a
// value (the activation is computed twice) alone would take 28 us.
// Beside two passes over memory (24 x 320 x 5184, SiLU): forward bf16 41 / 78, channels last 53 / 80,
// fp32 61 / 98 and 82 / 139; backward bf16 102 / 144 and 108 / 152, fp32 141 / 157 and 149 / 188.
#include <atomic>

#include "gn_common.cuh"

namespace igc {

namespace {

constexpr int GC_MAX_CG = 2048;            // channels of a group (their gammas sit in shared memory)
constexpr int GC_SMEM = 113 * 1024;        // of a block: two share an SM, or each waits with its SM
constexpr int GC_THREADS = 512;
constexpr int GC_ROW_THREADS = 384;        // NHWC: 80 registers a thread, 64 spill (95x101 backward 75 -> 65 us)
constexpr int GC_WARPS = GC_THREADS / 32;
constexpr int GC_SLOTS = 128;              // of a thread: its one-pass statistics lose up to log2 of that in bits
constexpr int GC_FWD_BYTES = 256, GC_BWD_BYTES = 96;  // of x a thread holds, at most where the block can grow

}  // namespace

// Bytes of shared memory beside the tiles.
static int gc_extra(const GnCluster& q, bool bwd)
{
    if (q.nhwc) return 16 * q.threads + 16 * GC_WARPS + 8 * q.W + 32 * q.groups + (bwd ? 8 * q.threads : 0);
    return 4 * 2 * (q.Cg + 1) + 32 * GC_WARPS + 64 + (bwd ? 8 * (q.K * q.threads + q.Cg + 1) : 0);
}

namespace {

__global__ void gc_probe() {}

// Clusters of S blocks that the device holds at once with b blocks an SM (clusters lie within a
// GPC, whose SMs do not divide evenly: 36 and not 38 of eight blocks, two an SM).  Asked for once a
// device; without one, what the SMs alone allow.
int gc_resident(const DevInfo& d, int S, int log_s, int b)
{
    constexpr int DEVICES = 16, BLOCKS = 32;
    static std::atomic<int> known[DEVICES][4][BLOCKS + 1];
    const int most = std::max(1, d.sms * b / S);
    if (S == 1 || b > BLOCKS || d.device < 0 || d.device >= DEVICES) return most;
    std::atomic<int>& k = known[d.device][log_s][b];
    int n = k.load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t c = {};
        cudaLaunchAttribute a;
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = S;
        a.val.clusterDim.y = a.val.clusterDim.z = 1;
        c.gridDim = dim3(S);
        c.blockDim = dim3(32);
        c.dynamicSmemBytes = size_t(227 * 1024) / b - 1024;
        c.attrs = &a;
        c.numAttrs = 1;
        if (cudaFuncSetAttribute(gc_probe, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 1024) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, gc_probe, &c) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = most;
        }
        k.store(std::min(n, most), std::memory_order_relaxed);
        n = std::min(n, most);
    }
    return n;
}

}  // namespace

GnCluster gn_cluster(const GnParams& p, int dt, const DevInfo& d, bool bwd)
{
    GnCluster q = {};
    const int es = dt == DT_F32 ? 4 : 2;
    // one position: both layouts are the same, and channels last reads it in wide vectors
    const bool nhwc = p.layout == CONV_LAYOUT_NHWC || p.P == 1;
    q.nhwc = nhwc;
    q.Cg = p.Cg;
    q.V = 16 / es;
    // A vector lies in two groups (NHWC) or two channels (NCHW) at most.  In the channels-last
    // backward one of two groups has at most 4 values: its sums take registers by place.
    if (nhwc) {
        while (p.C % q.V != 0 || (p.Cg % q.V != 0 && q.V > std::min(bwd ? 4 : 8, p.Cg))) q.V /= 2;
        q.one = p.Cg % q.V == 0;
    } else {
        while (p.M % q.V != 0 || q.V > p.P) q.V /= 2;
    }
    const int tiles = bwd ? 2 : 1, vb = q.V * es;
    if (p.Cg > GC_MAX_CG) return q;
    int lcm = p.Cg;
    while (lcm % q.V != 0) lcm += p.Cg;
    // NHWC: windows of whole vectors and whole groups, 64 bytes of a row (two sectors) or less.
    const int widest = nhwc ? std::max(1, std::min(ceil_div(64, lcm * es), ceil_div(p.C, lcm))) : 1;
    const int most_threads = nhwc ? GC_ROW_THREADS : GC_THREADS;
    for (int m = widest; m >= 1; --m) {
        int64_t vecs;  // of the unit
        if (nhwc) {
            q.W = std::min(m * lcm, p.C);
            q.cols = q.W / q.V;
            q.groups = q.W / p.Cg;
            q.wins = ceil_div(p.C, q.W);
            if (q.cols > most_threads) continue;
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
            // Threads: about so many that each holds GC_*_BYTES.  Of the counts up to twice that (from
            // half for large blocks) whose tiles fit, the one with the fewest slots a thread (and two
            // for what a sample costs besides) for the blocks that an SM holds by registers (80 or 64
            // a thread) and by shared memory (64 x 1024 x 256, 32 groups, channels last, fp32
            // backward: 384 threads and two blocks 58 us, 256 and three 47).
            const int bytes = bwd ? GC_BWD_BYTES : GC_FWD_BYTES, least = nhwc ? round_up(q.cols, 32) : 32;
            const int about = int(std::min<int64_t>(
                most_threads, std::max<int64_t>(least, (per * vb + bytes * 32 - 1) / (bytes * 32) * 32)));
            GnCluster r = {};
            int by_smem = 0, per_sm = 0;
            for (int t = std::max(least, about > 128 ? about / 64 * 32 : about); t <= std::min(most_threads, 2 * about); t += 32) {
                q.lanes = nhwc ? t / q.cols : 1;
                const int64_t n = nhwc ? (int64_t(ceil_div(p.P, S)) + q.lanes - 1) / q.lanes : (per + t - 1) / t;
                if (n > GC_SLOTS || n * t * vb * tiles > GC_SMEM) continue;
                q.threads = t;
                q.K = int(n);
                q.smem = q.K * t * vb * tiles + gc_extra(q, bwd);
                if (q.smem > GC_SMEM) continue;
                const int by = (227 * 1024) / (q.smem + 1024);
                const int blocks = std::min(std::max(1, std::min(32, (nhwc ? 768 : 1024) / t)), by);
                if (per_sm == 0 || (n + 2) * per_sm < int64_t(r.K + 2) * blocks) r = q, per_sm = blocks, by_smem = by;
            }
            if (per_sm == 0) continue;
            r.S = S;
            r.log_s = log;
            // larger clusters while the SMs are not filled and the blocks still have a few
            // kilobytes each
            if (S * 2 <= most && units * S < 2 * d.sms && per * vb > 4096) continue;
            // A larger cluster or a narrower window where tiles of half an SM's shared memory leave it
            // few threads that walk them long (24 x 320 x 5184 bf16, groups of 10, channels last,
            // backward, us: windows of 40 channels, clusters of eight, 512 threads an SM 135; 20,
            // four, 576 153; 20, eight, 768 107).
            if (by_smem <= 2 && r.threads * per_sm < 700 && r.K > 16) {
                if (S * 2 <= most) continue;
                if (m > 1) break;
            }
            r.chunks = std::max(1, std::min(p.B, gc_resident(d, S, log, per_sm) / q.wins));
            if (bwd) r.chunks = gn_bounded_chunks(r.chunks, std::max(1, p.B));
            r.dm_cols = FastDivmod(uint32_t(std::max(1, q.cols)));
            r.dm_cg = FastDivmod(uint32_t(p.Cg));
            r.dm_p = FastDivmod(uint32_t(p.P));
            r.dm_wins = FastDivmod(uint32_t(q.wins));
            r.ok = true;
            return r;
        }
    }
    return GnCluster{};
}

namespace {

template <int BYTES> __device__ __forceinline__ void copy_async(uint32_t dst, const void* src)
{
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

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

// The cluster barrier (the warp has to be converged for it).
__device__ __forceinline__ void cluster_barrier()
{
    __syncwarp();
    tc::cluster_sync();
}

// Where block r's part of n items begins (S is a power of two).
__device__ __forceinline__ int gc_cut(int n, const GnCluster& q, int r) { return int((int64_t(n) * r) >> q.log_s); }

// A vector's values as pairs; one value: (value, 0).
template <int V> constexpr int gc_pairs() { return (V + 1) / 2; }
template <typename T, int V>
__device__ __forceinline__ void gc_load(const unsigned char* slot, float2 (&f)[gc_pairs<V>()])
{
    Vec<T, V> v;
    v.load(reinterpret_cast<const T*>(slot));
#pragma unroll
    for (int h = 0; h < gc_pairs<V>(); ++h) f[h] = make_float2(v.get(2 * h), 2 * h + 1 < V ? v.get(2 * h + 1) : 0.f);
}
template <typename T, int V> __device__ __forceinline__ void gc_store(T* p, const float2 (&f)[gc_pairs<V>()])
{
    float r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
    Vec<T, V> v;
    v.set(r);
    v.store(p);
}

// A thread's statistics in one pass: each place of its vectors has sums about a pivot, the place's
// first value and, after 16, 32 and 64 values, the mean so far (gc_stats).  What the subtraction at
// the end takes away is at most 16 times what is left where it is the first value that is far off,
// and a small factor else, whatever the values' offset; equal values give zeros.  (With the first
// value as the pivot throughout, one value far off cost rstd 4e-5 at 125 values a place.)
template <int V> struct PivotSums {
    static constexpr int H = gc_pairs<V>();
    float2 c[H], s[H], s2[H];  // minus the pivot; sums of the differences and of their squares
    __device__ __forceinline__ void start(const float2 (&f)[H])
    {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            c[h] = mul2(f[h], both(-1.f));
            s[h] = s2[h] = both(0.f);
        }
    }
    __device__ __forceinline__ void add(const float2 (&f)[H])
    {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float2 e = add2(f[h], c[h]);
            s[h] = add2(s[h], e);
            s2[h] = fma2(e, e, s2[h]);
        }
    }
    __device__ __forceinline__ void move(int n) { recentre<H>(c, s, s2, float(n)); }
    // (mean, M2) of the values in the places [0, split) and in [split, V), n a place: the places'
    // results joined about one of their means.
    template <bool ONE> __device__ __forceinline__ float4 finish(int n, int split) const
    {
        const float inv = __fdiv_rn(1.f, float(n));
        float mu[V], m2[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float ci = i % 2 ? c[i / 2].y : c[i / 2].x, si = i % 2 ? s[i / 2].y : s[i / 2].x;
            mu[i] = fmaf(si, inv, -ci);
            m2[i] = fmaf(-si * inv, si, i % 2 ? s2[i / 2].y : s2[i / 2].x);
        }
        float a[3] = {0.f, 0.f, 0.f}, b[3] = {0.f, 0.f, 0.f};  // M2; sum and squares of the means' differences
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool first = ONE || i < split;
            const float e = mu[i] - (first ? mu[0] : mu[V - 1]);
            a[0] += first ? m2[i] : 0.f;
            a[1] += first ? e : 0.f;
            a[2] = first ? fmaf(e, e, a[2]) : a[2];
            if (!ONE) {
                b[0] += first ? 0.f : m2[i];
                b[1] += first ? 0.f : e;
                b[2] = first ? b[2] : fmaf(e, e, b[2]);
            }
        }
        const float ia = ONE ? 1.f / V : __fdiv_rn(1.f, float(split));
        float4 r = make_float4(fmaf(a[1], ia, mu[0]), fmaf(float(n), fmaf(-a[1] * ia, a[1], a[2]), a[0]), 0.f, 0.f);
        if (!ONE && split < V) {
            const float ib = __fdiv_rn(1.f, float(V - split));
            r.z = fmaf(b[1], ib, mu[V - 1]);
            r.w = fmaf(float(n), fmaf(-b[1] * ib, b[1], b[2]), b[0]);
        }
        return r;
    }
};

// The statistics of a thread's n > 0 slots, read as their copies arrive (the first half is one
// group of copies, the rest another).
template <typename T, int V, bool ONE>
__device__ __forceinline__ float4 gc_stats(const unsigned char* slot, int hop, int n, int split)
{
    PivotSums<V> w;
    float2 f[gc_pairs<V>()];
    const int half = n / 2;
    if (half > 0) copy_wait<1>();
    else copy_wait<0>();
    gc_load<T, V>(slot, f);
    w.start(f);
#pragma unroll 1
    for (int k = 1, stop = 16;;) {
        if (k == half) copy_wait<0>();
        const int end = min(k < half ? half : n, stop);
#pragma unroll 4
        for (; k < end; ++k) {
            gc_load<T, V>(slot + k * hop, f);
            w.add(f);
        }
        if (k >= n) break;
        if (k == stop) {
            w.move(k);
            stop *= 2;
        }
    }
    return w.template finish<ONE>(n, split);
}

// n, mean and M2 of the values of two sets.
struct Moments {
    float n, mean, m2;
    __device__ __forceinline__ void merge(float n2, float mean2, float m22)
    {
        if (n2 == 0.f) return;
        const float t = n + n2, dlt = mean2 - mean, w = __fdividef(n2, t);
        mean = n == 0.f ? mean2 : fmaf(dlt, w, mean);
        m2 += m22 + dlt * dlt * n * w;
        n = t;
    }
};

// The blocks' results of one value each (mean, M2) merged over the cluster: the unit's mean and
// rstd.  addr: the pair's shared address, the same in every block; count(r): block r's values.
template <class F>
__device__ __forceinline__ float2 gc_exchange(const GnParams& p, const GnCluster& q, uint32_t addr, F&& count)
{
    float mu[kMaxCluster], m2[kMaxCluster], sum = 0.f, sq = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < q.S) {
            mu[r] = tc::ld_dsmem_f32(tc::dsmem_addr(addr, r));
            m2[r] = tc::ld_dsmem_f32(tc::dsmem_addr(addr + 4, r));
        }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < q.S) sum += mu[r] * count(r);
    const float m = __fdiv_rn(sum, p.m);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < q.S) {
            const float dlt = mu[r] - m;
            sq += m2[r] + dlt * dlt * count(r);
        }
    return make_float2(m, rsqrtf(sq * p.inv_m + p.eps));
}
// The blocks' sums of a pair added up.
__device__ __forceinline__ float2 gc_add(const GnCluster& q, uint32_t addr)
{
    float a[kMaxCluster], b[kMaxCluster];
    float2 s = both(0.f);
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < q.S) {
            a[r] = tc::ld_dsmem_f32(tc::dsmem_addr(addr, r));
            b[r] = tc::ld_dsmem_f32(tc::dsmem_addr(addr + 4, r));
        }
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
        if (r < q.S) s = add2(s, make_float2(a[r], b[r]));
    return s;
}

// ---- channels last ---------------------------------------------------------------------------
// Block `rank` of a cluster holds the rows [r0, r1) of a window of W channels; thread (lane, col)
// the vector `col` of the rows r0 + lane, r0 + lane + lanes, ...
struct GcTile {
    int rank, chunk, c0, W, groups, g0, lane, col, r0, r1, mine, full, extra;
    int g, split;  // the group (in the window) of the vector's first channel, its channels in that group
    __device__ __forceinline__ GcTile(const GnParams& p, const GnCluster& q, int V)
    {
        uint32_t a, b;
        rank = q.S > 1 ? int(tc::cluster_rank()) : 0;
        q.dm_wins.divmod(blockIdx.x >> q.log_s, a, b);
        chunk = int(a);
        c0 = int(b) * q.W;
        W = min(q.W, p.C - c0);
        groups = int(q.dm_cg.div(uint32_t(W)));
        g0 = int(q.dm_cg.div(uint32_t(c0)));
        q.dm_cols.divmod(threadIdx.x, a, b);
        lane = int(a);
        col = int(b);
        r0 = gc_cut(p.P, q, rank);
        r1 = gc_cut(p.P, q, rank + 1);
        full = (r1 - r0) / q.lanes;
        extra = r1 - r0 - full * q.lanes;
        const bool in = lane < q.lanes && col * V < W;
        mine = in ? full + (lane < extra) : 0;
        g = in ? int(q.dm_cg.div(uint32_t(col * V))) : 0;
        split = in ? min(V, (g + 1) * p.Cg - col * V) : V;
    }
    __device__ __forceinline__ float rows(const GnParams& p, const GnCluster& q, int r) const
    {
        return float(gc_cut(p.P, q, r + 1) - gc_cut(p.P, q, r));
    }
};

// Calls f(integral_constant<n>, k) for the slots in order, two at a time and a last one.
template <class F> __device__ __forceinline__ void gc_pairwise(int slots, F&& f)
{
    int k = 0;
#pragma unroll 1
    for (; k + 1 < slots; k += 2) f(std::integral_constant<int, 2>(), k);
    if (k < slots) f(std::integral_constant<int, 1>(), k);
}

// Warps that share a group (a power of two).
__device__ __forceinline__ int gc_subs(int groups)
{
    int subs = 1;
    while (subs * 2 * groups <= int(blockDim.x) >> 5) subs *= 2;
    return subs;
}
// Hands every warp its share of a group's vectors: f(group, sub, for_each), where for_each(e)
// calls e(column vector, row lane) for the lane's part of the share.
template <int V, class F>
__device__ __forceinline__ void gc_group_warps(const GnParams& p, const GnCluster& q, const GcTile& t, int subs, F&& f)
{
    const int nw = int(blockDim.x) >> 5, lane = int(threadIdx.x & 31);
    int lw = 1;  // row lanes side by side in the warp
    while (lw < 32 && lw * 2 <= q.lanes) lw *= 2;
    const int l0 = lane & (lw - 1), across = 32 / lw;
    for (int i = int(threadIdx.x) >> 5; i < t.groups * subs; i += nw) {
        const int g = i / subs, sub = i - g * subs;
        const int v0 = g * p.Cg / V, v1 = (g * p.Cg + p.Cg - 1) / V;
        f(g, sub, [&](auto&& e) {
            for (int cv = v0 + sub * across + lane / lw; cv <= v1; cv += subs * across)
#pragma unroll 2
                for (int l = l0; l < q.lanes; l += lw) e(cv, l);
        });
    }
}

template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(GC_ROW_THREADS, 2)
gn_cluster_fwd_nhwc(const GnParams p, const __grid_constant__ GnCluster q, const T* x, const T* gamma, const T* beta,
                    T* y, float* mean_out, float* rstd_out)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T)), H = gc_pairs<V>();
    const GcTile t(p, q, V);
    const int nt = int(blockDim.x), hop = nt * VB, tile = q.K * hop;
    unsigned char* slot = dyn + threadIdx.x * VB;
    float4* rec = reinterpret_cast<float4*>(dyn + tile);  // threads x (mean, M2) of either group
    float4* wrec = rec + nt;                                   // warps x (n, mean, M2) of their share of a group
    float2* gs = reinterpret_cast<float2*>(wrec + GC_WARPS);   // 2 x groups (mean, M2) of the block, read by the others
    float2* stat = gs + 2 * q.groups;                          // groups x (mean, rstd) of the unit
    const int64_t at = t.c0 + t.col * V + int64_t(t.r0 + t.lane) * p.C, row_hop = int64_t(q.lanes) * p.C;
    tc::grid_dep_wait();
    {
        const T* src = x + int64_t(t.chunk) * p.N + at;
        for (int k = 0; k < t.mine; ++k, src += row_hop) {
            fetch_vec<T, V>(slot + k * hop, src);
            if (k == t.mine / 2 - 1) copy_commit();
        }
        copy_commit();
    }
    float2 ga[H], be[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int a = t.c0 + (t.mine ? t.col * V : 0) + 2 * h, b = V > 1 ? a + 1 : a;
        ga[h] = gamma ? make_float2(Elem<T>::ldg(gamma + a), Elem<T>::ldg(gamma + b)) : both(1.f);
        be[h] = beta ? make_float2(Elem<T>::ldg(beta + a), Elem<T>::ldg(beta + b)) : both(0.f);
    }
    const int subs = gc_subs(t.groups);
    int turn = 0;
    for (int b = t.chunk; b < p.B; b += q.chunks, turn ^= 1) {
        const bool more = b + q.chunks < p.B;
        rec[threadIdx.x] = t.mine ? gc_stats<T, V, ONE>(slot, hop, t.mine, t.split) : make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
        // A group's mean over its threads' means, then the squares about it; first by warp.
        gc_group_warps<V>(p, q, t, subs, [&](int g, int sub, auto&& for_each) {
            Moments w = {0.f, 0.f, 0.f};
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                float s = 0.f, n = 0.f;
                for_each([&](int cv, int l) {
                    const bool later = !ONE && cv * V < g * p.Cg;  // the vector begins in the group before
                    const int width = ONE ? V : min((g + 1) * p.Cg, cv * V + V) - max(g * p.Cg, cv * V);
                    const float4 r = rec[l * q.cols + cv];
                    const float c = float((t.full + (l < t.extra)) * width);
                    const float mu = later ? r.z : r.x, dlt = mu - w.mean;
                    s += pass == 0 ? c * mu : (later ? r.w : r.y) + c * dlt * dlt;
                    n += c;
                });
                s = warp_sum(s);
                if (pass == 0) {
                    w.n = warp_sum(n);
                    w.mean = w.n > 0.f ? __fdiv_rn(s, w.n) : 0.f;
                } else {
                    w.m2 = s;
                }
            }
            if ((threadIdx.x & 31) == 0) {
                if (subs > 1) wrec[g * subs + sub] = make_float4(w.n, w.mean, w.m2, 0.f);
                else if (q.S > 1) gs[turn * q.groups + g] = make_float2(w.mean, w.m2);
                else stat[g] = make_float2(w.mean, rsqrtf(w.m2 * p.inv_m + p.eps));
            }
        });
        if (subs > 1) {
            __syncthreads();
            if (int(threadIdx.x) < t.groups) {
                Moments w = {0.f, 0.f, 0.f};
                for (int i = 0; i < subs; ++i) {
                    const float4 r = wrec[threadIdx.x * subs + i];
                    w.merge(r.x, r.y, r.z);
                }
                if (q.S > 1) gs[turn * q.groups + threadIdx.x] = make_float2(w.mean, w.m2);
                else stat[threadIdx.x] = make_float2(w.mean, rsqrtf(w.m2 * p.inv_m + p.eps));
            }
        }
        if (q.S > 1) {
            cluster_barrier();
            for (int g = threadIdx.x; g < t.groups; g += nt)
                stat[g] = gc_exchange(p, q, tc::smem_u32(gs + turn * q.groups + g),
                                      [&](int r) { return t.rows(p, q, r) * float(p.Cg); });
        }
        __syncthreads();
        if (mean_out && t.rank == 0)
            for (int g = threadIdx.x; g < t.groups; g += nt) {
                mean_out[int64_t(b) * p.G + t.g0 + g] = stat[g].x;
                rstd_out[int64_t(b) * p.G + t.g0 + g] = stat[g].y;
            }
        if (t.mine) {
            const float2 s0 = stat[t.g], s1 = ONE ? s0 : stat[min(t.g + 1, t.groups - 1)];
            T* py = y + int64_t(b) * p.N + at;
            const T* px = x + int64_t(b + q.chunks) * p.N + at;
            with_act(p.act, [&](auto act) {
                float2 mu[H], rs[H], sc[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const bool f0 = ONE || 2 * h < t.split, f1 = ONE || 2 * h + 1 < t.split;
                    mu[h] = make_float2(f0 ? -s0.x : -s1.x, f1 ? -s0.x : -s1.x);
                    rs[h] = make_float2(f0 ? s0.y : s1.y, f1 ? s0.y : s1.y);
                    sc[h] = act.value == CONV_ACT_RELU ? ga[h] : mul2(ga[h], rs[h]);
                }
                gc_pairwise(t.mine, [&](auto n, int k) {
                    constexpr int U = n.value;
                    float2 f[U][H];
#pragma unroll
                    for (int u = 0; u < U; ++u) gc_load<T, V>(slot + (k + u) * hop, f[u]);
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            f[u][h] = gn_out<act.value>(add2(f[u][h], mu[h]), rs[h], sc[h], be[h]);
#pragma unroll
                    for (int u = 0; u < U; ++u, py += row_hop, px += row_hop) {
                        gc_store<T, V>(py, f[u]);
                        if (more) fetch_vec<T, V>(slot + (k + u) * hop, px);
                        if (k + u == t.mine / 2 - 1) copy_commit();
                    }
                });
                copy_commit();
            });
        }
    }
    if (q.S > 1) cluster_barrier();  // no block leaves while another still reads its shared memory
}

// part: chunks * S rows of (dgamma's, dbeta's) channel sums.
template <typename T, int V, bool ONE>
__global__ void __launch_bounds__(GC_ROW_THREADS, 2)
gn_cluster_bwd_nhwc(const GnParams p, const __grid_constant__ GnCluster q, const T* x, const T* dy, const T* gamma,
                    const T* beta, const float* mean, const float* rstd, T* dx, float* part)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T)), H = gc_pairs<V>();
    const GcTile t(p, q, V);
    const int nt = int(blockDim.x), hop = nt * VB, tile = q.K * hop;
    unsigned char* slot = dyn + threadIdx.x * VB;
    // threads x (sum dz*gamma*xhat, sum dz*gamma) of either group
    float4* rec = reinterpret_cast<float4*>(dyn + 2 * tile);
    float2* wrec = reinterpret_cast<float2*>(rec + nt);        // warps x the same of their share of a group
    float2* gs = wrec + GC_WARPS;                              // 2 x groups, the block's, read by the others
    float2* gt = gs + 2 * q.groups;                            // groups x (m2, m1) of the unit
    float* red = reinterpret_cast<float*>(rec);                // at the end: channel sums of the lanes
    const int64_t at = t.c0 + t.col * V + int64_t(t.r0 + t.lane) * p.C, row_hop = int64_t(q.lanes) * p.C;
    tc::grid_dep_wait();
    if (part) tc::grid_dep_launch();
    {
        int64_t src = int64_t(t.chunk) * p.N + at;
        for (int k = 0; k < t.mine; ++k, src += row_hop) {
            fetch_vec<T, V>(slot + k * hop, x + src);
            fetch_vec<T, V>(slot + tile + k * hop, dy + src);
            if (k == t.mine / 2 - 1) copy_commit();
        }
        copy_commit();
    }
    float2 ga[H], be[H], sg[H], sb[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int a = t.c0 + (t.mine ? t.col * V : 0) + 2 * h, b = V > 1 ? a + 1 : a;
        ga[h] = gamma ? make_float2(Elem<T>::ldg(gamma + a), Elem<T>::ldg(gamma + b)) : both(1.f);
        be[h] = beta ? make_float2(Elem<T>::ldg(beta + a), Elem<T>::ldg(beta + b)) : both(0.f);
        sg[h] = sb[h] = both(0.f);
    }
    const int subs = gc_subs(t.groups);
    int turn = 0;
    for (int b = t.chunk; b < p.B; b += q.chunks, turn ^= 1) {
        const bool more = b + q.chunks < p.B;
        const int64_t g0 = int64_t(b) * p.G + t.g0 + t.g;
        const float mu0 = -mean[g0], rs0 = rstd[g0];
        const bool next = !ONE && t.split < V;
        const float mu1 = next ? -mean[g0 + 1] : mu0, rs1 = next ? rstd[g0 + 1] : rs0;
        // by place: minus the mean, rstd (this sample's)
        float2 mu[H], rs[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            mu[h] = ONE ? both(mu0) : make_float2(2 * h < t.split ? mu0 : mu1, 2 * h + 1 < t.split ? mu0 : mu1);
            rs[h] = ONE ? both(rs0) : make_float2(2 * h < t.split ? rs0 : rs1, 2 * h + 1 < t.split ? rs0 : rs1);
        }
        {
            float2 a[H], c[H];  // this sample's sums of dz * (x - mean) and dz by place
#pragma unroll
            for (int h = 0; h < H; ++h) a[h] = c[h] = both(0.f);
            with_act(p.act, [&](auto act) {
                float2 sc[H];
#pragma unroll
                for (int h = 0; h < H; ++h) sc[h] = act.value == CONV_ACT_RELU ? ga[h] : mul2(ga[h], rs[h]);
                copy_wait<1>();  // the first half's copies
#pragma unroll 1
                for (int k = 0; k < t.mine; ++k) {
                    if (k == t.mine / 2) copy_wait<0>();
                    float2 d[H], dz[H];
                    gc_load<T, V>(slot + k * hop, d);
                    gc_load<T, V>(slot + tile + k * hop, dz);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        d[h] = add2(d[h], mu[h]);
                        dz[h] = gn_dz_at<act.value>(dz[h], d[h], rs[h], sc[h], be[h]);
                        c[h] = add2(c[h], dz[h]);
                        a[h] = fma2(dz[h], d[h], a[h]);
                    }
                    // dz in dy's place: exact in fp32, and not computed again
                    if constexpr (sizeof(T) == 4) gc_store<T, V>(reinterpret_cast<T*>(slot + tile + k * hop), dz);
                }
            });
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                a[h] = mul2(a[h], rs[h]);
                sg[h] = add2(sg[h], a[h]);
                sb[h] = add2(sb[h], c[h]);
                a[h] = mul2(a[h], ga[h]);
                c[h] = mul2(c[h], ga[h]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float e = i % 2 ? a[i / 2].y : a[i / 2].x, g = i % 2 ? c[i / 2].y : c[i / 2].x;
                const bool first = ONE || i < t.split;
                r.x += first ? e : 0.f;
                r.y += first ? g : 0.f;
                if (!ONE) {
                    r.z += first ? 0.f : e;
                    r.w += first ? 0.f : g;
                }
            }
            rec[threadIdx.x] = r;
        }
        __syncthreads();
        gc_group_warps<V>(p, q, t, subs, [&](int g, int sub, auto&& for_each) {
            float2 s = both(0.f);
            for_each([&](int cv, int l) {
                const bool later = !ONE && cv * V < g * p.Cg;  // the vector begins in the group before
                const float4 r = rec[l * q.cols + cv];
                s = add2(s, later ? make_float2(r.z, r.w) : make_float2(r.x, r.y));
            });
            s = make_float2(warp_sum(s.x), warp_sum(s.y));
            if ((threadIdx.x & 31) == 0) {
                if (subs > 1) wrec[g * subs + sub] = s;
                else if (q.S > 1) gs[turn * q.groups + g] = s;
                else gt[g] = mul2(s, both(p.inv_m));
            }
        });
        if (subs > 1) {
            __syncthreads();
            if (int(threadIdx.x) < t.groups) {
                float2 s = both(0.f);
                for (int i = 0; i < subs; ++i) s = add2(s, wrec[threadIdx.x * subs + i]);
                if (q.S > 1) gs[turn * q.groups + threadIdx.x] = s;
                else gt[threadIdx.x] = mul2(s, both(p.inv_m));
            }
        }
        if (q.S > 1) {
            cluster_barrier();
            for (int g = threadIdx.x; g < t.groups; g += nt)
                gt[g] = mul2(gc_add(q, tc::smem_u32(gs + turn * q.groups + g)), both(p.inv_m));
        }
        __syncthreads();
        if (t.mine) {
            const float2 s0 = gt[t.g], s1 = ONE ? s0 : gt[min(t.g + 1, t.groups - 1)];
            T* po = dx + int64_t(b) * p.N + at;
            int64_t src = int64_t(b + q.chunks) * p.N + at;
            with_act(p.act, [&](auto act) {
                // dx = dz * gamma * rstd - (x - mean) * rstd^2 * m2 - rstd * m1
                float2 sc[H], k1[H], k2[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const bool f0 = ONE || 2 * h < t.split, f1 = ONE || 2 * h + 1 < t.split;
                    sc[h] = mul2(ga[h], rs[h]);
                    k1[h] = mul2(make_float2(f0 ? -s0.y : -s1.y, f1 ? -s0.y : -s1.y), rs[h]);
                    k2[h] = mul2(make_float2(f0 ? -s0.x : -s1.x, f1 ? -s0.x : -s1.x), mul2(rs[h], rs[h]));
                }
#pragma unroll 1
                for (int k = 0; k < t.mine; ++k, po += row_hop, src += row_hop) {
                    float2 d[H], dz[H];
                    gc_load<T, V>(slot + tile + k * hop, dz);
                    gc_load<T, V>(slot + k * hop, d);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        d[h] = add2(d[h], mu[h]);
                        if constexpr (sizeof(T) == 2)
                            dz[h] = gn_dz_at<act.value>(dz[h], d[h], rs[h], act.value == CONV_ACT_RELU ? ga[h] : sc[h],
                                                        be[h]);
                        d[h] = fma2(dz[h], sc[h], fma2(d[h], k2[h], k1[h]));
                    }
                    gc_store<T, V>(po, d);
                    if (more) {
                        fetch_vec<T, V>(slot + k * hop, x + src);
                        fetch_vec<T, V>(slot + tile + k * hop, dy + src);
                    }
                    if (k == t.mine / 2 - 1) copy_commit();
                }
                copy_commit();
            });
        }
    }
    if (q.S > 1) cluster_barrier();  // no block leaves while another still reads its shared memory
    if (!part) return;
    // The lanes' channel sums, a kind and a few of a vector's values at a time (red holds four
    // floats a thread).
    const int64_t row = (int64_t(t.chunk) << q.log_s) + t.rank;
    constexpr int Q = V < 4 ? V : 4;
    int team = 1;  // lanes a channel
    while (team < 32 && team * 2 <= q.lanes && team * 2 * (t.W / V * Q) <= nt) team *= 2;
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int v0 = 0; v0 < V; v0 += Q) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float2 e = kind ? sb[(v0 + i) / 2] : sg[(v0 + i) / 2];
                red[i * nt + threadIdx.x] = (v0 + i) % 2 ? e.y : e.x;
            }
            __syncthreads();
            for (int j0 = 0; j0 < t.W / V * Q * team; j0 += nt) {
                const int j = j0 + int(threadIdx.x), c = j / team, cv = c / Q, i = c % Q;
                float s = 0.f;
                if (cv * V < t.W)
                    for (int l = j & (team - 1); l < q.lanes; l += team) s += red[i * nt + l * q.cols + cv];
                s = team_sum(s, team);
                if (cv * V < t.W && (j & (team - 1)) == 0) part[(row * 2 + kind) * p.C + t.c0 + cv * V + v0 + i] = s;
            }
        }
}

// ---- NCHW ------------------------------------------------------------------------------------
// A unit is a group's M consecutive values; block r holds the vectors [r*n/S, (r+1)*n/S), thread
// t the vectors t, t + T, ... of them.  A vector lies in one channel or spans two (V <= P).
struct GcRange {
    int g, chunk, rank, v0, v1, mine;
    int64_t base;
    __device__ __forceinline__ GcRange(const GnParams& p, const GnCluster& q, int V)
    {
        uint32_t a, b;
        rank = q.S > 1 ? int(tc::cluster_rank()) : 0;
        q.dm_wins.divmod(blockIdx.x >> q.log_s, a, b);
        chunk = int(a);
        g = int(b);
        v0 = gc_cut(q.vecs, q, rank);
        v1 = gc_cut(q.vecs, q, rank + 1);
        const int left = v1 - v0 - int(threadIdx.x);
        mine = left > 0 ? (left - 1) / int(blockDim.x) + 1 : 0;
        base = int64_t(g) * p.M + int64_t(v0 + int(threadIdx.x)) * V;
    }
    __device__ __forceinline__ float count(const GnCluster& q, int V, int r) const
    {
        return float((gc_cut(q.vecs, q, r + 1) - gc_cut(q.vecs, q, r)) * V);
    }
};

// The channel of a vector's first value, and how many of its values lie before the next channel.
struct GcChan {
    int c, split;
    __device__ __forceinline__ GcChan(const GnParams& p, const GnCluster& q, int v, int V)
    {
        uint32_t cc, r;
        q.dm_p.divmod(uint32_t(v) * uint32_t(V), cc, r);
        c = int(cc);
        split = p.P - int(r);
    }
};
// Calls f(gamma pairs, beta pairs) for the vector; gb: (gamma, beta) of each channel.
template <int V, class F> __device__ __forceinline__ void with_channels(const GcChan& ch, const float2* gb, F&& f)
{
    constexpr int H = gc_pairs<V>();
    const float2 a = gb[ch.c];
    float2 ga[H], be[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        ga[h] = both(a.x);
        be[h] = both(a.y);
    }
    if (ch.split < V) {
        const float2 b = gb[ch.c + 1];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (2 * h >= ch.split) ga[h].x = b.x, be[h].x = b.y;
            if (2 * h + 1 >= ch.split) ga[h].y = b.x, be[h].y = b.y;
        }
    }
    f(ga, be);
}

template <typename T, int V>
__global__ void __launch_bounds__(GC_THREADS, 2)
gn_cluster_fwd_nchw(const GnParams p, const __grid_constant__ GnCluster q, const T* x, const T* gamma, const T* beta,
                    T* y, float* mean_out, float* rstd_out)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T)), H = gc_pairs<V>();
    const GcRange t(p, q, V);
    const int nt = int(blockDim.x), hop = nt * VB, tile = q.K * hop, nw = nt >> 5, lane = int(threadIdx.x & 31);
    unsigned char* slot = dyn + threadIdx.x * VB;
    float4* wrec = reinterpret_cast<float4*>(dyn + tile);  // 2 x warps (n, mean, M2)
    float2* ex = reinterpret_cast<float2*>(wrec + 2 * GC_WARPS);  // 2: the block's mean and M2, read by the others
    float2* gb = ex + 2;                                          // Cg x (gamma, beta)
    tc::grid_dep_wait();
    {
        const T* src = x + int64_t(t.chunk) * p.N + t.base;
        for (int k = 0; k < t.mine; ++k, src += nt * V) {
            fetch_vec<T, V>(slot + k * hop, src);
            if (k == t.mine / 2 - 1) copy_commit();
        }
        copy_commit();
    }
    for (int c = threadIdx.x; c < p.Cg; c += nt)
        gb[c] = make_float2(gamma ? Elem<T>::ldg(gamma + t.g * p.Cg + c) : 1.f,
                            beta ? Elem<T>::ldg(beta + t.g * p.Cg + c) : 0.f);
    int turn = 0;
    for (int b = t.chunk; b < p.B; b += q.chunks, turn ^= 1) {
        const bool more = b + q.chunks < p.B;
        // the thread's mean and the squares about it; then the warp's, the block's, the cluster's
        Moments w = {float(t.mine * V), 0.f, 0.f};
        if (t.mine) {
            const float4 r = gc_stats<T, V, true>(slot, hop, t.mine, V);
            w.mean = r.x;
            w.m2 = r.y;
        }
        {
            const float n = warp_sum(w.n), m = n > 0.f ? __fdiv_rn(warp_sum(w.n * w.mean), n) : 0.f;
            const float dlt = w.mean - m;
            w = {n, m, warp_sum(w.m2 + w.n * dlt * dlt)};
        }
        if (nw > 1) {
            if (lane == 0) wrec[turn * GC_WARPS + (threadIdx.x >> 5)] = make_float4(w.n, w.mean, w.m2, 0.f);
            __syncthreads();
            const float4 r = lane < nw ? wrec[turn * GC_WARPS + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            const float n = warp_sum(r.x), m = __fdiv_rn(warp_sum(r.x * r.y), n), dlt = r.y - m;
            w = {n, m, warp_sum(r.z + r.x * dlt * dlt)};
        } else {
            __syncwarp();  // gb
        }
        float2 stat;
        if (q.S > 1) {
            if (threadIdx.x == 0) ex[turn] = make_float2(w.mean, w.m2);
            cluster_barrier();
            stat = gc_exchange(p, q, tc::smem_u32(ex + turn), [&](int r) { return t.count(q, V, r); });
        } else {
            stat = make_float2(w.mean, rsqrtf(w.m2 * p.inv_m + p.eps));
        }
        if (mean_out && t.rank == 0 && threadIdx.x == 0) {
            mean_out[int64_t(b) * p.G + t.g] = stat.x;
            rstd_out[int64_t(b) * p.G + t.g] = stat.y;
        }
        T* py = y + int64_t(b) * p.N + t.base;
        const T* px = x + int64_t(b + q.chunks) * p.N + t.base;
        with_act(p.act, [&](auto act) {
#pragma unroll 1
            for (int k = 0; k < t.mine; ++k, py += nt * V, px += nt * V) {
                const GcChan ch(p, q, t.v0 + int(threadIdx.x) + k * nt, V);
                float2 f[H];
                gc_load<T, V>(slot + k * hop, f);
                with_channels<V>(ch, gb, [&](const auto& ga, const auto& be) {
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        f[h] = gn_out<act.value>(add2(f[h], both(-stat.x)), both(stat.y),
                                                 act.value == CONV_ACT_RELU ? ga[h] : mul2(ga[h], both(stat.y)), be[h]);
                });
                gc_store<T, V>(py, f);
                if (more) fetch_vec<T, V>(slot + k * hop, px);
                if (k == t.mine / 2 - 1) copy_commit();
            }
            copy_commit();
        });
    }
    if (q.S > 1) cluster_barrier();  // no block leaves while another still reads its shared memory
}

template <typename T, int V>
__global__ void __launch_bounds__(GC_THREADS, 2)
gn_cluster_bwd_nchw(const GnParams p, const __grid_constant__ GnCluster q, const T* x, const T* dy, const T* gamma,
                    const T* beta, const float* mean, const float* rstd, T* dx, float* part)
{
    extern __shared__ __align__(16) unsigned char dyn[];
    constexpr int VB = V * int(sizeof(T)), H = gc_pairs<V>();
    const GcRange t(p, q, V);
    const int nt = int(blockDim.x), hop = nt * VB, tile = q.K * hop, nw = nt >> 5, lane = int(threadIdx.x & 31);
    unsigned char* slot = dyn + threadIdx.x * VB;
    float2* vs = reinterpret_cast<float2*>(dyn + 2 * tile);  // (dz*xhat, dz) sums of each vector's
                                                                              // values of its first channel,
    float2* over = vs + q.K * nt;           // of those that enter channel c with the vector that begins in c - 1
    float2* wrec = over + p.Cg + 1;         // 2 x warps
    float2* ex = wrec + 2 * GC_WARPS;       // 2: the block's sums, read by the others
    float2* gb = ex + 2;                    // Cg x (gamma, beta)
    tc::grid_dep_wait();
    if (part) tc::grid_dep_launch();
    {
        int64_t src = int64_t(t.chunk) * p.N + t.base;
        for (int k = 0; k < t.mine; ++k, src += nt * V) {
            fetch_vec<T, V>(slot + k * hop, x + src);
            fetch_vec<T, V>(slot + tile + k * hop, dy + src);
            if (k == t.mine / 2 - 1) copy_commit();
        }
        copy_commit();
    }
    for (int c = threadIdx.x; c < p.Cg; c += nt) {
        gb[c] = make_float2(gamma ? Elem<T>::ldg(gamma + t.g * p.Cg + c) : 1.f,
                            beta ? Elem<T>::ldg(beta + t.g * p.Cg + c) : 0.f);
        over[c] = both(0.f);
    }
    for (int k = 0; k < t.mine; ++k) vs[k * nt + threadIdx.x] = both(0.f);
    __syncthreads();
    int turn = 0;
    for (int b = t.chunk; b < p.B; b += q.chunks, turn ^= 1) {
        const bool more = b + q.chunks < p.B;
        const int64_t grp = int64_t(b) * p.G + t.g;
        const float mu = -mean[grp], rs = rstd[grp];
        float2 s = both(0.f);  // sum dz*gamma*xhat, sum dz*gamma
        with_act(p.act, [&](auto act) {
            copy_wait<1>();  // the first half's copies
#pragma unroll 1
            for (int k = 0; k < t.mine; ++k) {
                if (k == t.mine / 2) copy_wait<0>();
                const GcChan ch(p, q, t.v0 + int(threadIdx.x) + k * nt, V);
                float2 d[H], dz[H];
                gc_load<T, V>(slot + k * hop, d);
                gc_load<T, V>(slot + tile + k * hop, dz);
                with_channels<V>(ch, gb, [&](const auto& ga, const auto& be) {
                    float2 g = both(0.f), e = both(0.f);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        d[h] = add2(d[h], both(mu));
                        dz[h] = gn_dz_at<act.value>(dz[h], d[h], both(rs),
                                                    act.value == CONV_ACT_RELU ? ga[h] : mul2(ga[h], both(rs)), be[h]);
                        g = fma2(dz[h], d[h], g);
                        e = add2(e, dz[h]);
                    }
                    float2 first = V == 1 ? make_float2(g.x, e.x) : make_float2(g.x + g.y, e.x + e.y);
                    if (ch.split < V) {  // the values of either channel apart
                        float2 second = both(0.f);
                        first = both(0.f);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float di = i % 2 ? d[i / 2].y : d[i / 2].x, zi = i % 2 ? dz[i / 2].y : dz[i / 2].x;
                            const float2 v = make_float2(di * zi, zi);
                            if (i < ch.split) first = add2(first, v);
                            else second = add2(second, v);
                        }
                        second.x *= rs;
                        over[ch.c + 1] = add2(over[ch.c + 1], second);
                        s = fma2(second, both(ga[H - 1].y), s);
                    }
                    first.x *= rs;
                    s = fma2(first, both(ga[0].x), s);
                    vs[k * nt + threadIdx.x] = add2(vs[k * nt + threadIdx.x], first);
                });
                // dz in dy's place: exact in fp32, and not computed again
                if constexpr (sizeof(T) == 4) gc_store<T, V>(reinterpret_cast<T*>(slot + tile + k * hop), dz);
            }
        });
        s = make_float2(warp_sum(s.x), warp_sum(s.y));
        if (nw > 1) {
            if (lane == 0) wrec[turn * GC_WARPS + (threadIdx.x >> 5)] = s;
            __syncthreads();
            s = lane < nw ? wrec[turn * GC_WARPS + lane] : both(0.f);
            s = make_float2(warp_sum(s.x), warp_sum(s.y));
        }
        if (q.S > 1) {
            if (threadIdx.x == 0) ex[turn] = s;
            cluster_barrier();
            s = gc_add(q, tc::smem_u32(ex + turn));
        }
        // dx = dz * gamma * rstd - (x - mean) * rstd^2 * m2 - rstd * m1
        const float2 k2 = both(-s.x * p.inv_m * rs * rs), k1 = both(-s.y * p.inv_m * rs);
        T* po = dx + int64_t(b) * p.N + t.base;
        int64_t src = int64_t(b + q.chunks) * p.N + t.base;
        with_act(p.act, [&](auto act) {
#pragma unroll 1
            for (int k = 0; k < t.mine; ++k, po += nt * V, src += nt * V) {
                const GcChan ch(p, q, t.v0 + int(threadIdx.x) + k * nt, V);
                float2 d[H], dz[H];
                gc_load<T, V>(slot + tile + k * hop, dz);
                gc_load<T, V>(slot + k * hop, d);
                with_channels<V>(ch, gb, [&](const auto& ga, const auto& be) {
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const float2 sc = mul2(ga[h], both(rs));
                        d[h] = add2(d[h], both(mu));
                        if constexpr (sizeof(T) == 2)
                            dz[h] = gn_dz_at<act.value>(dz[h], d[h], both(rs), act.value == CONV_ACT_RELU ? ga[h] : sc,
                                                        be[h]);
                        d[h] = fma2(dz[h], sc, fma2(d[h], k2, k1));
                    }
                });
                gc_store<T, V>(po, d);
                if (more) {
                    fetch_vec<T, V>(slot + k * hop, x + src);
                    fetch_vec<T, V>(slot + tile + k * hop, dy + src);
                }
                if (k == t.mine / 2 - 1) copy_commit();
            }
            copy_commit();
        });
    }
    if (q.S > 1) cluster_barrier();  // no block leaves while another still reads its shared memory
    if (!part) return;
    __syncthreads();
    // Channel c's vectors are those that begin in it: [ceil(c*P/V), ceil((c+1)*P/V)), of which
    // this block holds some.  Few vectors a channel: a thread a channel, else a warp.
    const int64_t row = (int64_t(t.chunk) << q.log_s) + t.rank;
    const bool thin = p.P < 8 * V;
    const int l0 = thin ? 0 : lane, step = thin ? 1 : 32;
    for (int c = thin ? int(threadIdx.x) : int(threadIdx.x >> 5); c < p.Cg; c += thin ? nt : nw) {
        const int lo = max(t.v0, int(unsigned(c * p.P + V - 1) / V));
        const int hi = min(t.v1, int(unsigned((c + 1) * p.P + V - 1) / V));
        float2 s = both(0.f);
        for (int v = lo + l0; v < hi; v += step) s = add2(s, vs[v - t.v0]);
        if (!thin) s = make_float2(warp_sum(s.x), warp_sum(s.y));
        if (l0 == 0) {
            s = add2(s, over[c]);
            part[row * 2 * p.C + t.g * p.Cg + c] = s.x;
            part[(row * 2 + 1) * p.C + t.g * p.Cg + c] = s.y;
        }
    }
}

template <typename T>
cudaError_t cluster_fwd_t(const GnParams& p, const GnCluster& q, const T* x, const T* gamma, const T* beta, T* y,
                          float* mean, float* rstd, cudaStream_t s)
{
    const dim3 grid(unsigned(q.chunks) * unsigned(q.wins) * unsigned(q.S)), block(q.threads);
    cudaError_t e = cudaSuccess;
#define GN_LAUNCH(...)                                                                                             \
    do {                                                                                                           \
        e = ensure_smem<__VA_ARGS__>(q.smem);                                                                      \
        if (e == cudaSuccess)                                                                                      \
            e = launch_ex(__VA_ARGS__, grid, block, q.smem, s, q.S, true, p, q, x, gamma, beta, y, mean, rstd);    \
    } while (0)
#define GN_CALL(T_, V_)                                                       \
    do {                                                                      \
        if (!q.nhwc) GN_LAUNCH(gn_cluster_fwd_nchw<T_, V_>);                  \
        else if (q.one) GN_LAUNCH(gn_cluster_fwd_nhwc<T_, V_, true>);         \
        else GN_LAUNCH(gn_cluster_fwd_nhwc<T_, V_, false>);                   \
    } while (0)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
#undef GN_LAUNCH
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t cluster_bwd_t(const GnParams& p, const GnCluster& q, const T* x, const T* dy, const T* gamma,
                          const T* beta, const float* mean, const float* rstd, T* dx, float* part, cudaStream_t s)
{
    const dim3 grid(unsigned(q.chunks) * unsigned(q.wins) * unsigned(q.S)), block(q.threads);
    cudaError_t e = cudaSuccess;
#define GN_LAUNCH(...)                                                                                             \
    do {                                                                                                           \
        e = ensure_smem<__VA_ARGS__>(q.smem);                                                                      \
        if (e == cudaSuccess)                                                                                      \
            e = launch_ex(__VA_ARGS__, grid, block, q.smem, s, q.S, true, p, q, x, dy, gamma, beta, mean, rstd,    \
                          dx, part);                                                                               \
    } while (0)
#define GN_CALL(T_, V_)                                                       \
    do {                                                                      \
        if (!q.nhwc) GN_LAUNCH(gn_cluster_bwd_nchw<T_, V_>);                  \
        else if (q.one) GN_LAUNCH(gn_cluster_bwd_nhwc<T_, V_, true>);         \
        else if constexpr (V_ <= 4) GN_LAUNCH(gn_cluster_bwd_nhwc<T_, V_, false>); \
    } while (0)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
#undef GN_LAUNCH
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
