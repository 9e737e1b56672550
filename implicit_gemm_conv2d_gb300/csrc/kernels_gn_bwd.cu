// kernels_gn_bwd.cu -- group norm with an activation, backward.  With xhat and z as in the
// forward and dz = dy * act'(z):
//   dbeta[c] = sum_{b,p} dz,   dgamma[c] = sum_{b,p} dz * xhat,
//   dx = rstd * (dz*gamma - m1 - xhat*m2),  m1 = mean_group(dz*gamma),  m2 = mean_group(dz*gamma*xhat).
//
// x and dy in, dx out: bound by memory like the forward, and split the same way.  A group that
// fits a team is read once into registers; a lane keeps the channel sums of its own positions
// over all the samples its team walks, and a block adds them per channel once, at its end.
// Larger groups are held by a cluster (kernels_gn_cluster.cu).  Groups beyond that take a pass for
// the channels' sums (which give the group's m1 and m2 too: m1 = sum gamma*sum dz / M) and a pass
// for dx, channels last by row tiles (kernels_gn_nhwc.cu).  Channel sums over the batch are added
// in a fixed order by a last small kernel.
#include "gn_common.cuh"

namespace igc {

namespace {

// ---- small groups ----------------------------------------------------------------------------
// 8192 x 128 x 12, 16 groups, fp32, ReLU: 31 us with the channels' sums, 4.9 TB/s, 74% of the
// measured copy's; bound by the latency of its reads: the two sums a value keep an SM
// to 16 warps (128 registers), each with a sample of 96 bytes a lane on its way.  Beside a
// cluster's (us): 8192 x 128 x 12, SiLU, 34 / 51 fp32 and 31 / 96 bf16; 2048 x 256 x 24, 32 groups,
// 36 / 44 and 33 / 45; 1024 x 256 x 36, 32 groups, channels last 33 / 32 and 34 / 35.
template <typename T, int V, int K>
__global__ void __launch_bounds__(GN_THREADS, 2)
gn_team_bwd(const GnParams p, const GnTeam q, const T* x, const T* dy, const T* gamma, const T* beta,
            const float* mean_in, const float* rstd_in, T* dx, float* part)
{
    constexpr int H = K * V / 2;  // pairs of values
    // gamma and beta by position; at the end the block's channel sums by position
    extern __shared__ __align__(16) float tab[];
    const int L = q.L, m = int(p.M);
    const int ti = int(threadIdx.x) / L, lane = int(threadIdx.x) % L;
    const int gi = ti % q.gpc, si = ti / q.gpc;
    const int g0 = int(blockIdx.x) % q.gsets * q.gpc, g = g0 + gi, chunk = int(blockIdx.x) / q.gsets;
    const bool active = si < q.spc && g < p.G;
    const int nvec = m / V;
    int off[K], toff[K];  // in the sample and in the tables; a lane's vectors beyond the group stay at its start
    bool has[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        has[k] = active && lane + k * L < nvec;
        off[k] = has[k] ? gn_offset(p, q, g, lane + k * L) : 0;
        toff[k] = has[k] ? (lane + k * L) * V : 0;
    }
    const int step = q.chunks * q.spc, iters = ceil_div(p.B - chunk * q.spc, step);
    int b = chunk * q.spc + si;
    Vec<T, V> rx[K], rd[K];
    float nmu = 0.f, nrs = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        rx[k].zero();
        rd[k].zero();
    }
    auto fetch = [&](int at) {
        if (active && at < p.B) {
            nmu = mean_in[int64_t(at) * p.G + g];
            nrs = rstd_in[int64_t(at) * p.G + g];
            const T *px = x + int64_t(at) * p.N, *pd = dy + int64_t(at) * p.N;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (has[k]) {
                    rx[k].load(px + off[k]);
                    rd[k].load(pd + off[k]);
                }
        } else {  // a sample beyond the batch adds nothing
#pragma unroll
            for (int k = 0; k < K; ++k) rd[k].zero();
        }
    };
    tc::grid_dep_wait();
    if (part) tc::grid_dep_launch();
    fetch(b);
    gn_team_tables(p, q, g0, gamma, beta, tab, tab + q.gpc * m);
    __syncthreads();
    const float *gam = tab + gi * m, *bet = gam + q.gpc * m;
    float2 sb[H], sg[H];
#pragma unroll
    for (int h = 0; h < H; ++h) sb[h] = sg[h] = both(0.f);
#pragma unroll 1
    for (int it = 0; it < iters; ++it, b += step) {
        const float mu = nmu, rs = nrs;
        float2 xh[H], dg[H], s1 = both(0.f), s2 = both(0.f);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            xh[h] = mul2(add2(pair_of<T, V, K>(rx, h), both(-mu)), both(rs));
            dg[h] = pair_of<T, V, K>(rd, h);
        }
        if (it + 1 < iters) fetch(b + step);
        float2 ga[H];
        table_pairs<V, K>(gam, toff, ga);
        if (p.act != CONV_ACT_NONE) {
            float2 be[H];
            table_pairs<V, K>(bet, toff, be);
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int h = 0; h < H; ++h) dg[h] = gn_grad<act.value>(dg[h], xh[h], ga[h], be[h]);
            });
        }
        // a lane's vectors beyond the group have zeros for dy and add nothing
#pragma unroll
        for (int h = 0; h < H; ++h) {
            sb[h] = add2(sb[h], dg[h]);
            sg[h] = fma2(dg[h], xh[h], sg[h]);
            dg[h] = mul2(dg[h], ga[h]);
            s1 = add2(s1, dg[h]);
            s2 = fma2(dg[h], xh[h], s2);
        }
        const float m1 = team_sum(s1.x + s1.y, L) * p.inv_m, m2 = team_sum(s2.x + s2.y, L) * p.inv_m;
        if (b < p.B) {
            T* po = dx + int64_t(b) * p.N;
#pragma unroll
            for (int h = 0; h < H; ++h)
                dg[h] = mul2(both(rs), fma2(xh[h], both(-m2), add2(dg[h], both(-m1))));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float r[V];
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] = (k * V + i) % 2 ? dg[(k * V + i) / 2].y : dg[(k * V + i) / 2].x;
                Vec<T, V> o;
                o.set(r);
                if (has[k]) o.store(po + off[k]);
            }
        }
    }
    if (!part) return;
    // Channel sums of the block: dgamma's, then dbeta's, by position in shared memory; `lp` lanes
    // a channel add its positions over the block's samples in a fixed order: as many as there are
    // while every channel has its own.
    const int per = q.spc * p.P, nch = min(q.gpc, p.G - g0) * p.Cg;
    int lp = 1;
    while (lp < 32 && lp * 2 < per && lp * 2 * nch <= int(blockDim.x)) lp *= 2;
    const int sub = int(threadIdx.x) / lp, sl = int(threadIdx.x) % lp, teams = int(blockDim.x) / lp;
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        __syncthreads();
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float2 v = kind ? sb[h] : sg[h];
            const int k0 = 2 * h / V, k1 = (2 * h + 1) / V;
            if (has[k0]) tab[ti * m + (lane + k0 * L) * V + 2 * h % V] = v.x;
            if (has[k1]) tab[ti * m + (lane + k1 * L) * V + (2 * h + 1) % V] = v.y;
        }
        __syncthreads();
#pragma unroll 1
        for (int c0 = 0; c0 < nch; c0 += teams) {
            const int c = c0 + sub;
            float t = 0.f;
            if (c < nch) {
                uint32_t gj, cl;
                q.dm_cg.divmod(uint32_t(c), gj, cl);
                const float* base = tab + gj * m + (p.layout == CONV_LAYOUT_NHWC ? cl : cl * p.P);
                const int hop = p.layout == CONV_LAYOUT_NHWC ? p.Cg : 1;
#pragma unroll 4
                for (int o = sl; o < per; o += lp) {
                    uint32_t s, pp;
                    q.dm_p.divmod(uint32_t(o), s, pp);
                    t += base[int(s) * q.gpc * m + int(pp) * hop];
                }
            }
            t = team_sum(t, lp);
            if (sl == 0 && c < nch) part[(int64_t(chunk) * 2 + kind) * p.C + g0 * p.Cg + c] = t;
        }
    }
}

// dgamma (blockIdx.y = 0) and dbeta (1): the sums of each channel's `n` partials
// part[i * stride + kind * kind_stride + c].  Block: 32 channels by 32 lanes; the S blocks of a
// cluster take contiguous ranges of the partials, each lane its own in ascending order, then the
// lanes and the blocks are added by fixed butterflies.  About 5 us of each backward, most of them
// the launch behind the pass and one trip to memory.
template <typename T>
__global__ void __launch_bounds__(1024, 2) gn_chan_sum(int C, int64_t n, int S, int64_t stride, int64_t kind_stride,
                                                    const float* part, T* dgamma, T* dbeta)
{
    __shared__ float sm[32][33], total[32];
    const int rank = S > 1 ? int(tc::cluster_rank()) : 0;
    const int c = int(blockIdx.x) / S * 32 + int(threadIdx.x & 31), l = int(threadIdx.x >> 5);
    const int64_t i1 = n * (rank + 1) / S;
    float t = 0.f;
    tc::grid_dep_wait();
    if (c < C) {
        const float* at = part + blockIdx.y * kind_stride + c;
        for (int64_t i = n * rank / S + l; i < i1;) {  // 128 at a time, so that no chain is long
            float some = 0.f;
            const int64_t stop = min(i1, i + 32 * 128);
#pragma unroll 8
            for (; i < stop; i += 32) some += at[i * stride];
            t += some;
        }
    }
    sm[l][threadIdx.x & 31] = t;
    __syncthreads();
    // warp l adds channel l's lanes
    t = warp_sum(sm[threadIdx.x & 31][l]);
    const int out = int(blockIdx.x) / S * 32 + l;
    if (S > 1) {
        if ((threadIdx.x & 31) == 0) total[l] = t;
        __syncthreads();
        tc::cluster_sync();
        if (rank == 0) {
            t = int(threadIdx.x & 31) < S ? tc::ld_dsmem_f32(tc::dsmem_addr(tc::smem_u32(total + l), threadIdx.x & 31)) : 0.f;
            t = warp_sum(t);
        }
        __syncwarp();
        tc::cluster_sync();
    }
    if ((threadIdx.x & 31) == 0 && rank == 0 && out < C) Elem<T>::st((blockIdx.y ? dbeta : dgamma) + out, t);
}

// ---- large groups, NCHW ------------------------------------------------------------------------
// Two passes over x and dy: 4 x 128 x 16384, 8 groups, SiLU: 33 us in bf16 and 40 in fp32 (1.5 and
// 2.5 TB/s of two reads and a write); four launches.
template <typename T, int V>
__global__ void __launch_bounds__(256) gn_sums(const GnParams p, const GnPieces q, const T* x, const T* dy,
                                                    const T* gamma, const T* beta, const float* mean,
                                                    const float* rstd, float* psg, float* psb)
{
    constexpr int U = 2;
    __shared__ float sm[8][2];
    const GnRow t(p, q, V, blockIdx.x);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float sg = 0.f, sb = 0.f;
    if (t.in) {
        const int c = int(t.row % p.C);
        const int64_t grp = t.row / p.C * p.G + c / p.Cg;
        const float mu = mean[grp], rs = rstd[grp];
        const float ga = gamma ? Elem<T>::ldg(gamma + c) : 1.f, be = beta ? Elem<T>::ldg(beta + c) : 0.f;
        const T *px = x + t.row * p.P, *pd = dy + t.row * p.P;
        with_act(p.act, [&](auto act) {
            for (int e = t.e0; e < t.e1; e += t.hop * U) {
                Vec<T, V> vx[U], vd[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u * t.hop < t.e1) {
                        vx[u].load(px + e + u * t.hop);
                        vd[u].load(pd + e + u * t.hop);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (e + u * t.hop < t.e1)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float xh = gn_xhat(vx[u].get(i), mu, rs);
                            const float dz = gn_dz<act.value>(vd[u].get(i), gn_z(xh, ga, be));
                            sb += dz;
                            sg += dz * xh;
                        }
            }
        });
    }
    sg = warp_sum(sg);
    sb = warp_sum(sb);
    if (q.row_lanes > 32) {
        if ((threadIdx.x & 31) == 0) {
            sm[threadIdx.x >> 5][0] = sg;
            sm[threadIdx.x >> 5][1] = sb;
        }
        __syncthreads();
        if (t.lane == 0)
            for (int w = 1; w < q.row_lanes / 32; ++w) {
                sg += sm[w][0];
                sb += sm[w][1];
            }
    }
    if (t.lane == 0 && t.in) {
        const int64_t b = t.row / p.C, o = gn_part(p, q.pieces, b, int(t.row - b * p.C), t.pc);
        psg[o] = sg;
        psb[o] = sb;
    }
}

// One block a group: m1 and m2 from its channels' sums.
template <typename T>
__global__ void __launch_bounds__(128) gn_group_sums(const GnParams p, const GnPieces q, const T* gamma,
                                                     const float* psg, const float* psb, float* m1, float* m2)
{
    __shared__ float sm[64];
    int turn = 0;
    const int b = int(blockIdx.x / p.G), g = int(blockIdx.x % p.G);
    const int np = p.Cg * q.pieces;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float2 s = both(0.f);
    gn_stretches(np, s, [&](int i, float2& some) {
        const int pc = i / p.Cg, c = g * p.Cg + i - pc * p.Cg;
        const float ga = gamma ? Elem<T>::ldg(gamma + c) : 1.f;
        const int64_t o = gn_part(p, q.pieces, b, c, pc);
        some.x += ga * psb[o];
        some.y += ga * psg[o];
    });
    const float s1 = block_total(s.x, sm, turn) * p.inv_m;
    const float s2 = block_total(s.y, sm, turn) * p.inv_m;
    if (threadIdx.x == 0) {
        m1[blockIdx.x] = s1;
        m2[blockIdx.x] = s2;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) gn_dx(const GnParams p, const GnPieces q, const T* x, const T* dy,
                                                  const T* gamma, const T* beta, const float* mean, const float* rstd,
                                                  const float* m1, const float* m2, T* dx)
{
    constexpr int U = 2;
    const GnRow t(p, q, V, q.blocks - 1 - blockIdx.x);
    tc::grid_dep_wait();
    if (!t.in) return;
    const int c = int(t.row % p.C);
    const int64_t grp = t.row / p.C * p.G + c / p.Cg;
    const float mu = mean[grp], rs = rstd[grp], a1 = m1[grp], a2 = m2[grp];
    const float ga = gamma ? Elem<T>::ldg(gamma + c) : 1.f, be = beta ? Elem<T>::ldg(beta + c) : 0.f;
    const T *px = x + t.row * p.P, *pd = dy + t.row * p.P;
    T* po = dx + t.row * p.P;
    with_act(p.act, [&](auto act) {
        for (int e = t.e0; e < t.e1; e += t.hop * U) {
            Vec<T, V> vx[U], vd[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u * t.hop < t.e1) {
                    vx[u].load(px + e + u * t.hop);
                    vd[u].load(pd + e + u * t.hop);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u * t.hop < t.e1) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float xh = gn_xhat(vx[u].get(i), mu, rs);
                        const float dz = gn_dz<act.value>(vd[u].get(i), gn_z(xh, ga, be));
                        o[i] = rs * (dz * ga - a1 - xh * a2);
                    }
                    vx[u].set(o);
                    vx[u].store(po + e + u * t.hop);
                }
        }
    });
}

template <typename T>
cudaError_t chan_sum(const GnParams& p, int64_t n, int64_t stride, int64_t kind_stride, const float* part, T* dgamma,
                     T* dbeta, cudaStream_t s)
{
    const int S = n > 512 ? kMaxCluster : 1;  // 32 lanes take up to 16 partials each
    return launch_ex(gn_chan_sum<T>, dim3(ceil_div(p.C, 32) * S, 2), dim3(1024), 0, s, S, true, p.C, n, S, stride,
                     kind_stride, part, dgamma, dbeta);
}

template <typename T>
cudaError_t bwd_t(const GnParams& p, int dt, const DevInfo& d, const T* x, const T* dy, const T* gamma, const T* beta,
                  const float* mean, const float* rstd, T* dx, T* dgamma, T* dbeta, void* ws, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    float* part = static_cast<float*>(ws);
    if (p.B == 0) {
        if (!dgamma) return cudaSuccess;
        e = cudaMemsetAsync(dgamma, 0, size_t(p.C) * sizeof(T), s);
        return e != cudaSuccess ? e : cudaMemsetAsync(dbeta, 0, size_t(p.C) * sizeof(T), s);
    }
    const GnTeam t = gn_team(p, dt, d, true);
    if (t.ok) {
        const GnTeam& q = t;
        const dim3 grid(unsigned(q.gsets) * unsigned(q.chunks)), block(q.threads);
        const size_t smem = size_t(4) * std::max(2 * q.gpc, q.gpc * q.spc) * size_t(p.M);
        float* out = dgamma ? part : nullptr;
#define GN_CALL(T_, V_, K_)                                                                                          \
    e = launch_ex(gn_team_bwd<T_, V_, K_>, grid, block, smem, s, 1, true, p, q, x, dy, gamma, beta, mean, rstd, dx, out)
        GN_DISPATCH_TEAM(T, false, GN_CALL);
#undef GN_CALL
        if (e == cudaSuccess && dgamma) e = chan_sum<T>(p, q.chunks, 2 * int64_t(p.C), p.C, part, dgamma, dbeta, s);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const GnCluster cl = gn_cluster(p, dt, d, true);
    if (cl.ok) {
        e = run_gn_cluster_bwd(p, cl, dt, x, dy, gamma, beta, mean, rstd, dx, dgamma ? part : nullptr, s);
        if (e == cudaSuccess && dgamma) e = chan_sum<T>(p, int64_t(cl.chunks) * cl.S, 2 * int64_t(p.C), p.C, part, dgamma, dbeta, s);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    if (gn_by_rows(p)) {
        const GnRows q = gn_rows(p, dt, d, true);
        float* rows = part + 2 * int64_t(p.B) * p.G * q.parts;
        e = run_gn_rows_bwd(p, q, dt, x, dy, gamma, beta, mean, rstd, dx, dgamma ? rows : nullptr, ws, s);
        if (e == cudaSuccess && dgamma)
            e = chan_sum<T>(p, int64_t(p.B) * q.pieces, 2 * int64_t(p.C), p.C, rows, dgamma, dbeta, s);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const GnPieces q = gn_pieces(p, dt, d);
    const int64_t np = int64_t(p.B) * p.C * q.pieces;
    float* psg = part;
    float* psb = psg + np;
    float* m1 = psb + np;
    float* m2 = m1 + int64_t(p.B) * p.G;
    const dim3 grid(static_cast<unsigned>(q.blocks));
#define GN_CALL(T_, V_)                                                                                       \
    e = launch_ex(gn_sums<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, dy, gamma, beta, mean, rstd, \
                  psg, psb)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    if (e != cudaSuccess) return e;
    const float *cg = psg, *cb = psb, *c1 = m1, *c2 = m2;
    e = launch_ex(gn_group_sums<T>, dim3(unsigned(p.B) * unsigned(p.G)), dim3(128), 0, s, 1, true, p, q, gamma, cg, cb,
                  m1, m2);
    if (e != cudaSuccess) return e;
    if (dgamma) {
        e = chan_sum<T>(p, int64_t(p.B) * q.pieces, p.C, np, psg, dgamma, dbeta, s);
        if (e != cudaSuccess) return e;
    }
#define GN_CALL(T_, V_)                                                                                       \
    e = launch_ex(gn_dx<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, dy, gamma, beta, mean, rstd,  \
                  c1, c2, dx)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t gn_bwd_workspace(const GnParams& p, int dt, const DevInfo& d)
{
    if (p.B == 0) return 0;
    const GnTeam t = gn_team(p, dt, d, true);
    if (t.ok) return size_t(8) * t.chunks * p.C;
    const GnCluster cl = gn_cluster(p, dt, d, true);
    if (cl.ok) return size_t(8) * cl.chunks * cl.S * p.C;
    if (gn_by_rows(p)) {
        const GnRows q = gn_rows(p, dt, d, true);
        return size_t(8) * (size_t(p.B) * p.G * q.parts + size_t(p.B) * q.pieces * p.C);
    }
    const GnPieces q = gn_pieces(p, dt, d);
    return size_t(4) * (2 * size_t(p.B) * p.C * q.pieces + 2 * size_t(p.B) * p.G);
}

cudaError_t run_gn_bwd(const GnParams& p, int dt, const DevInfo& d, const void* x, const void* dy, const void* gamma,
                       const void* beta, const float* mean, const float* rstd, void* dx, void* dgamma, void* dbeta,
                       void* ws, cudaStream_t s)
{
    if (dt == DT_F32)
        return bwd_t<float>(p, dt, d, (const float*)x, (const float*)dy, (const float*)gamma, (const float*)beta, mean,
                            rstd, (float*)dx, (float*)dgamma, (float*)dbeta, ws, s);
    using H = __nv_bfloat16;
    return bwd_t<H>(p, dt, d, (const H*)x, (const H*)dy, (const H*)gamma, (const H*)beta, mean, rstd, (H*)dx,
                    (H*)dgamma, (H*)dbeta, ws, s);
}

}  // namespace igc
