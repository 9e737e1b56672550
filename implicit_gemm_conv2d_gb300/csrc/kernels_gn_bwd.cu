// kernels_gn_bwd.cu -- group norm with an activation, backward.  With xhat and z as in the
// forward and dz = dy * act'(z):
//   dbeta[c] = sum_{b,p} dz,   dgamma[c] = sum_{b,p} dz * xhat,
//   dx = rstd * (dz*gamma - m1 - xhat*m2),  m1 = mean_group(dz*gamma),  m2 = mean_group(dz*gamma*xhat).
//
// x and dy in, dx out: bound by memory like the forward, and split the same way.  A group that
// fits a team is read once into registers; a lane keeps the channel sums of its own positions
// over all the samples its team walks, and a block adds them per channel once, at its end.
// Larger groups take a pass for the channels' sums (which give the group's m1 and m2 too:
// m1 = sum gamma*sum dz / M) and a pass for dx.  Channel sums over the batch are added in a
// fixed order by a last small kernel.
#include "gn_common.cuh"

namespace igc {

namespace {

template <typename T, int V, int K, bool WIDE>
__global__ void __launch_bounds__(WIDE ? GN_TEAM_MAX : GN_THREADS, WIDE ? 1 : 2)
gn_team_bwd(const GnParams p, const GnTeam q, const T* x, const T* dy, const T* gamma, const T* beta,
            const float* mean_in, const float* rstd_in, T* dx, float* part)
{
    constexpr int E = K * V;
    extern __shared__ float dyn[];  // the block's channel sums by position, one kind at a time
    __shared__ float sm[64];
    int turn = 0;
    const int L = q.L;
    const int ti = WIDE ? 0 : int(threadIdx.x) / L, lane = WIDE ? int(threadIdx.x) : int(threadIdx.x) % L;
    const int gi = ti % q.gpc, si = ti / q.gpc;
    const int gset = int(blockIdx.x) % q.gsets, chunk = int(blockIdx.x) / q.gsets;
    const int g = gset * q.gpc + gi;
    const bool active = si < q.spc && g < p.G;
    const int nvec = int(p.M / V), cgv = p.Cg / V;
    const bool nhwc = p.layout == CONV_LAYOUT_NHWC;
    int off[K];
    bool has[K];
    float ga[E], be[E], sb[E], sg[E];
    tc::grid_dep_wait();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int j = lane + k * L;
        has[k] = active && j < nvec;
        const int row = nhwc ? j / cgv : 0;
        off[k] = nhwc ? row * p.C + g * p.Cg + (j - row * cgv) * V : int(g * p.M) + j * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = g * p.Cg + (nhwc ? (j - row * cgv) * V + i : (j * V + i) / p.P);
            ga[k * V + i] = !has[k] ? 0.f : gamma ? Elem<T>::ldg(gamma + c) : 1.f;
            be[k * V + i] = has[k] && beta ? Elem<T>::ldg(beta + c) : 0.f;
            sb[k * V + i] = sg[k * V + i] = 0.f;
        }
    }
    const int step = q.chunks * q.spc;
    const int b0 = chunk * q.spc + si;
    const int iters = ceil_div(p.B - chunk * q.spc, step);
    Vec<T, V> cx[K], cd[K], nx[K], nd[K];
    float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;
    auto fetch = [&](Vec<T, V>(&vx)[K], Vec<T, V>(&vd)[K], float& m, float& r, int b) {
        const bool in = active && b < p.B;
        m = in ? mean_in[int64_t(b) * p.G + g] : 0.f;
        r = in ? rstd_in[int64_t(b) * p.G + g] : 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (has[k] && b < p.B) {
                vx[k].load(x + int64_t(b) * p.N + off[k]);
                vd[k].load(dy + int64_t(b) * p.N + off[k]);
            } else {
                vx[k].zero();
                vd[k].zero();
            }
        }
    };
    fetch(cx, cd, mu, rs, b0);
    for (int it = 0; it < iters; ++it) {
        const int b = b0 + it * step;
        if (it + 1 < iters) fetch(nx, nd, nmu, nrs, b + step);
        float xh[E], dg[E], s1 = 0.f, s2 = 0.f;
        with_act(p.act, [&](auto act) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = k * V + i;
                    xh[e] = gn_xhat(cx[k].get(i), mu, rs);
                    const float dz = gn_dz<act.value>(cd[k].get(i), xh[e], ga[e], be[e]);
                    sb[e] += dz;
                    sg[e] += dz * xh[e];
                    dg[e] = dz * ga[e];
                    s1 += dg[e];
                    s2 += dg[e] * xh[e];
                }
        });
        const float m1 = team_total<WIDE>(s1, L, sm, turn) * p.inv_m;
        const float m2 = team_total<WIDE>(s2, L, sm, turn) * p.inv_m;
        if (b < p.B) {
            T* po = dx + int64_t(b) * p.N;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float r[V];
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] = rs * (dg[k * V + i] - m1 - xh[k * V + i] * m2);
                Vec<T, V> o;
                o.set(r);
                if (has[k]) o.store(po + off[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            cx[k] = nx[k];
            cd[k] = nd[k];
        }
        mu = nmu;
        rs = nrs;
    }
    if (!part) return;
    // Channel sums of the block: dgamma's, then dbeta's, by position in shared memory; a warp a
    // channel adds its positions over the block's samples in a fixed order.
    const int m = int(p.M), lane_w = int(threadIdx.x) & 31, nw = int(blockDim.x) >> 5;
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (has[k])
#pragma unroll
                for (int i = 0; i < V; ++i)
                    dyn[(si * q.gpc + gi) * m + (lane + k * L) * V + i] = kind ? sb[k * V + i] : sg[k * V + i];
        __syncthreads();
        for (int w = int(threadIdx.x) >> 5; w < q.gpc * p.Cg; w += nw) {
            const int gj = w / p.Cg, cl = w - gj * p.Cg;
            if (gset * q.gpc + gj >= p.G) break;
            float t = 0.f;
            for (int o = lane_w; o < q.spc * p.P; o += 32) {
                const int s = o / p.P, pp = o - s * p.P;
                t += dyn[(s * q.gpc + gj) * m + (nhwc ? pp * p.Cg + cl : cl * p.P + pp)];
            }
            t = warp_sum(t);
            if (lane_w == 0)
                part[(int64_t(chunk) * 2 + kind) * p.C + (gset * q.gpc + gj) * p.Cg + cl] = t;
        }
    }
}

// dgamma (y = 0) and dbeta (y = 1): the sum of the `n` partials of each channel.  Block: 32
// channels by 32 lanes, each lane its partials in ascending order, the lanes in ascending order.
// Partial i of (kind, channel) is part[i / inner * outer_stride + i % inner * inner_stride +
// kind * kind_stride + channel * chan_stride].
struct ChanSum {
    int64_t n;
    int inner;
    int64_t outer_stride, inner_stride, kind_stride, chan_stride;
};
template <typename T>
__global__ void __launch_bounds__(1024) gn_chan_sum(int C, const ChanSum q, const float* part, T* dgamma, T* dbeta)
{
    __shared__ float sm[32][33];
    const int c = int(blockIdx.x) * 32 + int(threadIdx.x & 31), l = int(threadIdx.x >> 5);
    float t = 0.f;
    tc::grid_dep_wait();
    if (c < C)
        for (int64_t i = l; i < q.n; i += 32) {
            const int64_t o = i / q.inner;
            t += part[o * q.outer_stride + (i - o * q.inner) * q.inner_stride + blockIdx.y * q.kind_stride +
                      c * q.chan_stride];
        }
    sm[l][threadIdx.x & 31] = t;
    __syncthreads();
    if (l == 0 && c < C) {
        t = 0.f;
        for (int i = 0; i < 32; ++i) t += sm[i][threadIdx.x & 31];
        Elem<T>::st((blockIdx.y ? dbeta : dgamma) + c, t);
    }
}

// ---- large groups ----------------------------------------------------------------------------
template <typename T, int V>
__global__ void __launch_bounds__(256) gn_sums_nhwc(const GnParams p, const GnPieces q, const T* x, const T* dy,
                                                    const T* gamma, const T* beta, const float* mean,
                                                    const float* rstd, float* psg, float* psb)
{
    constexpr int U = 2;
    __shared__ float sm_g[256 * V], sm_b[256 * V];
    const GnTile t(p, q, V, blockIdx.x);
    const int lanes = t.lanes;
    tc::grid_dep_wait();
    if (t.in()) {
        float mu[V], rs[V], ga[V], be[V], sg[V], sb[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = (t.cv0 + t.col) * V + i;
            const int64_t o = int64_t(t.b) * p.G + c / p.Cg;
            mu[i] = mean[o];
            rs[i] = rstd[o];
            ga[i] = gamma ? Elem<T>::ldg(gamma + c) : 1.f;
            be[i] = beta ? Elem<T>::ldg(beta + c) : 0.f;
            sg[i] = sb[i] = 0.f;
        }
        const int64_t base = int64_t(t.b) * p.N + int64_t(t.cv0 + t.col) * V;
        with_act(p.act, [&](auto act) {
            for (int r = t.r0 + t.lane; r < t.r1; r += lanes * U) {
                Vec<T, V> vx[U], vd[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (r + u * lanes < t.r1) {
                        vx[u].load(x + base + int64_t(r + u * lanes) * p.C);
                        vd[u].load(dy + base + int64_t(r + u * lanes) * p.C);
                    } else {
                        vx[u].zero();
                        vd[u].zero();
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r + u * lanes < t.r1)
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float xh = gn_xhat(vx[u].get(i), mu[i], rs[i]);
                            const float dz = gn_dz<act.value>(vd[u].get(i), xh, ga[i], be[i]);
                            sb[i] += dz;
                            sg[i] += dz * xh;
                        }
            }
        });
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sm_g[(t.lane * q.cols + t.col) * V + i] = sg[i];
            sm_b[(t.lane * q.cols + t.col) * V + i] = sb[i];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < t.cols * V; c += blockDim.x) {
        float a = 0.f, b = 0.f;
        for (int l = 0; l < lanes; ++l) {
            a += sm_g[l * q.cols * V + c];
            b += sm_b[l * q.cols * V + c];
        }
        const int64_t o = gn_part(p, q.pieces, t.b, t.cv0 * V + c, t.pc);
        psg[o] = a;
        psb[o] = b;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) gn_sums_nchw(const GnParams p, const GnPieces q, const T* x, const T* dy,
                                                    const T* gamma, const T* beta, const float* mean,
                                                    const float* rstd, float* psg, float* psb)
{
    constexpr int U = 2;
    __shared__ float sm[8][2];
    const GnRow t(p, q, V, blockIdx.x);
    tc::grid_dep_wait();
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
                            const float dz = gn_dz<act.value>(vd[u].get(i), xh, ga, be);
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
        psg[t.row * q.pieces + t.pc] = sg;
        psb[t.row * q.pieces + t.pc] = sb;
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
    float s1 = 0.f, s2 = 0.f;
    for (int i = threadIdx.x; i < np; i += blockDim.x) {
        const int cl = p.layout == CONV_LAYOUT_NHWC ? i % p.Cg : i / q.pieces;
        const int pc = p.layout == CONV_LAYOUT_NHWC ? i / p.Cg : i % q.pieces;
        const int c = g * p.Cg + cl;
        const float ga = gamma ? Elem<T>::ldg(gamma + c) : 1.f;
        const int64_t o = gn_part(p, q.pieces, b, c, pc);
        s1 += ga * psb[o];
        s2 += ga * psg[o];
    }
    s1 = team_total<true>(s1, blockDim.x, sm, turn) * p.inv_m;
    s2 = team_total<true>(s2, blockDim.x, sm, turn) * p.inv_m;
    if (threadIdx.x == 0) {
        m1[blockIdx.x] = s1;
        m2[blockIdx.x] = s2;
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) gn_dx_nhwc(const GnParams p, const GnPieces q, const T* x, const T* dy,
                                                  const T* gamma, const T* beta, const float* mean, const float* rstd,
                                                  const float* m1, const float* m2, T* dx)
{
    constexpr int U = 2;
    const GnTile t(p, q, V, q.blocks - 1 - blockIdx.x);
    const int lanes = t.lanes;
    tc::grid_dep_wait();
    if (!t.in()) return;
    float mu[V], rs[V], ga[V], be[V], a1[V], a2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = (t.cv0 + t.col) * V + i;
        const int64_t o = int64_t(t.b) * p.G + c / p.Cg;
        mu[i] = mean[o];
        rs[i] = rstd[o];
        a1[i] = m1[o];
        a2[i] = m2[o];
        ga[i] = gamma ? Elem<T>::ldg(gamma + c) : 1.f;
        be[i] = beta ? Elem<T>::ldg(beta + c) : 0.f;
    }
    const int64_t base = int64_t(t.b) * p.N + int64_t(t.cv0 + t.col) * V;
    with_act(p.act, [&](auto act) {
        for (int r = t.r0 + t.lane; r < t.r1; r += lanes * U) {
            Vec<T, V> vx[U], vd[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * lanes < t.r1) {
                    vx[u].load(x + base + int64_t(r + u * lanes) * p.C);
                    vd[u].load(dy + base + int64_t(r + u * lanes) * p.C);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (r + u * lanes < t.r1) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float xh = gn_xhat(vx[u].get(i), mu[i], rs[i]);
                        const float dz = gn_dz<act.value>(vd[u].get(i), xh, ga[i], be[i]);
                        o[i] = rs[i] * (dz * ga[i] - a1[i] - xh * a2[i]);
                    }
                    vx[u].set(o);
                    vx[u].store(dx + base + int64_t(r + u * lanes) * p.C);
                }
        }
    });
}

template <typename T, int V>
__global__ void __launch_bounds__(256) gn_dx_nchw(const GnParams p, const GnPieces q, const T* x, const T* dy,
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
                        const float dz = gn_dz<act.value>(vd[u].get(i), xh, ga, be);
                        o[i] = rs * (dz * ga - a1 - xh * a2);
                    }
                    vx[u].set(o);
                    vx[u].store(po + e + u * t.hop);
                }
        }
    });
}

template <typename T>
cudaError_t chan_sum(const GnParams& p, const ChanSum& q, const float* part, T* dgamma, T* dbeta, cudaStream_t s)
{
    return launch_ex(gn_chan_sum<T>, dim3(ceil_div(p.C, 32), 2), dim3(1024), 0, s, 1, true, p.C, q, part, dgamma, dbeta);
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
        const size_t smem = dgamma ? size_t(4) * q.gpc * q.spc * size_t(p.M) : 0;
        if (!dgamma) part = nullptr;
#define GN_CALL(T_, V_, K_)                                                                                           \
    e = q.L > 32 ? launch_ex(gn_team_bwd<T_, V_, K_, true>, grid, block, smem, s, 1, true, p, q, x, dy, gamma, beta,  \
                             mean, rstd, dx, part)                                                                    \
                 : launch_ex(gn_team_bwd<T_, V_, K_, false>, grid, block, smem, s, 1, true, p, q, x, dy, gamma, beta, \
                             mean, rstd, dx, part)
        GN_DISPATCH_TEAM(T, GN_CALL);
#undef GN_CALL
        if (e != cudaSuccess || !dgamma) return e != cudaSuccess ? e : cudaGetLastError();
        const ChanSum cs = {q.chunks, q.chunks, 0, 2 * int64_t(p.C), p.C, 1};
        e = chan_sum<T>(p, cs, part, dgamma, dbeta, s);
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const GnPieces q = gn_pieces(p, dt, d);
    const int64_t np = int64_t(p.B) * p.C * q.pieces;
    float* psg = part;
    float* psb = psg + np;
    float* m1 = psb + np;
    float* m2 = m1 + int64_t(p.B) * p.G;
    const bool nhwc = p.layout == CONV_LAYOUT_NHWC;
    const dim3 grid(static_cast<unsigned>(q.blocks));
#define GN_CALL(T_, V_)                                                                                            \
    e = nhwc ? launch_ex(gn_sums_nhwc<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, dy, gamma, beta,     \
                         mean, rstd, psg, psb)                                                                     \
             : launch_ex(gn_sums_nchw<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, dy, gamma, beta,     \
                         mean, rstd, psg, psb)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    if (e != cudaSuccess) return e;
    const float *cg = psg, *cb = psb, *c1 = m1, *c2 = m2;
    e = launch_ex(gn_group_sums<T>, dim3(unsigned(p.B) * unsigned(p.G)), dim3(128), 0, s, 1, true, p, q, gamma, cg, cb,
                  m1, m2);
    if (e != cudaSuccess) return e;
    if (dgamma) {
        const ChanSum cs = nhwc ? ChanSum{int64_t(p.B) * q.pieces, q.pieces, int64_t(q.pieces) * p.C, p.C, np, 1}
                                : ChanSum{int64_t(p.B) * q.pieces, q.pieces, int64_t(p.C) * q.pieces, 1, np, q.pieces};
        e = chan_sum<T>(p, cs, psg, dgamma, dbeta, s);
        if (e != cudaSuccess) return e;
    }
#define GN_CALL(T_, V_)                                                                                               \
    e = nhwc ? launch_ex(gn_dx_nhwc<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, dy, gamma, beta, mean,    \
                         rstd, c1, c2, dx)                                                                            \
             : launch_ex(gn_dx_nchw<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, dy, gamma, beta, mean,    \
                         rstd, c1, c2, dx)
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
