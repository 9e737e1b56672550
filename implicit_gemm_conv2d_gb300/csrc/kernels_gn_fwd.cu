// kernels_gn_fwd.cu -- group norm with an activation, forward:
//   mean = sum x / M,  rstd = 1 / sqrt(sum (x - mean)^2 / M + eps),
//   y = act((x - mean) * rstd * gamma[c] + beta[c]).
//
// About ten operations a value against 2 (bf16) or 4 bytes in and out: bound by memory in fp32, so
// what counts is to read x once.  A group that fits a team of lanes is held in its registers: the
// sum, then the squares about the mean, then the result, one read and one write.  Larger groups
// are held by a thread-block cluster (kernels_gn_cluster.cu).  Groups beyond that are read twice:
// channels last by row tiles (kernels_gn_nhwc.cu), NCHW here by pieces of rows whose (mean, sum of
// squares about it) partials are combined by Chan, Golub & LeVeque's update ("Updating formulae
// and a pairwise algorithm for computing sample variances", 1979).  No path subtracts a squared
// mean from a mean of squares, so a large common offset costs no digits.
#include "gn_common.cuh"

namespace igc {

GnTeam gn_team(const GnParams& p, int dt, const DevInfo& d, bool bwd)
{
    GnTeam q = {};
    const int es = dt == DT_F32 ? 4 : 2, most = gn_team_values(dt, bwd);
    if (p.M > 32 * most) return q;
    // Vector width, vectors a lane and lanes: the fewest instructions a value by this count of
    // them -- a value's own, the team's butterflies (two sums of one word, two steps an
    // instruction pair), a vector's address and access, and what every lane does once -- with
    // idle lanes counted.
    double best = 1e30;
    for (int V = 16 / es; V >= 1; V /= 2) {
        if ((p.layout == CONV_LAYOUT_NCHW ? p.M : p.Cg) % V != 0) continue;
        const int64_t nvec = p.M / V;
        for (int K = 1; K * V <= most; ++K) {
            if (!gn_team_k(V, K)) continue;
            int L = 1, steps = 0;
            while (int64_t(L) * K < nvec) { L *= 2; ++steps; }
            if (L > 32) continue;
            const double cost = double(L) * ((bwd ? 18.0 : 9.0) * K * V + 4.0 * steps + (bwd ? 9.0 : 6.0) * K + 25.0);
            if (cost < best) { best = cost; q.V = V; q.K = K; q.L = L; }
        }
    }
    if (best == 1e30) return q;
    const int teams = GN_THREADS / q.L;
    q.gpc = std::min(p.G, teams);
    q.spc = std::max(1, std::min(teams / q.gpc, std::max(1, p.B)));
    q.threads = round_up(q.gpc * q.spc * q.L, 32);
    q.gsets = ceil_div(p.G, q.gpc);
    const int per_sm = std::max(1, (bwd ? 512 : 1024) / q.threads);
    const int want = std::max(1, d.sms * per_sm / q.gsets);
    q.chunks = std::min(ceil_div(std::max(1, p.B), q.spc), want);
    if (bwd) q.chunks = gn_bounded_chunks(q.chunks, ceil_div(std::max(1, p.B), q.spc));
    q.dm_cgv = FastDivmod(uint32_t(std::max(1, p.Cg / q.V)));
    q.dm_p = FastDivmod(uint32_t(p.P));
    q.dm_cg = FastDivmod(uint32_t(p.Cg));
    q.dm_m = FastDivmod(uint32_t(p.M));
    q.ok = true;
    return q;
}

GnPieces gn_pieces(const GnParams& p, int dt, const DevInfo& d)
{
    GnPieces q = {};
    const int es = dt == DT_F32 ? 4 : 2;
    q.threads = 256;
    int v = 16 / es;
    while (v > 1 && p.P % v != 0) v /= 2;
    q.V = v;
    const int U = 4;  // vectors a thread merges at a time
    // two merges a thread while that leaves enough pieces for the SMs
    int len = q.threads * U * v * 2;
    while (len > q.threads * v && int64_t(p.B) * p.C * ceil_div(p.P, len) < 4 * d.sms) len /= 2;
    q.len = std::min(len, p.P);
    // rows of at most U vectors a lane of a warp: a warp each, eight rows a block
    q.row_lanes = p.P <= 32 * U * v ? 32 : q.threads;
    if (q.row_lanes == 32) q.len = p.P;
    q.pieces = ceil_div(p.P, q.len);
    const int rows = q.threads / q.row_lanes;
    q.blocks = (int64_t(p.B) * p.C * q.pieces + rows - 1) / rows;
    return q;
}

namespace {

// ---- small groups ----------------------------------------------------------------------------
// 32768 x 128 x 12, 16 groups, bf16, SiLU: 41 us, 5.1 TB/s, 76% of the measured copy's; bound by
// instructions (22 a value, of which the activation takes 4, at 0.71 an issue slot), as two
// samples read ahead instead of one change nothing.  fp32, 8192 x 128 x 12: 22 us, 4.5 TB/s.
// 256 x 128 x 2, 8 groups: 5 to 6 us, a launch.  Groups of up to 384 (bf16: 512) values; beside a
// cluster's (us): 1024 x 256 x 36, 32 groups, 17 / 25 bf16 and 19 / 23 fp32.
template <typename T, int V, int K>
__global__ void __launch_bounds__(GN_THREADS, 4)
gn_team_fwd(const GnParams p, const GnTeam q, const T* x, const T* gamma, const T* beta, T* y, float* mean_out,
            float* rstd_out)
{
    constexpr int H = K * V / 2;  // pairs of values
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
    Vec<T, V> raw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].zero();
    auto fetch = [&](int at) {
        if (at >= p.B) return;
        const T* px = x + int64_t(at) * p.N;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (has[k]) raw[k].load(px + off[k]);
    };
    tc::grid_dep_wait();
    fetch(b);
    gn_team_tables(p, q, g0, gamma, beta, tab, tab + q.gpc * m);
    __syncthreads();
    const float *gam = tab + gi * m, *bet = gam + q.gpc * m;
#pragma unroll 1
    for (int it = 0; it < iters; ++it, b += step) {
        float2 v[H], s = both(0.f);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            v[h] = pair_of<T, V, K>(raw, h);
            s = add2(s, v[h]);
        }
        if (it + 1 < iters) fetch(b + step);
        const float mean = div_m(p, team_sum(s.x + s.y, L));
        s = both(0.f);
#pragma unroll
        for (int h = 0; h < H; ++h) {  // a lane's vectors beyond the group stay zero
            v[h] = add2(v[h], make_float2(has[2 * h / V] ? -mean : 0.f, has[(2 * h + 1) / V] ? -mean : 0.f));
            s = fma2(v[h], v[h], s);
        }
        const float rstd = rsqrtf(team_sum(s.x + s.y, L) * p.inv_m + p.eps);
        if (active && b < p.B) {
            T* py = y + int64_t(b) * p.N;
            float2 w[H];
            table_pairs<V, K>(gam, toff, w);
#pragma unroll
            for (int h = 0; h < H; ++h) v[h] = mul2(mul2(v[h], both(rstd)), w[h]);  // x - mean, rounded, is in v
            table_pairs<V, K>(bet, toff, w);
            with_act(p.act, [&](auto act) {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float2 z = act.value == CONV_ACT_RELU ? add2_apart(v[h], w[h]) : add2(v[h], w[h]);
                    v[h] = act_value<act.value>(z);
                }
            });
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float r[V];
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] = (k * V + i) % 2 ? v[(k * V + i) / 2].y : v[(k * V + i) / 2].x;
                Vec<T, V> o;
                o.set(r);
                if (has[k]) o.store(py + off[k]);
            }
            if (lane == 0 && mean_out) {
                mean_out[int64_t(b) * p.G + g] = mean;
                rstd_out[int64_t(b) * p.G + g] = rstd;
            }
        }
    }
}

// ---- large groups, NCHW ------------------------------------------------------------------------
// Two passes over x, the second out of L2 as far as it holds: 4 x 128 x 16384, 8 groups, SiLU: 16 us
// in bf16 and 25 in fp32 (2.1 and 2.8 TB/s of one read and one write); three launches.
// A running (mean, M2) over n values, and the merge of another (n2, mean2, m22).
__device__ __forceinline__ void chan_merge(float& n, float& mean, float& m2, float n2, float mean2, float m22)
{
    const float t = n + n2;
    if (n2 == 0.f) return;
    const float dlt = mean2 - mean, w = __fdividef(n2, t);
    mean += dlt * w;
    m2 += m22 + dlt * dlt * n * w;
    n = t;
}

// A block (or a warp) a row's piece.
template <typename T, int V>
__global__ void __launch_bounds__(256) gn_stats(const GnParams p, const GnPieces q, const T* x, float* pmean,
                                                     float* pm2)
{
    constexpr int U = 4;
    __shared__ float sm[8][3];
    const GnRow t(p, q, V, blockIdx.x);
    const T* px = x + t.row * p.P;
    float n = 0.f, mean = 0.f, m2 = 0.f;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    for (int e = t.e0; e < t.e1; e += t.hop * U) {
        Vec<T, V> v[U];
        int cnt = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (e + u * t.hop < t.e1) { v[u].load(px + e + u * t.hop); cnt += V; }
            else v[u].zero();
        }
        float s = 0.f, sq = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) s += v[u].get(i);
        const float mu = __fdiv_rn(s, float(cnt));
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float dlt = u * V < cnt ? v[u].get(i) - mu : 0.f;
                sq += dlt * dlt;
            }
        chan_merge(n, mean, m2, float(cnt), mu, sq);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float n2 = __shfl_down_sync(0xFFFFFFFFu, n, o), mean2 = __shfl_down_sync(0xFFFFFFFFu, mean, o),
                    m22 = __shfl_down_sync(0xFFFFFFFFu, m2, o);
        chan_merge(n, mean, m2, n2, mean2, m22);
    }
    if (q.row_lanes > 32) {
        if ((threadIdx.x & 31) == 0) {
            sm[threadIdx.x >> 5][0] = n;
            sm[threadIdx.x >> 5][1] = mean;
            sm[threadIdx.x >> 5][2] = m2;
        }
        __syncthreads();
        if (t.lane == 0)
            for (int w = 1; w < q.row_lanes / 32; ++w) chan_merge(n, mean, m2, sm[w][0], sm[w][1], sm[w][2]);
    }
    if (t.lane == 0 && t.in) {
        const int64_t b = t.row / p.C, o = gn_part(p, q.pieces, b, int(t.row - b * p.C), t.pc);
        pmean[o] = mean;
        pm2[o] = m2;
    }
}

// One block a group: the mean from the pieces' means, then the squares about it.
__global__ void __launch_bounds__(128) gn_combine(const GnParams p, const GnPieces q, const float* pmean,
                                                  const float* pm2, float* mean, float* rstd, float* mean_out,
                                                  float* rstd_out)
{
    __shared__ float sm[64];
    int turn = 0;
    const int b = int(blockIdx.x / p.G), g = int(blockIdx.x % p.G);
    const int np = p.Cg * q.pieces;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float s = 0.f;
    auto at = [&](int i, int& cnt) {
        const int pc = i / p.Cg, cl = i - pc * p.Cg;
        cnt = min(q.len, p.P - pc * q.len);
        return gn_part(p, q.pieces, b, g * p.Cg + cl, pc);
    };
    gn_stretches(np, s, [&](int i, float& some) {
        int cnt;
        const int64_t o = at(i, cnt);
        some += pmean[o] * float(cnt);
    });
    const float mu = __fdiv_rn(block_total(s, sm, turn), p.m);
    float v = 0.f;
    gn_stretches(np, v, [&](int i, float& some) {
        int cnt;
        const int64_t o = at(i, cnt);
        const float dlt = pmean[o] - mu;
        some += pm2[o] + dlt * dlt * float(cnt);
    });
    const float r = rsqrtf(block_total(v, sm, turn) * p.inv_m + p.eps);
    if (threadIdx.x == 0) {
        mean[blockIdx.x] = mu;
        rstd[blockIdx.x] = r;
        if (mean_out) {
            mean_out[blockIdx.x] = mu;
            rstd_out[blockIdx.x] = r;
        }
    }
}

// The second pass walks the pieces backwards: the first pass's last pieces are still in L2.
template <typename T, int V>
__global__ void __launch_bounds__(256) gn_apply(const GnParams p, const GnPieces q, const T* x, const T* gamma,
                                                     const T* beta, T* y, const float* mean, const float* rstd)
{
    constexpr int U = 4;
    const GnRow t(p, q, V, q.blocks - 1 - blockIdx.x);
    tc::grid_dep_wait();
    if (!t.in) return;
    const int c = int(t.row % p.C);
    const int64_t grp = t.row / p.C * p.G + c / p.Cg;
    const float mu = mean[grp], rs = rstd[grp];
    const float ga = gamma ? Elem<T>::ldg(gamma + c) : 1.f, be = beta ? Elem<T>::ldg(beta + c) : 0.f;
    const T* px = x + t.row * p.P;
    T* py = y + t.row * p.P;
    with_act(p.act, [&](auto act) {
        for (int e = t.e0; e < t.e1; e += t.hop * U) {
            Vec<T, V> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u * t.hop < t.e1) v[u].load(px + e + u * t.hop);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e + u * t.hop < t.e1) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = act_value<act.value>(gn_z(gn_xhat(v[u].get(i), mu, rs), ga, be));
                    v[u].set(o);
                    v[u].store(py + e + u * t.hop);
                }
        }
    });
}

template <typename T>
cudaError_t fwd_t(const GnParams& p, int dt, const DevInfo& d, const T* x, const T* gamma, const T* beta, T* y,
                  float* mean, float* rstd, void* ws, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    const GnTeam t = gn_team(p, dt, d, false);
    if (t.ok) {
        const GnTeam& q = t;
        const dim3 grid(unsigned(q.gsets) * unsigned(q.chunks)), block(q.threads);
        const size_t smem = size_t(8) * q.gpc * size_t(p.M);
#define GN_CALL(T_, V_, K_) \
    e = launch_ex(gn_team_fwd<T_, V_, K_>, grid, block, smem, s, 1, true, p, q, x, gamma, beta, y, mean, rstd)
        GN_DISPATCH_TEAM(T, true, GN_CALL);
#undef GN_CALL
        return e != cudaSuccess ? e : cudaGetLastError();
    }
    const GnCluster cl = gn_cluster(p, dt, d, false);
    if (cl.ok) return run_gn_cluster_fwd(p, cl, dt, x, gamma, beta, y, mean, rstd, s);
    if (gn_by_rows(p)) return run_gn_rows_fwd(p, gn_rows(p, dt, d, false), dt, x, gamma, beta, y, mean, rstd, ws, s);
    const GnPieces q = gn_pieces(p, dt, d);
    const int64_t np = int64_t(p.B) * p.C * q.pieces;
    float* pmean = static_cast<float*>(ws);
    float* pm2 = pmean + np;
    float* mu = pm2 + np;
    float* rs = mu + int64_t(p.B) * p.G;
    const dim3 grid(static_cast<unsigned>(q.blocks));
#define GN_CALL(T_, V_) e = launch_ex(gn_stats<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, pmean, pm2)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    if (e != cudaSuccess) return e;
    e = launch_ex(gn_combine, dim3(unsigned(p.B) * unsigned(p.G)), dim3(128), 0, s, 1, true, p, q,
                  static_cast<const float*>(pmean), static_cast<const float*>(pm2), mu, rs, mean, rstd);
    if (e != cudaSuccess) return e;
#define GN_CALL(T_, V_)                                                                                      \
    e = launch_ex(gn_apply<T_, V_>, grid, dim3(q.threads), 0, s, 1, true, p, q, x, gamma, beta, y,           \
                  static_cast<const float*>(mu), static_cast<const float*>(rs))
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t gn_fwd_workspace(const GnParams& p, int dt, const DevInfo& d)
{
    if (p.B == 0 || gn_team(p, dt, d, false).ok || gn_cluster(p, dt, d, false).ok) return 0;
    if (gn_by_rows(p)) return size_t(8) * p.B * p.G * gn_rows(p, dt, d, false).parts;
    const GnPieces q = gn_pieces(p, dt, d);
    return size_t(4) * (2 * size_t(p.B) * p.C * q.pieces + 2 * size_t(p.B) * p.G);
}

cudaError_t run_gn_fwd(const GnParams& p, int dt, const DevInfo& d, const void* x, const void* gamma,
                       const void* beta, void* y, float* mean, float* rstd, void* ws, cudaStream_t s)
{
    if (dt == DT_F32)
        return fwd_t<float>(p, dt, d, (const float*)x, (const float*)gamma, (const float*)beta, (float*)y, mean, rstd,
                            ws, s);
    using H = __nv_bfloat16;
    return fwd_t<H>(p, dt, d, (const H*)x, (const H*)gamma, (const H*)beta, (H*)y, mean, rstd, ws, s);
}

}  // namespace igc
