// kernels_gn_nhwc.cu -- channels-last group norm of groups too large for a team of lanes: two
// streaming passes over row tiles, the second one out of L2 as far as it holds.
//
// A thread keeps its columns (V consecutive channels) and walks rows, so everything that depends
// on the channel sits in registers, loads are whole row segments, and a value costs little more
// than its own arithmetic -- which is what bounds these kernels in bf16 (about 12 instructions a
// value over both passes of the forward, 30 of the backward, against 4 and 6 bytes).  The first
// pass leaves each tile's groups' partial results; the second one's blocks merge those of their
// groups first (a few hundred numbers), so no launch stands between the passes.  The second pass
// walks the tiles backwards: the first pass's last tiles are the ones still in L2.
//
// Measured (no cluster holds a group's window of 136 channels): 8 x 3860 x 1088, 32 groups, SiLU: forward 72
// us in bf16 and 114 in fp32, backward 150 and 187 (with its channels' sums): 1.9, 2.4, 1.3 and 2.2 TB/s of
// one read of each input and one write.
#include "gn_common.cuh"

namespace igc {

namespace {

constexpr int GR_THREADS = 256;
constexpr int GR_MAX_PARTS = 256;   // partial results of a group

}  // namespace

GnRows gn_rows(const GnParams& p, int dt, const DevInfo& d, bool bwd)
{
    GnRows q = {};
    const int es = dt == DT_F32 ? 4 : 2;
    // the backward keeps six numbers a channel: 4 channels a thread leave it 64 registers
    q.V = bwd ? 4 : 16 / es;
    while (p.C % q.V != 0) q.V /= 2;
    int lcm = p.Cg;
    while (lcm % q.V != 0) lcm += p.Cg;
    if (lcm / q.V <= GR_THREADS) {  // windows of whole groups
        q.per = 1;
        q.W = lcm * std::min(GR_THREADS / (lcm / q.V), p.C / lcm);
        q.wins = ceil_div(p.C, q.W);
        // windows of about equal widths
        q.W = ceil_div(p.C / lcm, q.wins) * lcm;
        q.wins = ceil_div(p.C, q.W);
    } else {  // a group in several windows
        while (p.Cg % q.V != 0) q.V /= 2;
        q.per = ceil_div(p.Cg / q.V, GR_THREADS);
        q.W = ceil_div(p.Cg / q.V, q.per) * q.V;
        q.per = ceil_div(p.Cg, q.W);
        q.wins = p.G * q.per;
    }
    q.cols = q.W / q.V;
    q.lanes = std::max(1, std::min(GR_THREADS / q.cols, p.P));
    q.threads = round_up(q.lanes * q.cols, 32);
    // Rows a thread: 16 where that fills the SMs, down to 4; more where a group would have more
    // partial results than the second pass should merge.  The backward's sums over a thread's rows are
    // one chain of additions each, so it takes GN_CHAIN rows at most (2048 rows of equal values lost
    // 2.3e-5 of their sum; a second accumulator in the loop costs registers, and 3 to 12%).
    int R = 16;
    const int most = bwd ? GN_CHAIN : INT32_MAX;
    while (R > 4 && int64_t(p.B) * q.wins * ceil_div(p.P, q.lanes * R) < 6 * d.sms) R /= 2;
    while (int64_t(ceil_div(p.P, q.lanes * R)) * q.per > GR_MAX_PARTS && q.lanes * R < p.P && R < most) R *= 2;
    // A block of the second pass merges the partial results of all its window's groups: longer
    // tiles while those are more than a quarter of the tile's bytes (backward: half of one tensor's;
    // its merge is two additions) and the SMs stay filled (8 x 3860 x 1088 bf16, 32 groups a window,
    // forward: 16 rows 121 us, 64 rows 70; 6 x 13115 x 224 bf16, 8 groups, backward: 64 rows 72, 128 82).
    const int64_t groups = q.per == 1 ? q.W / p.Cg : 1;
    while (int64_t(ceil_div(p.P, q.lanes * R)) * q.per * groups * (bwd ? 16 : 32) > int64_t(q.lanes) * R * q.W * es &&
           int64_t(p.B) * q.wins * ceil_div(p.P, q.lanes * R * 2) >= 2 * d.sms && R < most)
        R *= 2;
    q.len = int(std::min<int64_t>(p.P, int64_t(q.lanes) * R));
    q.pieces = ceil_div(p.P, q.len);
    q.parts = q.pieces * q.per;
    q.blocks = int64_t(p.B) * q.pieces * q.wins;
    q.dm_cols = FastDivmod(uint32_t(q.cols));
    q.dm_cg = FastDivmod(uint32_t(p.Cg));
    q.dm_wins = FastDivmod(uint32_t(q.wins));
    q.dm_pieces = FastDivmod(uint32_t(q.pieces));
    q.dm_per = FastDivmod(uint32_t(q.per));
    return q;
}

namespace {

// A block's tile: rows [r0, r1) of W channels from c0; thread (lane, col) the vector `col` of the
// rows r0 + lane, r0 + lane + lanes, ...
struct GrTile {
    int b, pc, part, c0, W, groups, g0, lane, col, r0, r1, mine, full, extra;
    bool in;
    __device__ __forceinline__ GrTile(const GnParams& p, const GnRows& q, uint32_t at)
    {
        uint32_t a, w, x;
        q.dm_wins.divmod(at, a, w);
        q.dm_pieces.divmod(a, x, a);
        b = int(x);
        pc = int(a);
        if (q.per == 1) {
            part = 0;
            c0 = int(w) * q.W;
            W = min(q.W, p.C - c0);
            groups = int(q.dm_cg.div(uint32_t(W)));
            g0 = int(q.dm_cg.div(uint32_t(c0)));
        } else {
            q.dm_per.divmod(w, x, a);
            g0 = int(x);
            part = int(a);
            c0 = g0 * p.Cg + part * q.W;
            W = min(q.W, p.Cg - part * q.W);
            groups = 1;
        }
        q.dm_cols.divmod(threadIdx.x, x, a);
        lane = int(x);
        col = int(a);
        r0 = pc * q.len;
        r1 = r0 + min(p.P - r0, q.len);  // (r0 + len may pass 2^31)
        full = (r1 - r0) / q.lanes;
        extra = r1 - r0 - full * q.lanes;
        in = lane < q.lanes && col * q.V < W;
        mine = in ? full + (lane < extra) : 0;
    }
    // the group (in the tile) of the tile's channel c
    __device__ __forceinline__ int group(const GnRows& q, int c) const
    {
        return q.per == 1 ? int(q.dm_cg.div(uint32_t(c))) : 0;
    }
};
// Values of the group that partial e stands for.
__device__ __forceinline__ float gr_count(const GnParams& p, const GnRows& q, int e)
{
    uint32_t pc, part;
    q.dm_per.divmod(uint32_t(e), pc, part);
    const int width = q.per == 1 ? p.Cg : min(q.W, p.Cg - int(part) * q.W);
    return float(min(q.len, p.P - int(pc) * q.len)) * float(width);
}

template <typename T, int V> __device__ __forceinline__ void gr_pairs(const Vec<T, V>& v, float2 (&f)[(V + 1) / 2])
{
#pragma unroll
    for (int h = 0; h < (V + 1) / 2; ++h) f[h] = make_float2(v.get(2 * h), 2 * h + 1 < V ? v.get(2 * h + 1) : 0.f);
}
template <typename T, int V> __device__ __forceinline__ void gr_store(T* p, const float2 (&f)[(V + 1) / 2])
{
    float r[V];
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = i % 2 ? f[i / 2].y : f[i / 2].x;
    Vec<T, V> v;
    v.set(r);
    v.store(p);
}
// Pairs of f(channel) over the thread's channels.
template <int V, class F> __device__ __forceinline__ void gr_params(float2 (&v)[(V + 1) / 2], F&& f)
{
#pragma unroll
    for (int h = 0; h < (V + 1) / 2; ++h) v[h] = make_float2(f(2 * h), f(2 * h + 1 < V ? 2 * h + 1 : 2 * h));
}

// First pass of the forward.  A thread's sums of a column, d and d^2, are about a pivot: the first
// value it reads, then, after 16, 32 and 64 rows and every 64 from there, the mean so far.  So
// few rows are summed about a value that may be far off, and what is subtracted stays within a
// small factor of the column's own spread, whatever its offset; the squares of each stretch are
// summed apart, so no chain is longer than 64 rows and the stretches.  A thread takes as many rows
// as gn_rows gives it, some thousands for the longest samples.  (With the first value as the pivot
// of all rows, one value far off at the start cost rstd 1.8e-4 at 128 rows and 1.2e-2 at 1024.)
// out: (sample, group, part) x (mean, M2).
template <typename T, int V>
__global__ void __launch_bounds__(GR_THREADS)
gn_rows_stats(const GnParams p, const __grid_constant__ GnRows q, const T* x, float2* out)
{
    constexpr int H = (V + 1) / 2, U = 4;
    __shared__ float2 rec[GR_THREADS * V];  // (mean, M2) of (row lane, channel)
    const GrTile t(p, q, blockIdx.x);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (t.mine) {
        const T* px = x + int64_t(t.b) * p.N + t.c0 + t.col * V + int64_t(t.r0 + t.lane) * p.C;
        const int64_t hop = int64_t(q.lanes) * p.C;
        float2 c[H], s[H], sq[H];  // minus the pivot; sums about it
        float2* r = rec + t.lane * t.W + t.col * V;  // .y: the squares of earlier stretches
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < t.mine) v[u].load(px + u * hop);
        gr_pairs<T, V>(v[0], c);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            c[h] = mul2(c[h], both(-1.f));
            s[h] = sq[h] = both(0.f);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) r[i].y = 0.f;
        static_assert(16 % U == 0, "a stretch ends between two steps");
#pragma unroll 1
        for (int k = 0, stop = 16;; stop += min(stop, 64)) {
            for (; k < min(stop, t.mine); k += U) {
                Vec<T, V> w[U];
                px += U * hop;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    w[u] = v[u];
                    if (k + U + u < t.mine) v[u].load(px + u * hop);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k + u < t.mine) {
                        float2 f[H];
                        gr_pairs<T, V>(w[u], f);
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            f[h] = add2(f[h], c[h]);
                            s[h] = add2(s[h], f[h]);
                            sq[h] = fma2(f[h], f[h], sq[h]);
                        }
                    }
            }
            if (k >= t.mine) break;
            recentre<H>(c, s, sq, float(k));
#pragma unroll
            for (int i = 0; i < V; ++i) r[i].y += i % 2 ? sq[i / 2].y : sq[i / 2].x;
#pragma unroll
            for (int h = 0; h < H; ++h) sq[h] = both(0.f);
        }
        const float inv = __fdividef(1.f, float(t.mine));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float sc = i % 2 ? s[i / 2].y : s[i / 2].x, qc = r[i].y + (i % 2 ? sq[i / 2].y : sq[i / 2].x);
            const float mu = sc * inv;
            r[i] = make_float2(mu - (i % 2 ? c[i / 2].y : c[i / 2].x), fmaxf(0.f, fmaf(-sc, mu, qc)));
            if (qc != qc) r[i].y = qc;  // NaN stays
        }
    }
    __syncthreads();
    // A warp a group: the mean of its records' means, then the squares about it.
    const int width = q.per == 1 ? p.Cg : t.W, lanes = min(q.lanes, t.r1 - t.r0);
    int cw = 1;  // channels side by side in the warp
    while (cw < 32 && cw < width) cw *= 2;
    const int wl = int(threadIdx.x & 31);
    for (int g = int(threadIdx.x >> 5); g < t.groups; g += int(blockDim.x) >> 5) {
        const float n = float(t.r1 - t.r0) * float(width);
        float mean = 0.f, m2 = 0.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            float a = 0.f;
            for (int l = wl / cw; l < lanes; l += 32 / cw) {
                const float rows = float(t.full + (l < t.extra));
                for (int c = wl & (cw - 1); c < width; c += cw) {
                    const float2 r = rec[l * t.W + g * width + c];
                    const float dlt = r.x - mean;
                    a += pass == 0 ? rows * r.x : fmaf(rows * dlt, dlt, r.y);
                }
            }
            a = warp_sum(a);
            if (pass == 0) mean = __fdiv_rn(a, n);
            else m2 = a;
        }
        if (wl == 0)
            out[(int64_t(t.b) * p.G + t.g0 + g) * q.parts + t.pc * q.per + t.part] = make_float2(mean, m2);
    }
}

// Second pass of the forward.
template <typename T, int V>
__global__ void __launch_bounds__(GR_THREADS)
gn_rows_apply(const GnParams p, const __grid_constant__ GnRows q, const T* x, const T* gamma, const T* beta, T* y,
              const float2* in, float* mean_out, float* rstd_out)
{
    constexpr int H = (V + 1) / 2, U = 4;
    __shared__ float2 stat[GR_THREADS * V];  // (mean, rstd) of the tile's groups
    const GrTile t(p, q, uint32_t(q.blocks - 1 - blockIdx.x));
    const int c0 = t.c0 + (t.in ? t.col * V : 0);
    tc::grid_dep_wait();
    const T* px = x + int64_t(t.b) * p.N + c0 + int64_t(t.r0 + t.lane) * p.C;
    T* py = y + (px - x);
    const int64_t hop = int64_t(q.lanes) * p.C;
    Vec<T, V> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u < t.mine) v[u].load(px + u * hop);
    const int wl = int(threadIdx.x & 31);
    for (int g = int(threadIdx.x >> 5); g < t.groups; g += int(blockDim.x) >> 5) {
        const float2* r = in + (int64_t(t.b) * p.G + t.g0 + g) * q.parts;
        float mean = 0.f, rstd = 0.f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            float a = 0.f;
#pragma unroll 4
            for (int e = wl; e < q.parts; e += 32) {
                const float2 f = r[e];
                const float n = gr_count(p, q, e), dlt = f.x - mean;
                a += pass == 0 ? n * f.x : fmaf(n * dlt, dlt, f.y);
            }
            a = warp_sum(a);
            if (pass == 0) mean = div_m(p, a);
            else rstd = rsqrtf(a * p.inv_m + p.eps);
        }
        if (wl == 0) {
            stat[g] = make_float2(mean, rstd);
            if (mean_out && t.pc == 0 && t.part == 0) {
                mean_out[int64_t(t.b) * p.G + t.g0 + g] = mean;
                rstd_out[int64_t(t.b) * p.G + t.g0 + g] = rstd;
            }
        }
    }
    __syncthreads();
    if (!t.mine) return;
    float2 mu[H], rs[H], ga[H], be[H];
    gr_params<V>(mu, [&](int i) { return -stat[t.group(q, t.col * V + i)].x; });
    gr_params<V>(rs, [&](int i) { return stat[t.group(q, t.col * V + i)].y; });
    gr_params<V>(ga, [&](int i) { return gamma ? Elem<T>::ldg(gamma + c0 + i) : 1.f; });
    gr_params<V>(be, [&](int i) { return beta ? Elem<T>::ldg(beta + c0 + i) : 0.f; });
    with_act(p.act, [&](auto act) {
        if constexpr (act.value != CONV_ACT_RELU)
#pragma unroll
            for (int h = 0; h < H; ++h) ga[h] = mul2(ga[h], rs[h]);
        for (int k = 0; k < t.mine; k += U, px += U * hop, py += U * hop) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k + u < t.mine) {
                    float2 f[H];
                    gr_pairs<T, V>(v[u], f);
                    if (k + U + u < t.mine) v[u].load(px + (U + u) * hop);
#pragma unroll
                    for (int h = 0; h < H; ++h) f[h] = gn_out<act.value>(add2(f[h], mu[h]), rs[h], ga[h], be[h]);
                    gr_store<T, V>(py + u * hop, f);
                }
        }
    });
}

// First pass of the backward: each channel's sums of dz*xhat and dz over the tile (part, rows
// (sample, piece) of dgamma's, then dbeta's), and each group's of dz*gamma*xhat and dz*gamma.
template <typename T, int V>
__global__ void __launch_bounds__(GR_THREADS, 4)
gn_rows_sums(const GnParams p, const __grid_constant__ GnRows q, const T* x, const T* dy, const T* gamma,
             const T* beta, const float* mean, const float* rstd, float2* out, float* part)
{
    constexpr int H = (V + 1) / 2, U = 2;
    __shared__ float2 rec[GR_THREADS * V];   // (row lane, channel)
    __shared__ float2 sums[GR_THREADS * V];  // channel
    const GrTile t(p, q, blockIdx.x);
    const int c0 = t.c0 + (t.in ? t.col * V : 0);
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (t.mine) {
        const int64_t at = int64_t(t.b) * p.N + c0 + int64_t(t.r0 + t.lane) * p.C, hop = int64_t(q.lanes) * p.C;
        const T *px = x + at, *pd = dy + at;
        Vec<T, V> vx[U], vd[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < t.mine) {
                vx[u].load(px + u * hop);
                vd[u].load(pd + u * hop);
            }
        float2 mu[H], rs[H], ga[H], be[H], sg[H], sb[H];
        const int64_t g0 = int64_t(t.b) * p.G + t.g0;
        gr_params<V>(mu, [&](int i) { return -mean[g0 + t.group(q, t.col * V + i)]; });
        gr_params<V>(rs, [&](int i) { return rstd[g0 + t.group(q, t.col * V + i)]; });
        gr_params<V>(ga, [&](int i) { return gamma ? Elem<T>::ldg(gamma + c0 + i) : 1.f; });
        gr_params<V>(be, [&](int i) { return beta ? Elem<T>::ldg(beta + c0 + i) : 0.f; });
#pragma unroll
        for (int h = 0; h < H; ++h) sg[h] = sb[h] = both(0.f);
        with_act(p.act, [&](auto act) {
            for (int k = 0; k < t.mine; k += U, px += U * hop, pd += U * hop) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (k + u < t.mine) {
                        float2 xh[H], dz[H];
                        gr_pairs<T, V>(vx[u], xh);
                        gr_pairs<T, V>(vd[u], dz);
                        if (k + U + u < t.mine) {
                            vx[u].load(px + (U + u) * hop);
                            vd[u].load(pd + (U + u) * hop);
                        }
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            xh[h] = mul2(add2(xh[h], mu[h]), rs[h]);
                            dz[h] = gn_grad<act.value>(dz[h], xh[h], ga[h], be[h]);
                            sb[h] = add2(sb[h], dz[h]);
                            sg[h] = fma2(dz[h], xh[h], sg[h]);
                        }
                    }
            }
        });
        float2* r = rec + t.lane * t.W + t.col * V;
#pragma unroll
        for (int i = 0; i < V; ++i)
            r[i] = i % 2 ? make_float2(sg[i / 2].y, sb[i / 2].y) : make_float2(sg[i / 2].x, sb[i / 2].x);
    }
    __syncthreads();
    // channels' sums over the row lanes: `team` lanes a channel, in a fixed order
    const int lanes = min(q.lanes, t.r1 - t.r0), nt = int(blockDim.x);
    int team = 1;
    while (team < 32 && team * 2 * t.W <= nt && team * 2 <= lanes) team *= 2;
    const int64_t row = int64_t(t.b) * q.pieces + t.pc;
    for (int i0 = 0; i0 < t.W * team; i0 += nt) {
        const int i = i0 + int(threadIdx.x), c = i / team;
        float2 s = both(0.f);
        if (c < t.W)
            for (int l = i & (team - 1); l < lanes; l += team) s = add2(s, rec[l * t.W + c]);
        s = make_float2(team_sum(s.x, team), team_sum(s.y, team));
        if (c < t.W && (i & (team - 1)) == 0) {
            sums[c] = s;
            if (part) {
                part[row * 2 * p.C + t.c0 + c] = s.x;
                part[(row * 2 + 1) * p.C + t.c0 + c] = s.y;
            }
        }
    }
    __syncthreads();
    const int width = q.per == 1 ? p.Cg : t.W, wl = int(threadIdx.x & 31);
    for (int g = int(threadIdx.x >> 5); g < t.groups; g += nt >> 5) {
        float2 s = both(0.f);
        for (int c = g * width + wl; c < (g + 1) * width; c += 32)
            s = fma2(sums[c], both(gamma ? Elem<T>::ldg(gamma + t.c0 + c) : 1.f), s);
        s = make_float2(warp_sum(s.x), warp_sum(s.y));
        if (wl == 0) out[(int64_t(t.b) * p.G + t.g0 + g) * q.parts + t.pc * q.per + t.part] = s;
    }
}

// Second pass of the backward.
template <typename T, int V>
__global__ void __launch_bounds__(GR_THREADS, 4)
gn_rows_dx(const GnParams p, const __grid_constant__ GnRows q, const T* x, const T* dy, const T* gamma,
           const T* beta, const float* mean, const float* rstd, T* dx, const float2* in)
{
    constexpr int H = (V + 1) / 2, U = 2;
    __shared__ float2 sums[GR_THREADS * V];  // (m2, m1) of the tile's groups
    const GrTile t(p, q, uint32_t(q.blocks - 1 - blockIdx.x));
    const int c0 = t.c0 + (t.in ? t.col * V : 0);
    tc::grid_dep_wait();
    const int64_t at = int64_t(t.b) * p.N + c0 + int64_t(t.r0 + t.lane) * p.C, hop = int64_t(q.lanes) * p.C;
    const T *px = x + at, *pd = dy + at;
    T* po = dx + at;
    Vec<T, V> vx[U], vd[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u < t.mine) {
            vx[u].load(px + u * hop);
            vd[u].load(pd + u * hop);
        }
    const int wl = int(threadIdx.x & 31);
    const int64_t g0 = int64_t(t.b) * p.G + t.g0;
    for (int g = int(threadIdx.x >> 5); g < t.groups; g += int(blockDim.x) >> 5) {
        const float2* r = in + (g0 + g) * q.parts;
        float2 s = both(0.f);
#pragma unroll 4
        for (int e = wl; e < q.parts; e += 32) s = add2(s, r[e]);
        s = make_float2(warp_sum(s.x), warp_sum(s.y));
        if (wl == 0) sums[g] = mul2(s, both(p.inv_m));
    }
    __syncthreads();
    if (!t.mine) return;
    float2 mu[H], rs[H], ga[H], be[H], m1[H], m2[H];
    gr_params<V>(mu, [&](int i) { return -mean[g0 + t.group(q, t.col * V + i)]; });
    gr_params<V>(rs, [&](int i) { return rstd[g0 + t.group(q, t.col * V + i)]; });
    gr_params<V>(ga, [&](int i) { return gamma ? Elem<T>::ldg(gamma + c0 + i) : 1.f; });
    gr_params<V>(be, [&](int i) { return beta ? Elem<T>::ldg(beta + c0 + i) : 0.f; });
    gr_params<V>(m1, [&](int i) { return -sums[t.group(q, t.col * V + i)].y; });
    gr_params<V>(m2, [&](int i) { return -sums[t.group(q, t.col * V + i)].x; });
    with_act(p.act, [&](auto act) {
        for (int k = 0; k < t.mine; k += U, px += U * hop, pd += U * hop, po += U * hop) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (k + u < t.mine) {
                    float2 xh[H], dz[H];
                    gr_pairs<T, V>(vx[u], xh);
                    gr_pairs<T, V>(vd[u], dz);
                    if (k + U + u < t.mine) {
                        vx[u].load(px + (U + u) * hop);
                        vd[u].load(pd + (U + u) * hop);
                    }
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        xh[h] = mul2(add2(xh[h], mu[h]), rs[h]);
                        dz[h] = gn_grad<act.value>(dz[h], xh[h], ga[h], be[h]);
                        xh[h] = mul2(rs[h], fma2(xh[h], m2[h], fma2(dz[h], ga[h], m1[h])));
                    }
                    gr_store<T, V>(po + u * hop, xh);
                }
        }
    });
}

template <typename T>
cudaError_t rows_fwd_t(const GnParams& p, const GnRows& q, const T* x, const T* gamma, const T* beta, T* y,
                       float* mean, float* rstd, void* ws, cudaStream_t s)
{
    float2* st = static_cast<float2*>(ws);
    const float2* in = st;
    const dim3 grid(static_cast<unsigned>(q.blocks)), block(q.threads);
    cudaError_t e = cudaSuccess;
#define GN_CALL(T_, V_)                                                                                      \
    do {                                                                                                     \
        e = launch_ex(gn_rows_stats<T_, V_>, grid, block, 0, s, 1, true, p, q, x, st);                       \
        if (e == cudaSuccess)                                                                                \
            e = launch_ex(gn_rows_apply<T_, V_>, grid, block, 0, s, 1, true, p, q, x, gamma, beta, y, in,    \
                          mean, rstd);                                                                       \
    } while (0)
    GN_DISPATCH_V(T, q.V, GN_CALL);
#undef GN_CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t rows_bwd_t(const GnParams& p, const GnRows& q, const T* x, const T* dy, const T* gamma, const T* beta,
                       const float* mean, const float* rstd, T* dx, float* part, void* ws, cudaStream_t s)
{
    float2* st = static_cast<float2*>(ws);
    const float2* in = st;
    const dim3 grid(static_cast<unsigned>(q.blocks)), block(q.threads);
    cudaError_t e = cudaSuccess;
#define GN_CALL(T_, V_)                                                                                      \
    do {                                                                                                     \
        e = launch_ex(gn_rows_sums<T_, V_>, grid, block, 0, s, 1, true, p, q, x, dy, gamma, beta, mean,      \
                      rstd, st, part);                                                                       \
        if (e == cudaSuccess)                                                                                \
            e = launch_ex(gn_rows_dx<T_, V_>, grid, block, 0, s, 1, true, p, q, x, dy, gamma, beta, mean,    \
                          rstd, dx, in);                                                                     \
    } while (0)
    if (q.V == 4) { GN_CALL(T, 4); }
    else if (q.V == 2) { GN_CALL(T, 2); }
    else { GN_CALL(T, 1); }
#undef GN_CALL
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t run_gn_rows_fwd(const GnParams& p, const GnRows& q, int dt, const void* x, const void* gamma,
                            const void* beta, void* y, float* mean, float* rstd, void* ws, cudaStream_t s)
{
    if (dt == DT_F32)
        return rows_fwd_t<float>(p, q, (const float*)x, (const float*)gamma, (const float*)beta, (float*)y, mean, rstd,
                                 ws, s);
    using H = __nv_bfloat16;
    return rows_fwd_t<H>(p, q, (const H*)x, (const H*)gamma, (const H*)beta, (H*)y, mean, rstd, ws, s);
}

cudaError_t run_gn_rows_bwd(const GnParams& p, const GnRows& q, int dt, const void* x, const void* dy,
                            const void* gamma, const void* beta, const float* mean, const float* rstd, void* dx,
                            float* part, void* ws, cudaStream_t s)
{
    if (dt == DT_F32)
        return rows_bwd_t<float>(p, q, (const float*)x, (const float*)dy, (const float*)gamma, (const float*)beta,
                                 mean, rstd, (float*)dx, part, ws, s);
    using H = __nv_bfloat16;
    return rows_bwd_t<H>(p, q, (const H*)x, (const H*)dy, (const H*)gamma, (const H*)beta, mean, rstd, (H*)dx, part,
                         ws, s);
}

}  // namespace igc
