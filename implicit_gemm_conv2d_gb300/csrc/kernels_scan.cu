// kernels_scan.cu -- the gated scan over time, h[t] = h[t-1] + z[t] (x[t] - h[t-1]) with
// z = 1 / (1 + exp(-gate)), and its backward s[t] = dh[t] + (1 - z[t+1]) s[t+1].
//
// A stretch of steps acts on the state that enters it as state -> A * state + H, with A the product
// of its 1 - z and H what it makes of 0; stretches are joined by (A2 A1, A2 H1 + H2).  A thread takes
// L consecutive steps of V channels: it finds its stretch's (A, H), the block joins those of its
// threads along time in shared memory, a cluster those of its blocks through distributed shared
// memory, and the thread walks its steps again from registers with the state it now knows.  So
// each input is read once, whatever the length, and a long sequence is worked on by many blocks.
// A block's rows of time (TY), its channels (LX * V) and its batch rows (BY) follow from the sizes.
//
// z (x - h) + h instead of (1 - z) h + z x, and A - z A: where z is small, a long memory, z's own
// relative error is all that enters, not the rounding of 1 - z.  State, A and H are fp32.
// A stretch with a reset in it has A = -1: what enters it, be it NaN, is left out and not multiplied by 0.
#include <algorithm>
#include <cfloat>

#include "gn_common.cuh"
#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int SCAN_THREADS = 256;

// e = exp(-gate), infinite where the gate is far below 0, and z = 1 / (1 + e), which is 0 there.
template <typename T> __device__ __forceinline__ float scan_gate(float g, float& e)
{
    if constexpr (sizeof(T) == 4) e = expf(-g);
    else e = fast_exp2(g * -kLog2e);
    return fast_rcp(1.f + e);
}

// (A, H) followed by (a, h).
__device__ __forceinline__ void scan_join(float& A, float& H, float a, float h)
{
    H = a < 0.f ? h : fmaf(a, H, h);
    A = a < 0.f || A < 0.f ? -1.f : A * a;
}
__device__ __forceinline__ float scan_enter(float A, float H, float state) { return A < 0.f ? H : fmaf(A, state, H); }

// One side's place in the work.
struct ScanAt {
    int lx, seg, by;       // thread: lane over channels, stretch, batch row
    int LX, TY, NC;        // NC: columns (batch row, channel) of the block
    int C, rank;
    int b0, c0;            // block: first batch row, first channel
    __device__ __forceinline__ ScanAt(const ScanPlan& p, int V)
    {
        LX = 1 << p.lx_log;
        TY = 1 << p.ty_log;
        C = p.cluster;
        lx = int(threadIdx.x) & (LX - 1);
        seg = (int(threadIdx.x) >> p.lx_log) & (TY - 1);
        by = int(threadIdx.x) >> (p.lx_log + p.ty_log);
        NC = (LX * V) << p.by_log;
        rank = int(blockIdx.x) % C;
        const int unit = int(blockIdx.x) / C;
        b0 = (unit / p.tiles) << p.by_log;
        c0 = (unit % p.tiles) * LX * V;
    }
};

__device__ __forceinline__ int scan_length(const ScanPlan& p, const int32_t* lengths, int b)
{
    return lengths ? min(max(lengths[b], 0), p.T) : p.T;
}

// The block's shared memory: (A, H) of each thread's stretch, then of what lies in front of it; the
// state that enters the block's and the next blocks' steps; the blocks' (A, H), twice in turn.
struct ScanShared {
    float *A, *H, *enter, *state, *total;
    __device__ __forceinline__ ScanShared(float* sm, const ScanAt& q)
    {
        const int n = q.TY * q.NC;
        A = sm;
        H = A + n;
        enter = H + n;
        state = enter + q.NC;
        total = state + q.NC;
    }
};

// Joins the stretches of the block and the cluster along time.  On entry A, H hold each thread's stretch; on
// return what lies in front of it within the block, `enter` the state that enters the block, `state` the one
// behind the cluster.  Every thread of the cluster takes part.
__device__ __forceinline__ void scan_block(const ScanAt& q, const ScanShared& s, int round)
{
    __syncthreads();
    for (int c = int(threadIdx.x); c < q.NC; c += int(blockDim.x)) {
        float A = 1.f, H = 0.f;
        for (int k = 0; k < q.TY; ++k) {
            const float a = s.A[k * q.NC + c], h = s.H[k * q.NC + c];
            s.A[k * q.NC + c] = A;
            s.H[k * q.NC + c] = H;
            scan_join(A, H, a, h);
        }
        if (q.C == 1) {
            const float v = s.state[c];
            s.enter[c] = v;
            s.state[c] = scan_enter(A, H, v);
        } else {
            const uint32_t at = tc::smem_u32(s.total + (((round & 1) * q.C + q.rank) * q.NC + c) * 2);
            for (int r = 0; r < q.C; ++r) tc::st_dsmem_f2(tc::dsmem_addr(at, uint32_t(r)), A, H);
        }
    }
    if (q.C > 1) {
        tc::cluster_sync();
        for (int c = int(threadIdx.x); c < q.NC; c += int(blockDim.x)) {
            float v = s.state[c];
            for (int r = 0; r < q.C; ++r) {
                if (r == q.rank) s.enter[c] = v;
                const float2 t = reinterpret_cast<const float2*>(s.total)[((round & 1) * q.C + r) * q.NC + c];
                v = scan_enter(t.x, t.y, v);
            }
            s.state[c] = v;
        }
    }
    __syncthreads();
}

// Bit i is set where step t0 + dir * i, i < L, is one of the row's (below len) and a reset.  The lanes of a
// group of LX, which have the steps in common, read one each.
template <int L>
__device__ __forceinline__ uint32_t scan_flags(const ScanAt& q, const uint8_t* row, int64_t t0, int dir, int len)
{
    uint32_t mask = 0;
    const int group = int(threadIdx.x) & 31 & ~(q.LX - 1);
    for (int i0 = 0; i0 < L; i0 += q.LX) {
        const int64_t t = t0 + dir * (i0 + q.lx);
        const bool set = i0 + q.lx < L && t >= 0 && t < len && row[t] != 0;
        const uint32_t all = __ballot_sync(0xFFFFFFFFu, set) >> group;
        mask |= (q.LX == 32 ? all : all & ((1u << q.LX) - 1u)) << i0;
    }
    return mask;
}

template <typename T, int V, int L, bool RESET>
__global__ void __launch_bounds__(SCAN_THREADS)
scan_fwd_kernel(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const float* h0, const uint8_t* reset,
                const int32_t* lengths, T* h, float* last)
{
    extern __shared__ __align__(16) float sm[];
    const ScanAt q(p, V);
    const ScanShared s(sm, q);
    const int b = q.b0 + q.by, c = q.c0 + q.lx * V;
    const bool row_in = b < p.B, mine = row_in && c < p.D;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int row_len = row_in ? scan_length(p, lengths, b) : 0, len = mine ? row_len : 0;
    for (int k = int(threadIdx.x); k < q.NC; k += int(blockDim.x)) {
        const int kb = q.b0 + k / (q.LX * V), kc = q.c0 + k % (q.LX * V);
        s.state[k] = h0 && kb < p.B && kc < p.D ? h0[int64_t(kb) * p.D + kc] : 0.f;
    }
    if (q.C > 1) tc::cluster_sync();  // every block of the cluster is there, and has read its h0

    const int first = (q.rank * q.TY + q.seg) * L, span = q.C * q.TY * L;
    const int64_t xs = p.x.step, gs = p.gate.step, hs = p.h.step;
    const T* px = x + (mine ? int64_t(b) * p.x.batch + c : 0);
    const T* pg = gate + (mine ? int64_t(b) * p.gate.batch + c : 0);
    T* ph = h + (mine ? int64_t(b) * p.h.batch + c : 0);
    const uint8_t* pr = RESET && row_in ? reset + int64_t(b) * p.T : nullptr;

    Vec<T, V> rx[L], rg[L];
    uint32_t flags = 0;
    auto load = [&](int64_t t0) {
        const int n = t0 >= len ? 0 : int(min(int64_t(L), len - t0));
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i < n) {
                rx[i].load(px + (t0 + i) * xs);
                rg[i].load(pg + (t0 + i) * gs);
            }
        }
        if constexpr (RESET) flags = scan_flags<L>(q, pr, t0, 1, row_len);
    };
    load(first);
    int round = 0;
    for (int64_t base = 0; base < p.T; base += span, ++round) {
        const int64_t t0 = base + first;
        const int n = t0 >= len ? 0 : int(min(int64_t(L), len - t0));
        float z[L][V], xv[L][V];
        const uint32_t cut = flags;
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float e;
                z[i][v] = 0.f;
                xv[i][v] = 0.f;
                if (i < n) {
                    z[i][v] = scan_gate<T>(rg[i].get(v), e);
                    xv[i][v] = rx[i].get(v);
                }
            }
        if (base + span < p.T) load(t0 + span);
        float A[V], H[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            H[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (RESET && (cut >> i & 1u)) H[v] = 0.f;
                if (i < n) H[v] = fmaf(z[i][v], xv[i][v] - H[v], H[v]);
                if (i < n) A[v] = fmaf(-z[i][v], A[v], A[v]);
            }
        const int col = (q.by * q.LX + q.lx) * V, slot = q.seg * q.NC + col;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s.A[slot + v] = RESET && cut != 0 ? -1.f : A[v];
            s.H[slot + v] = H[v];
        }
        scan_block(q, s, round);
        float st[V];
#pragma unroll
        for (int v = 0; v < V; ++v) st[v] = scan_enter(s.A[slot + v], s.H[slot + v], s.enter[col + v]);
        if (mine) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                float out[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (RESET && (cut >> i & 1u)) st[v] = 0.f;
                    if (i < n) st[v] = fmaf(z[i][v], xv[i][v] - st[v], st[v]);
                    out[v] = i < n ? st[v] : 0.f;
                }
                if (t0 + i < p.T) {
                    Vec<T, V> o;
                    o.set(out);
                    o.store(ph + (t0 + i) * hs);
                }
            }
        }
    }
    if (last && q.rank == 0) {
        __syncthreads();
        for (int k = int(threadIdx.x); k < q.NC; k += int(blockDim.x)) {
            const int kb = q.b0 + k / (q.LX * V), kc = q.c0 + k % (q.LX * V);
            if (kb < p.B && kc < p.D) last[int64_t(kb) * p.D + kc] = s.state[k];
        }
    }
}

// Time runs backwards: a thread's stretch is the steps t = T - 1 - u, u = u0 .. u0 + L - 1, and the state is what
// flows from step t into t - 1, (1 - z[t]) s[t].
template <typename T, int V, int L, bool RESET>
__global__ void __launch_bounds__(SCAN_THREADS)
scan_bwd_kernel(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const T* h, const T* dh, const float* h0,
                const float* dlast, const uint8_t* reset, const int32_t* lengths, T* dx, T* dgate, float* dh0)
{
    extern __shared__ __align__(16) float sm[];
    const ScanAt q(p, V);
    const ScanShared s(sm, q);
    const int b = q.b0 + q.by, c = q.c0 + q.lx * V;
    const bool row_in = b < p.B, mine = row_in && c < p.D;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int row_len = row_in ? scan_length(p, lengths, b) : 0, len = mine ? row_len : 0;
    for (int k = int(threadIdx.x); k < q.NC; k += int(blockDim.x)) {
        const int kb = q.b0 + k / (q.LX * V), kc = q.c0 + k % (q.LX * V);
        s.state[k] = dlast && kb < p.B && kc < p.D ? dlast[int64_t(kb) * p.D + kc] : 0.f;
    }
    if (q.C > 1) tc::cluster_sync();

    const int first = (q.rank * q.TY + q.seg) * L, span = q.C * q.TY * L;
    const int64_t row = mine ? b : 0, ch = mine ? c : 0;
    const T* px = x + row * p.x.batch + ch;
    const T* pg = gate + row * p.gate.batch + ch;
    const T* ph = h + row * p.h.batch + ch;
    const T* pd = dh + row * p.dh.batch + ch;
    T* ox = dx + row * p.dx.batch + ch;
    T* og = dgate + row * p.dgate.batch + ch;
    const uint8_t* pr = RESET && row_in ? reset + int64_t(b) * p.T : nullptr;

    Vec<T, V> rx[L], rg[L], rh[L], rd[L];
    uint32_t flags = 0;
    auto load = [&](int64_t u0) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t t = p.T - 1 - u0 - i;
            if (t >= 0 && t < len) {
                rx[i].load(px + t * p.x.step);
                rg[i].load(pg + t * p.gate.step);
                rd[i].load(pd + t * p.dh.step);
                if (t > 0) rh[i].load(ph + (t - 1) * p.h.step);
            }
        }
        if constexpr (RESET) flags = scan_flags<L>(q, pr, p.T - 1 - u0, -1, row_len);
    };
    load(first);
    int round = 0;
    for (int64_t base = 0; base < p.T; base += span, ++round) {
        const int64_t u0 = base + first;
        float z[L][V], zz[L][V], d[L][V], xh[L][V];
        const uint32_t cut = flags;
        uint32_t has = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int64_t t = p.T - 1 - u0 - i;
            if (t >= 0 && t < len) has |= 1u << i;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                z[i][v] = zz[i][v] = d[i][v] = xh[i][v] = 0.f;
                if (has >> i & 1u) {
                    float e;
                    z[i][v] = scan_gate<T>(rg[i].get(v), e);
                    zz[i][v] = fminf(e, FLT_MAX) * z[i][v] * z[i][v];  // z (1 - z); 0 where e is infinite
                    d[i][v] = rd[i].get(v);
                    float before = t > 0 ? rh[i].get(v) : (h0 ? h0[row * p.D + ch + v] : 0.f);
                    if (RESET && (cut >> i & 1u)) before = 0.f;
                    xh[i][v] = rx[i].get(v) - before;
                }
            }
        }
        if (base + span < p.T) load(u0 + span);
        float A[V], H[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.f;
            H[v] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (has >> i & 1u) {
                    const float f = d[i][v] + H[v];
                    H[v] = RESET && (cut >> i & 1u) ? 0.f : fmaf(-z[i][v], f, f);
                    A[v] = fmaf(-z[i][v], A[v], A[v]);
                }
            }
        const int col = (q.by * q.LX + q.lx) * V, slot = q.seg * q.NC + col;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s.A[slot + v] = RESET && cut != 0 ? -1.f : A[v];
            s.H[slot + v] = H[v];
        }
        scan_block(q, s, round);
        float st[V];
#pragma unroll
        for (int v = 0; v < V; ++v) st[v] = scan_enter(s.A[slot + v], s.H[slot + v], s.enter[col + v]);
        if (mine) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                float a[V], g[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    a[v] = g[v] = 0.f;
                    if (has >> i & 1u) {
                        const float f = d[i][v] + st[v];
                        a[v] = z[i][v] * f;
                        g[v] = f * xh[i][v] * zz[i][v];
                        st[v] = RESET && (cut >> i & 1u) ? 0.f : fmaf(-z[i][v], f, f);
                    }
                }
                const int64_t t = p.T - 1 - u0 - i;
                if (t >= 0) {
                    Vec<T, V> o;
                    o.set(a);
                    o.store(ox + t * p.dx.step);
                    o.set(g);
                    o.store(og + t * p.dgate.step);
                }
            }
        }
    }
    if (dh0 && q.rank == 0) {
        __syncthreads();
        for (int k = int(threadIdx.x); k < q.NC; k += int(blockDim.x)) {
            const int kb = q.b0 + k / (q.LX * V), kc = q.c0 + k % (q.LX * V);
            if (kb < p.B && kc < p.D) dh0[int64_t(kb) * p.D + kc] = s.state[k];
        }
    }
}

int log2_up(int64_t n)
{
    int k = 0;
    while ((int64_t(1) << k) < n) ++k;
    return k;
}

}  // namespace

// V channels a thread: two bf16 where every row begins at a multiple of 4 bytes.
ScanPlan scan_plan(const conv_scan_desc_t& e, const DevInfo& d, bool bwd, bool pairs)
{
    ScanPlan p = {};
    p.B = e.B; p.T = e.T; p.D = e.D;
    p.x = e.x; p.gate = e.gate; p.h = e.h; p.dh = e.dh; p.dx = e.dx; p.dgate = e.dgate;
    p.V = e.dtype == CONV_BF16 && pairs && e.D % 2 == 0 ? 2 : 1;
    p.L = e.T <= 8 ? 4 : bwd ? 8 : 16;
    const int64_t cols = (int64_t(e.D) + p.V - 1) / p.V, segs = std::max<int64_t>(1, (int64_t(e.T) + p.L - 1) / p.L);
    const int all = log2_up(SCAN_THREADS);
    int log_c = 0;
    int64_t blocks = 0;
    p.lx_log = std::min(5, log2_up(cols));
    for (;;) {
        p.ty_log = std::min(all - p.lx_log, log2_up(segs));
        p.by_log = std::max(std::min(all - p.lx_log - p.ty_log, log2_up(std::max(1, e.B))), 5 - p.lx_log - p.ty_log);
        p.tiles = int((cols + (1 << p.lx_log) - 1) >> p.lx_log);
        blocks = int64_t(p.tiles) * ((int64_t(e.B) + (1 << p.by_log) - 1) >> p.by_log);
        log_c = 0;
        while (log_c < 3 && (blocks << log_c) < 2 * d.sms && (int64_t(1) << (log_c + p.ty_log)) < segs) ++log_c;
        if ((blocks << log_c) >= d.sms || p.lx_log <= 3 || (int64_t(1) << (log_c + p.ty_log)) >= segs) break;
        --p.lx_log;
    }
    p.cluster = 1 << log_c;
    p.blocks = blocks << log_c;
    p.threads = 1 << (p.lx_log + p.ty_log + p.by_log);
    return p;
}

namespace {

int scan_smem(const ScanPlan& p)
{
    const int nc = (p.V << p.lx_log) << p.by_log, n = nc << p.ty_log;
    return 4 * (2 * n + 2 * nc + (p.cluster > 1 ? 4 * p.cluster * nc : 0));
}

// Calls f(T(), V, L, RESET), the last three as types, for the plan; LONG: the larger L.
template <int LONG, class F> cudaError_t scan_with(const ScanPlan& p, int dt, bool reset, F&& f)
{
    auto on_reset = [&](auto t, auto v, auto l) {
        return reset ? f(t, v, l, std::true_type()) : f(t, v, l, std::false_type());
    };
    auto on_steps = [&](auto t, auto v) {
        return p.L == 4 ? on_reset(t, v, std::integral_constant<int, 4>())
                        : on_reset(t, v, std::integral_constant<int, LONG>());
    };
    if (dt == DT_F32) return on_steps(float(), std::integral_constant<int, 1>());
    if (p.V == 2) return on_steps(__nv_bfloat16(), std::integral_constant<int, 2>());
    return on_steps(__nv_bfloat16(), std::integral_constant<int, 1>());
}

bool rows_even(const conv_rows_t& r) { return r.batch % 2 == 0 && r.step % 2 == 0; }
bool at_pair(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

cudaError_t run_scan_fwd(const conv_scan_desc_t& e, const DevInfo& d, const void* x, const void* gate, const float* h0,
                         const uint8_t* reset, const int32_t* lengths, void* h, float* last, cudaStream_t s)
{
    const bool pairs = rows_even(e.x) && rows_even(e.gate) && rows_even(e.h) && at_pair(x) && at_pair(gate) && at_pair(h);
    const ScanPlan p = scan_plan(e, d, false, pairs);
    return scan_with<16>(p, e.dtype, reset != nullptr, [&](auto t, auto v, auto l, auto r) {
        using T = decltype(t);
        return launch_ex(scan_fwd_kernel<T, decltype(v)::value, decltype(l)::value, decltype(r)::value>, dim3(unsigned(p.blocks)), dim3(p.threads), scan_smem(p), s,
                         p.cluster, true, p, static_cast<const T*>(x), static_cast<const T*>(gate), h0, reset, lengths,
                         static_cast<T*>(h), last);
    });
}

cudaError_t run_scan_bwd(const conv_scan_desc_t& e, const DevInfo& d, const void* x, const void* gate, const void* h,
                         const void* dh, const float* h0, const float* dlast, const uint8_t* reset,
                         const int32_t* lengths, void* dx, void* dgate, float* dh0, cudaStream_t s)
{
    const bool pairs = rows_even(e.x) && rows_even(e.gate) && rows_even(e.h) && rows_even(e.dh) && rows_even(e.dx) &&
                       rows_even(e.dgate) && at_pair(x) && at_pair(gate) && at_pair(h) && at_pair(dh) && at_pair(dx) &&
                       at_pair(dgate);
    const ScanPlan p = scan_plan(e, d, true, pairs);
    return scan_with<8>(p, e.dtype, reset != nullptr, [&](auto t, auto v, auto l, auto r) {
        using T = decltype(t);
        return launch_ex(scan_bwd_kernel<T, decltype(v)::value, decltype(l)::value, decltype(r)::value>, dim3(unsigned(p.blocks)), dim3(p.threads), scan_smem(p), s,
                         p.cluster, true, p, static_cast<const T*>(x), static_cast<const T*>(gate),
                         static_cast<const T*>(h), static_cast<const T*>(dh), h0, dlast, reset, lengths,
                         static_cast<T*>(dx), static_cast<T*>(dgate), dh0);
    });
}

}  // namespace igc
