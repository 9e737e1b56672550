// kernels_scan.cu -- the gated scan over time, h[t] = h[t-1] + z[t] (x[t] - h[t-1]) with
// z = 1 / (1 + exp(-gate)), and its backward s[t] = dh[t] + (1 - z[t+1]) s[t+1].
//
// Two ways through time.  Where rows times channels fill the GPU, or there are few steps, a thread walks
// all steps of two channels, reading a few steps ahead ("walk").  Else time is cut ("parts"):
// a stretch of steps acts on the state that enters it as state -> A * state + H, with A the product
// of its 1 - z and H what it makes of 0; stretches are joined by (A2 A1, A2 H1 + H2).  A lane takes
// L consecutive steps of two channels, a warp 8 such stretches of 8 channels: the warp joins them by
// shuffles, the warps of a cluster's blocks, which share a sequence's round, through distributed shared
// memory (stores that count on a barrier), and each lane walks its steps again, from registers, with the state it now
// knows.  So each
// input is read once, whatever the length, and a long sequence is worked on by many blocks.
// Where even a cluster of 8 blocks a sequence leaves most of the GPU idle, time is cut into pieces first: one kernel
// finds each piece's (A, H), the other joins those in front of its own and walks it.
// Rounds travel through shared memory in both directions, whole rows at a time: inputs by
// asynchronous copies (16 bytes where the rows allow it) that run a round or two ahead, results in
// the places of the inputs.
//
// State, A and H are fp32, and so is 1 - z, taken from z: where z is small, a long memory, z's error is
// small beside the rounding of 1 - z, which is that of one more operation a step.  Where z is near 1, what is left of
// the state is off by up to 2^-23 of the state, as in h + z (x - h) itself.
// What enters a stretch with a reset in it, be it NaN, is left out and not multiplied by 0: a warp votes on its
// stretches' resets; where a stretch travels further, A = -1 says it.
//
// Floor: 3 values an element are read and written (backward 6).  Measured, with the share of that floor at the
// measured copy's bandwidth: 1024 x 64 x 128 fp32 forward 18.2 us (82 %, walk), 2 x 32768 x 1024 bf16 forward 79.5
// (75 %), 8 x 4096 x 1024 bf16 backward 76.1 (78 %), with resets 88.5 (67 %), 5 x 1999 x 777 fp32 padded backward 55 (41 %).
// Bound by instructions and the latency between a round's phases at two or three blocks an SM (0.44 to 0.57 issued a
// slot); a step of few rows by its launch.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "gn_common.cuh"
#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int SCAN_THREADS = 256, SCAN_WARPS = 8;
constexpr int SCAN_SEGS = 8;                 // stretches of a warp
constexpr int SCAN_LENS = 128;               // bytes for the batch rows' lengths
constexpr int WALK_THREADS = 128;

__device__ unsigned g_scan_status = 0;       // CONV_STATUS_SCAN: a bounded wait ran out

__device__ __forceinline__ float2 one_minus(float2 a) { return fma2(a, both(-1.f), both(1.f)); }

// e = exp(-gate), infinite where the gate is far below 0, and z = 1 / (1 + e), which is 0 there.  fp32 takes
// expf; for bf16 a rounded argument of 2^x, up to |gate| 2^-24 off, is far below the rounding of h.
template <typename T> __device__ __forceinline__ float2 scan_gate(float2 g, float2& e)
{
    if constexpr (sizeof(T) == 4) {
        e = make_float2(expf(-g.x), expf(-g.y));
    } else {
        e = mul2(g, both(-kLog2e));
        e = make_float2(fast_exp2(e.x), fast_exp2(e.y));
    }
    const float2 w = add2(e, both(1.f));
    return make_float2(fast_rcp(w.x), fast_rcp(w.y));
}
// z (1 - z) = e z z, also 0 where e is infinite
__device__ __forceinline__ float2 scan_slope(float2 e, float2 z)
{
    return mul2(mul2(make_float2(fminf(e.x, FLT_MAX), fminf(e.y, FLT_MAX)), z), z);
}

// What a stretch (A, H) makes of the state that enters it.
template <bool RESET> __device__ __forceinline__ float2 scan_enter(float2 A, float2 H, float2 state)
{
    const float2 r = fma2(A, state, H);
    if constexpr (RESET) return make_float2(A.x < 0.f ? H.x : r.x, A.y < 0.f ? H.y : r.y);
    return r;
}
// (A, H) behind (a, h).
template <bool RESET> __device__ __forceinline__ void scan_join(float2& A, float2& H, float2 a, float2 h)
{
    H = scan_enter<RESET>(A, H, h);
    const float2 r = mul2(A, a);
    A = RESET ? make_float2(A.x < 0.f || a.x < 0.f ? -1.f : r.x, A.y < 0.f || a.y < 0.f ? -1.f : r.y) : r;
}
__device__ __forceinline__ float2 shfl_up(float2 v, int by)
{
    return make_float2(__shfl_up_sync(0xFFFFFFFFu, v.x, by), __shfl_up_sync(0xFFFFFFFFu, v.y, by));
}
__device__ __forceinline__ float2 shfl(float2 v, int lane)
{
    return make_float2(__shfl_sync(0xFFFFFFFFu, v.x, lane), __shfl_sync(0xFFFFFFFFu, v.y, lane));
}

__device__ __forceinline__ int scan_length(const ScanPlan& p, const int32_t* lengths, int b)
{
    return lengths ? min(max(lengths[b], 0), p.T) : p.T;
}

// ---- walk: a thread takes all steps of V channels -------------------------------------------
template <typename T, int V> __device__ __forceinline__ float2 widen(const Vec<T, V>& r)
{
    return make_float2(r.get(0), V == 2 ? r.get(V - 1) : 0.f);
}
template <typename T, int V> __device__ __forceinline__ void put(T* o, float2 v)
{
    Vec<T, V> r;
    if constexpr (V == 2) {
        const float f[2] = {v.x, v.y};
        r.set(f);
    } else {
        const float f[1] = {v.x};
        r.set(f);
    }
    r.store(o);
}
template <int V> __device__ __forceinline__ float2 walk_state(const float* from, int64_t at)
{
    return from ? make_float2(from[at], V == 2 ? from[at + V - 1] : 0.f) : both(0.f);
}
template <int V> __device__ __forceinline__ void walk_store(float* to, int64_t at, float2 v)
{
    if (!to) return;
    to[at] = v.x;
    if constexpr (V == 2) to[at + 1] = v.y;
}

template <typename T, int V, int L, bool RESET>
__global__ void __launch_bounds__(WALK_THREADS)
scan_walk_fwd(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const float* h0, const uint8_t* reset,
              const int32_t* lengths, T* h, float* last)
{
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int64_t unit = int64_t(blockIdx.x) * WALK_THREADS + threadIdx.x, b = unit / p.cols, c = unit % p.cols * V;
    if (b >= p.B) return;
    const int len = scan_length(p, lengths, int(b));
    const T *px = x + b * p.x.batch + c, *pg = gate + b * p.gate.batch + c;
    T* ph = h + b * p.h.batch + c;
    const uint8_t* pr = RESET ? reset + b * p.T : nullptr;
    float2 st = walk_state<V>(h0, b * p.D + c);
    Vec<T, V> rx[L], rg[L];
    uint8_t rr[L];
    auto load = [&](int n) {
        if (n >= L) {
#pragma unroll
            for (int i = 0; i < L; ++i, px += p.x.step, pg += p.gate.step) {
                rx[i].load(px);
                rg[i].load(pg);
                if (RESET) rr[i] = pr[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (i < n) {
                    rx[i].load(px + i * p.x.step);
                    rg[i].load(pg + i * p.gate.step);
                    if (RESET) rr[i] = pr[i];
                }
        }
        if (RESET) pr += L;
    };
    load(len);
    for (int t = 0; t < len; t += L) {
        float2 keep[L], in[L];
        uint32_t cut = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float2 e;
            const float2 z = scan_gate<T>(widen(rg[i]), e);
            keep[i] = one_minus(z);
            in[i] = mul2(z, widen(rx[i]));
            if (RESET && rr[i] != 0) cut |= 1u << i;
        }
        load(len - t - L);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (t + i < len) {
                if (RESET && (cut >> i & 1u)) st = both(0.f);
                st = fma2(keep[i], st, in[i]);
                put<T, V>(ph, st);
                ph += p.h.step;
            }
        }
    }
    for (int t = len; t < p.T; ++t, ph += p.h.step) put<T, V>(ph, both(0.f));
    walk_store<V>(last, b * p.D + c, st);
}

template <typename T, int V, int L, bool RESET>
__global__ void __launch_bounds__(WALK_THREADS)
scan_walk_bwd(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const T* h, const T* dh, const float* h0,
              const float* dlast, const uint8_t* reset, const int32_t* lengths, T* dx, T* dgate, float* dh0)
{
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int64_t unit = int64_t(blockIdx.x) * WALK_THREADS + threadIdx.x, b = unit / p.cols, c = unit % p.cols * V;
    if (b >= p.B) return;
    const int len = scan_length(p, lengths, int(b));
    const int64_t end = len - 1;  // the pointers are at the next step to read, and the next one to write
    const T *px = x + b * p.x.batch + c + end * p.x.step, *pg = gate + b * p.gate.batch + c + end * p.gate.step;
    const T *ph = h + b * p.h.batch + c + (end - 1) * p.h.step, *pd = dh + b * p.dh.batch + c + end * p.dh.step;
    T *ox = dx + b * p.dx.batch + c + end * p.dx.step, *og = dgate + b * p.dgate.batch + c + end * p.dgate.step;
    for (int t = len; t < p.T; ++t) {
        put<T, V>(ox + (t - end) * p.dx.step, both(0.f));
        put<T, V>(og + (t - end) * p.dgate.step, both(0.f));
    }
    const uint8_t* pr = RESET ? reset + b * p.T + end : nullptr;
    float2 st = walk_state<V>(dlast, b * p.D + c);
    Vec<T, V> rx[L], rg[L], rh[L], rd[L];
    uint8_t rr[L];
    auto load = [&](int n) {  // n steps are left, the last of them step 0, with nothing kept before it
        if (n > L) {
#pragma unroll
            for (int i = 0; i < L; ++i, px -= p.x.step, pg -= p.gate.step, ph -= p.h.step, pd -= p.dh.step) {
                rx[i].load(px);
                rg[i].load(pg);
                rd[i].load(pd);
                rh[i].load(ph);
                if (RESET) rr[i] = *(pr - i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (i < n) {
                    rx[i].load(px - i * p.x.step);
                    rg[i].load(pg - i * p.gate.step);
                    rd[i].load(pd - i * p.dh.step);
                    if (i < n - 1) rh[i].load(ph - i * p.h.step);
                    if (RESET) rr[i] = *(pr - i);
                }
        }
        if (RESET) pr -= L;
    };
    load(len);
    for (int n = len; n > 0; n -= L) {
        float2 z[L], d[L], w[L];
        uint32_t cut = 0;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float2 e;
            z[i] = scan_gate<T>(widen(rg[i]), e);
            d[i] = widen(rd[i]);
            float2 before = widen(rh[i]);
            if (i == n - 1) before = walk_state<V>(h0, b * p.D + c);
            if (RESET && rr[i] != 0) {
                cut |= 1u << i;
                before = both(0.f);
            }
            w[i] = mul2(scan_slope(e, z[i]), fma2(before, both(-1.f), widen(rx[i])));
        }
        load(n - L);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i < n) {
                const float2 f = add2(d[i], st);
                put<T, V>(ox, mul2(z[i], f));
                put<T, V>(og, mul2(w[i], f));
                ox -= p.dx.step;
                og -= p.dgate.step;
                st = mul2(one_minus(z[i]), f);
                if (RESET && (cut >> i & 1u)) st = both(0.f);
            }
        }
    }
    walk_store<V>(dh0, b * p.D + c, st);
}

// The same with the steps to come in shared memory, for fewer threads: their asynchronous copies go to their own
// places, RING groups of RING_STEPS steps ahead, and need no barrier.  [group][step][array][thread] elements of V values.
constexpr int RING_STEPS = 8;
template <int BYTES> __device__ __forceinline__ void ring_copy(uint32_t to, const void* from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
template <typename T, int V> __device__ __forceinline__ float2 ring_read(uint32_t at)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t u = tc::lds32(at);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    } else if constexpr (V == 2) {
        const uint2 u = tc::lds64(at);
        return make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    } else {
        return make_float2(__uint_as_float(tc::lds32(at)), 0.f);
    }
}

template <typename T, int V, int RING, bool RESET>
__global__ void __launch_bounds__(WALK_THREADS)
scan_ring_fwd(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const float* h0, const uint8_t* reset,
              const int32_t* lengths, T* h, float* last)
{
    extern __shared__ __align__(128) uint8_t sm[];
    constexpr int SIZE = V * int(sizeof(T)), LINE = WALK_THREADS * SIZE, GROUP = RING_STEPS * 2 * LINE;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int64_t unit = int64_t(blockIdx.x) * WALK_THREADS + threadIdx.x, b = unit / p.cols, c = unit % p.cols * V;
    if (b >= p.B) return;
    const int len = scan_length(p, lengths, int(b));
    const T *px = x + b * p.x.batch + c, *pg = gate + b * p.gate.batch + c;
    T* ph = h + b * p.h.batch + c;
    const uint8_t* pr = RESET ? reset + b * p.T : nullptr;
    float2 st = walk_state<V>(h0, b * p.D + c);
    const uint32_t ring = tc::smem_u32(sm) + threadIdx.x * SIZE;
    int ahead = 0;
    auto fetch = [&](uint32_t to) {
#pragma unroll
        for (int i = 0; i < RING_STEPS; ++i, px += p.x.step, pg += p.gate.step)
            if (ahead + i < len) {
                ring_copy<SIZE>(to + uint32_t(i * 2 * LINE), px);
                ring_copy<SIZE>(to + uint32_t((i * 2 + 1) * LINE), pg);
            }
        ahead += RING_STEPS;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int k = 0; k < RING; ++k) fetch(ring + uint32_t(k * GROUP));
    uint32_t at = ring;
    uint8_t flags[RING_STEPS];  // of the steps ahead, one group's
    auto look = [&](int t) {
        if (RESET)
#pragma unroll
            for (int i = 0; i < RING_STEPS; ++i) {
                flags[i] = 0;
                if (t + i < len) flags[i] = pr[t + i];
            }
    };
    look(0);
    for (int t = 0; t < len; t += RING_STEPS) {
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        uint32_t cut = 0;
        if (RESET)
#pragma unroll
            for (int i = 0; i < RING_STEPS; ++i) cut |= flags[i] != 0 ? 1u << i : 0u;
        float2 keep[RING_STEPS], in[RING_STEPS];
#pragma unroll
        for (int i = 0; i < RING_STEPS; ++i) {
            float2 e;
            const float2 z = scan_gate<T>(ring_read<T, V>(at + uint32_t((i * 2 + 1) * LINE)), e);
            keep[i] = one_minus(z);
            in[i] = mul2(z, ring_read<T, V>(at + uint32_t(i * 2 * LINE)));
        }
        fetch(at);
        look(t + RING_STEPS);
        at = at + GROUP == ring + RING * GROUP ? ring : at + GROUP;
#pragma unroll
        for (int i = 0; i < RING_STEPS; ++i) {
            if (t + i < len) {
                if (RESET && (cut >> i & 1u)) st = both(0.f);
                st = fma2(keep[i], st, in[i]);
                put<T, V>(ph, st);
                ph += p.h.step;
            }
        }
    }
    for (int t = len; t < p.T; ++t, ph += p.h.step) put<T, V>(ph, both(0.f));
    walk_store<V>(last, b * p.D + c, st);
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int V, int RING, bool RESET>
__global__ void __launch_bounds__(WALK_THREADS)
scan_ring_bwd(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const T* h, const T* dh, const float* h0,
              const float* dlast, const uint8_t* reset, const int32_t* lengths, T* dx, T* dgate, float* dh0)
{
    extern __shared__ __align__(128) uint8_t sm[];
    constexpr int SIZE = V * int(sizeof(T)), LINE = WALK_THREADS * SIZE, GROUP = RING_STEPS * 4 * LINE;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int64_t unit = int64_t(blockIdx.x) * WALK_THREADS + threadIdx.x, b = unit / p.cols, c = unit % p.cols * V;
    if (b >= p.B) return;
    const int len = scan_length(p, lengths, int(b));
    const int64_t end = len - 1;  // the pointers are at the next step to read, and the next one to write
    const T *px = x + b * p.x.batch + c + end * p.x.step, *pg = gate + b * p.gate.batch + c + end * p.gate.step;
    const T *ph = h + b * p.h.batch + c + (end - 1) * p.h.step, *pd = dh + b * p.dh.batch + c + end * p.dh.step;
    T *ox = dx + b * p.dx.batch + c + end * p.dx.step, *og = dgate + b * p.dgate.batch + c + end * p.dgate.step;
    for (int t = len; t < p.T; ++t) {
        put<T, V>(ox + (t - end) * p.dx.step, both(0.f));
        put<T, V>(og + (t - end) * p.dgate.step, both(0.f));
    }
    const uint8_t* pr = RESET ? reset + b * p.T : nullptr;
    float2 st = walk_state<V>(dlast, b * p.D + c);
    const uint32_t ring = tc::smem_u32(sm) + threadIdx.x * SIZE;
    int ahead = len;  // steps that are not on their way yet
    auto fetch = [&](uint32_t to) {
#pragma unroll
        for (int i = 0; i < RING_STEPS; ++i, px -= p.x.step, pg -= p.gate.step, ph -= p.h.step, pd -= p.dh.step)
            if (i < ahead) {
                const uint32_t line = to + uint32_t(i * 4 * LINE);
                ring_copy<SIZE>(line, px);
                ring_copy<SIZE>(line + LINE, pg);
                ring_copy<SIZE>(line + 2 * LINE, pd);
                if (i < ahead - 1) ring_copy<SIZE>(line + 3 * LINE, ph);
            }
        ahead -= RING_STEPS;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int k = 0; k < RING; ++k) fetch(ring + uint32_t(k * GROUP));
    uint32_t at = ring;
    uint8_t flags[RING_STEPS];
    auto look = [&](int n) {
        if (RESET)
#pragma unroll
            for (int i = 0; i < RING_STEPS; ++i) {
                flags[i] = 0;
                if (i < n) flags[i] = pr[n - 1 - i];
            }
    };
    look(len);
    for (int n = len; n > 0; n -= RING_STEPS) {
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        uint32_t cut = 0;
        if (RESET)
#pragma unroll
            for (int i = 0; i < RING_STEPS; ++i) cut |= flags[i] != 0 ? 1u << i : 0u;
        float2 z[RING_STEPS], d[RING_STEPS], w[RING_STEPS];
#pragma unroll
        for (int i = 0; i < RING_STEPS; ++i) {
            const uint32_t line = at + uint32_t(i * 4 * LINE);
            float2 e;
            z[i] = scan_gate<T>(ring_read<T, V>(line + LINE), e);
            d[i] = ring_read<T, V>(line + 2 * LINE);
            float2 before = ring_read<T, V>(line + 3 * LINE);
            if (i == n - 1) before = walk_state<V>(h0, b * p.D + c);
            if (RESET && (cut >> i & 1u)) before = both(0.f);
            w[i] = mul2(scan_slope(e, z[i]), fma2(before, both(-1.f), ring_read<T, V>(line)));
        }
        fetch(at);
        look(n - RING_STEPS);
        at = at + GROUP == ring + RING * GROUP ? ring : at + GROUP;
#pragma unroll
        for (int i = 0; i < RING_STEPS; ++i) {
            if (i < n) {
                const float2 f = add2(d[i], st);
                put<T, V>(ox, mul2(z[i], f));
                put<T, V>(og, mul2(w[i], f));
                ox -= p.dx.step;
                og -= p.dgate.step;
                st = mul2(one_minus(z[i]), f);
                if (RESET && (cut >> i & 1u)) st = both(0.f);
            }
        }
    }
    walk_store<V>(dh0, b * p.D + c, st);
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---- parts: warps of 8 stretches of 8 channels ------------------------------------------------
// A block has 8 warps: WX of them side by side over the channels, BY batch rows.  A round of a block is
// RT = 8 L steps, of a cluster C of those, one behind the other.
//
// Shared memory of a stage: [array][step][warp][8 channels], where the 16-byte pieces of a step's row
// are permuted by the step's stretch, so that the 8 stretches that a warp reads at once lie in
// different banks.
template <typename T, int L> struct ScanTile {
    static constexpr int ES = int(sizeof(T)), ROW = 64 * ES, RT = SCAN_SEGS * L, ARRAY = RT * ROW;
    // Byte `at` of the row of step u.
    static __device__ __forceinline__ uint32_t place(int u, int at)
    {
        const int seg = u / L;
        return uint32_t(u * ROW + (at ^ (seg * (ES * 8) & (ROW - 16))));
    }
};

struct ScanAt {
    int warp, pair, seg;   // a lane's pair of channels (of the warp's 8) and stretch
    int C, rank;
    int b0, c0;            // block: first batch row, first channel
    int b, c;              // lane: batch row and first channel
    int piece, begin, end; // of time, in steps from the side that the scan begins at
    __device__ __forceinline__ ScanAt(const ScanPlan& p)
    {
        warp = int(threadIdx.x) >> 5;
        pair = int(threadIdx.x) & 3;
        seg = (int(threadIdx.x) & 31) >> 2;
        C = p.cluster;
        rank = int(blockIdx.x) % C;
        const int WX = 1 << p.wx_log, all = int(blockIdx.x) / C;
        piece = all % p.pieces;
        const int unit = all / p.pieces;
        begin = piece * p.piece;
        end = min(p.T - begin, p.piece) + begin;
        b0 = (unit / p.tiles) << p.by_log;
        c0 = (unit % p.tiles) * WX * 8;
        b = b0 + (warp >> p.wx_log);
        c = c0 + (warp & (WX - 1)) * 8 + pair * 2;
    }
};

// One array on its way between memory and the stages.  A thread moves CB bytes of every ROWS-th step of a round,
// always of the same channels; DIR = -1: the rounds and their steps run down in time.
template <typename T, int L, int CB, int DIR> struct ScanCopy {
    using Tile = ScanTile<T, L>;
    static constexpr int ES = Tile::ES, CPR = Tile::ROW / CB, ROWS = SCAN_THREADS / CPR, N = Tile::RT / ROWS;
    static constexpr int UNROLL = std::min(N, CB == 2 ? 8 : 16);
    struct Cursor {
        T* at;               // of the thread's first step of the round
        int64_t hop, round;  // from one of its steps, and of its rounds, to the next
    };
    int byte, u0;      // in a step's row; first step
    int by, column;    // batch row and channel in the block
    int len;           // of the batch row, 0 where the thread's channels are not there
    bool out;          // they are: results are written

    __device__ __forceinline__ ScanCopy(const ScanPlan& p, const ScanAt& q, const int* lens)
    {
        byte = int(threadIdx.x) % CPR * CB;
        u0 = int(threadIdx.x) / CPR;
        const int el = byte / ES, w = el >> 3;
        column = ((w & ((1 << p.wx_log) - 1)) << 3) + (el & 7);
        by = w >> p.wx_log;
        const bool in = q.c0 + column < p.D;
        len = in ? lens[by] : 0;
        out = in && q.b0 + by < p.B;
    }
    // first: step 0 of the block's first round.
    __device__ __forceinline__ Cursor cursor(const ScanAt& q, const void* array, const conv_rows_t& r, int64_t first,
                                             int64_t span) const
    {
        T* a = static_cast<T*>(const_cast<void*>(array));
        return {a + (q.b0 + by) * r.batch + q.c0 + column + (first + DIR * u0) * r.step, DIR * ROWS * r.step,
                DIR * span * r.step};
    }
    // The round that begins at step first: the steps that the row has, and `shift` steps earlier too.  (What is not
    // copied is not used.)
    __device__ __forceinline__ void fill(Cursor& c, uint32_t to, int first, int shift) const
    {
        const T* src = c.at;
        const int last = first + DIR * (Tile::RT - 1), low = DIR > 0 ? first : last, high = DIR > 0 ? last : first;
        if (low >= shift && high < len) {
#pragma unroll UNROLL
            for (int k = 0; k < N; ++k, src += c.hop) copy(to + Tile::place(u0 + k * ROWS, byte), src);
        } else if (low < len) {
            const unsigned some = unsigned(len - shift);  // len > low >= -RT: steps shift .. len - 1, none if len <= shift
#pragma unroll UNROLL
            for (int k = 0; k < N; ++k, src += c.hop)
                if (len > shift && unsigned(first + DIR * (u0 + k * ROWS) - shift) < some)
                    copy(to + Tile::place(u0 + k * ROWS, byte), src);
        }
        c.at += c.round;
    }
    static __device__ __forceinline__ void copy(uint32_t dst, const T* src)
    {
        if constexpr (CB == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        else if constexpr (CB >= 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(CB) : "memory");
        else
            tc::sts16(dst, *reinterpret_cast<const uint16_t*>(src));
    }
    // A round's results back to memory.
    __device__ __forceinline__ void drain(Cursor& c, uint32_t from, int first, int T_) const
    {
        T* dst = c.at;
        const int last = first + DIR * (Tile::RT - 1);
        if (out && first >= 0 && first < T_ && last >= 0 && last < T_) {
#pragma unroll UNROLL
            for (int k = 0; k < N; ++k, dst += c.hop) back(dst, from + Tile::place(u0 + k * ROWS, byte));
        } else if (out) {
#pragma unroll UNROLL
            for (int k = 0; k < N; ++k, dst += c.hop)
                if (unsigned(first + DIR * (u0 + k * ROWS)) < unsigned(T_))
                    back(dst, from + Tile::place(u0 + k * ROWS, byte));
        }
        c.at += c.round;
    }
    static __device__ __forceinline__ void back(T* dst, uint32_t src)
    {
        if constexpr (CB == 16) *reinterpret_cast<int4*>(dst) = tc::lds128(src);
        else if constexpr (CB == 8) *reinterpret_cast<uint2*>(dst) = tc::lds64(src);
        else if constexpr (CB == 4) *reinterpret_cast<uint32_t*>(dst) = tc::lds32(src);
        else *reinterpret_cast<uint16_t*>(dst) = uint16_t(tc::lds16(src));
    }
};

// A lane's two channels of its stretch's steps.
template <typename T, int L> struct ScanLane {
    using Tile = ScanTile<T, L>;
    uint32_t at;
    __device__ __forceinline__ explicit ScanLane(const ScanAt& q)
        : at(Tile::place(q.seg * L, q.warp * 8 * Tile::ES + q.pair * 2 * Tile::ES)) {}
    __device__ __forceinline__ float2 read(uint32_t stage, int array, int i) const
    {
        const uint32_t a = stage + at + uint32_t(array * Tile::ARRAY + i * Tile::ROW);
        if constexpr (sizeof(T) == 4) {
            const uint2 u = tc::lds64(a);
            return make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        } else {
            const uint32_t u = tc::lds32(a);
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
        }
    }
    __device__ __forceinline__ void write(uint32_t stage, int array, int i, float2 v) const
    {
        const uint32_t a = stage + at + uint32_t(array * Tile::ARRAY + i * Tile::ROW);
        if constexpr (sizeof(T) == 4) {
            tc::sts64(a, __float_as_uint(v.x), __float_as_uint(v.y));
        } else {
            const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
            tc::sts32(a, *reinterpret_cast<const uint32_t*>(&r));
        }
    }
};

// Inputs whose rows begin anywhere, for blocks of one batch row: a step's row of the tile comes as the 16-byte pieces of
// memory that it lies in, one more than it is long, and is read from where it begins in the first of them.  Where
// that is goes by the step's place in its stretch alone: L steps are a multiple of 16 bytes apart.  Stretches begin
// `SKEW` bytes further on each, in other banks.  Rows begin at multiples of CB bytes.
template <typename T, int L, int CB, int DIR> struct ScanWindow {
    using Tile = ScanTile<T, L>;
    static constexpr int ES = Tile::ES, CHUNKS = Tile::ROW / 16, ROWS = SCAN_THREADS / CHUNKS, N = Tile::RT / ROWS;
    static constexpr int PITCH = Tile::ROW + 16, SKEW = ES == 2 ? 16 : L == 4 ? 96 : 32;
    static constexpr int ARRAY = Tile::RT * PITCH + SCAN_SEGS * SKEW;
    static_assert(L * ES % 16 == 0, "a stretch's steps repeat their places");
    struct Cursor {
        const char *at, *last;  // the row of the thread's first step, and of the one whose last piece it takes
        const char* lowest;     // of the array
        int64_t hop, round;
    };
    int chunk, u0, bytes, len;
    static __device__ __forceinline__ uint32_t place(int u) { return uint32_t(u * PITCH + u / L * SKEW); }
    __device__ __forceinline__ ScanWindow(const ScanPlan& p, const ScanAt& q, const int* lens)
    {
        chunk = int(threadIdx.x) % CHUNKS;
        u0 = int(threadIdx.x) / CHUNKS;
        bytes = min(64, p.D - q.c0) * ES;
        len = lens[0];
    }
    __device__ __forceinline__ Cursor cursor(const ScanAt& q, const void* array, const conv_rows_t& r, int64_t first,
                                             int64_t span) const
    {
        const char* a = static_cast<const char*>(array);
        const int64_t row = q.b0 * r.batch + q.c0 + first * r.step;
        return {a + (row + DIR * u0 * r.step) * ES, a + (row + DIR * int(threadIdx.x) * r.step) * ES, a,
                DIR * ROWS * r.step * ES, DIR * span * r.step * ES};
    }
    // Where the first step of a lane's stretch begins in its first piece.
    static __device__ __forceinline__ uint32_t begins(const ScanAt& q, const void* array, const conv_rows_t& r, int64_t first)
    {
        const int64_t row = q.b0 * r.batch + q.c0 + (first + DIR * q.seg * L) * r.step;
        return uint32_t((reinterpret_cast<uintptr_t>(array) + uint64_t(row) * ES) & 15);
    }
    __device__ __forceinline__ void piece(uint32_t row, int k, const char* at, const char* lowest) const
    {
        const int off = k * 16 - int(reinterpret_cast<uintptr_t>(at) & 15);  // of the piece, from the row's first byte
        if (off >= bytes) return;
        const uint32_t to = row + uint32_t(k * 16);
        if (off < 0 && at + off < lowest) {  // the array's first piece, which begins before the array does
#pragma unroll
            for (int e = 0; e < 16; e += ES)
                if (off + e >= 0 && off + e < bytes) {
                    if constexpr (ES == 4) tc::sts32(to + e, *reinterpret_cast<const uint32_t*>(at + off + e));
                    else tc::sts16(to + e, *reinterpret_cast<const uint16_t*>(at + off + e));
                }
        } else {
            const int size = min(16, bytes - off);  // (what lies behind the row's last channel may not be there)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(at + off), "r"(size) : "memory");
        }
    }
    __device__ __forceinline__ void fill(Cursor& c, uint32_t to, int first, int shift) const
    {
        const char* src = c.at;
        const unsigned some = unsigned(max(0, len - shift));
#pragma unroll
        for (int k = 0; k < N; ++k, src += c.hop)
            if (unsigned(first + DIR * (u0 + k * ROWS) - shift) < some) piece(to + place(u0 + k * ROWS), chunk, src, c.lowest);
        const int u = int(threadIdx.x);
        if (u < Tile::RT && unsigned(first + DIR * u - shift) < some) piece(to + place(u), CHUNKS, c.last, c.lowest);
        c.at += c.round;
        c.last += c.round;
    }
    static __device__ __forceinline__ uint32_t lane(const ScanAt& q)
    {
        return place(q.seg * L) + uint32_t(q.warp * 8 * ES + q.pair * 2 * ES);
    }
    // Two channels of the row that begins at byte `at` and `begin` more.
    static __device__ __forceinline__ float2 read(uint32_t at, uint32_t begin)
    {
        at += begin & 15u;
        if constexpr (ES == 4 && CB == 8) {
            const uint2 u = tc::lds64(at);
            return make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        } else if constexpr (ES == 4) {
            return make_float2(__uint_as_float(tc::lds32(at)), __uint_as_float(tc::lds32(at + 4)));
        } else {
            const uint32_t word = at & ~3u;
            const uint32_t u = CB == 4 ? tc::lds32(at)
                                       : __funnelshift_r(tc::lds32(word), tc::lds32(word + 4), (at & 2u) * 8u);
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
        }
    }
};

// The warp's stretches joined along time, and with those of the same warp in the cluster's other blocks.
struct ScanExchange {
    uint32_t bars, slots;  // two mbarriers a warp; [parity][rank][warp][pair] of (A, H) twice
    bool dead = false;

    __device__ __forceinline__ void init(const ScanAt& q, uint32_t sm)
    {
        bars = sm + uint32_t(q.warp * 16);
        slots = sm + SCAN_WARPS * 16;
        if (q.C > 1 && (threadIdx.x & 31) == 0) {
            tc::mbar_init(bars, 1);
            tc::mbar_init(bars + 8, 1);
            tc::fence_mbar_init();
        }
    }
    // Behind a barrier of the cluster: the first two rounds may come in.
    __device__ __forceinline__ void arm(const ScanAt& q, int parity) const
    {
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive_expect_tx(bars + uint32_t(parity) * 8, uint32_t(q.C) * 64u);
    }
    // (A, H) of each of eight neighbours, four lanes apart, joined with all before it.
    template <bool RESET> static __device__ __forceinline__ void join_all(float2& A, float2& H)
    {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
            const float2 a = shfl_up(A, o), h = shfl_up(H, o);
            if (int(threadIdx.x & 31) >= o) scan_join<RESET>(A, H, a, h);
        }
    }
    // The same where some have a reset in them: not by their A, but by a vote, as bits 28 to 31 for the lane's own, 24 to
    // 27 for the one before it and so on.  Two instructions a step less for each of four values.
    static __device__ __forceinline__ void join_all(float2& A, float2& H, uint32_t cuts)
    {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
            const float2 a = shfl_up(A, o), h = shfl_up(H, o);
            if (int(threadIdx.x & 31) >= o) {
                if (cuts < 1u << (32 - o)) H = fma2(A, h, H);  // none among those that are joined already
                A = mul2(A, a);
            }
        }
    }
    static __device__ __forceinline__ uint32_t vote(const ScanAt& q, bool cut)
    {
        return __ballot_sync(0xFFFFFFFFu, cut) << (28 - 4 * q.seg);
    }
    template <bool RESET> static __device__ __forceinline__ float2 enter(float2 A, float2 H, uint32_t cuts, float2 state)
    {
        return RESET && cuts != 0 ? H : fma2(A, state, H);
    }
    // Joins the warp's stretches; (A, H) become the lane's and all before it, cuts the resets among them.  With a
    // cluster, tells its blocks.
    template <bool RESET>
    __device__ __forceinline__ void send(const ScanAt& q, int round, float2& A, float2& H, bool cut, uint32_t& cuts) const
    {
        cuts = RESET ? vote(q, cut) : 0u;
        if constexpr (RESET) join_all(A, H, cuts);
        else join_all<false>(A, H);
        if (q.C == 1) return;
        // the last stretch's lanes hold the warp's; lane (seg, pair) tells rank seg
        float2 a = shfl(A, 28 + q.pair);
        const float2 h = shfl(H, 28 + q.pair);
        if (RESET && __any_sync(0xFFFFFFFFu, cut)) a = both(-1.f);
        if (q.seg < q.C && !dead) {
            const int parity = round & 1;
            const uint32_t to = slots + uint32_t(((parity * q.C + q.rank) * SCAN_WARPS + q.warp) * 64 + q.pair * 16);
            tc::st_async_f4(tc::dsmem_addr(to, uint32_t(q.seg)),
                            tc::dsmem_addr(bars + uint32_t(parity) * 8, uint32_t(q.seg)), a.x, a.y, h.x, h.y);
        }
    }
    // state: in, what enters the round; out, what enters the next one.  Returns what enters the lane's stretch.
    template <bool RESET>
    __device__ __forceinline__ float2 receive(const ScanAt& q, int round, float2 A, float2 H, uint32_t cuts, float2& state)
    {
        float2 in = state;
        if (q.C > 1) {
            const int parity = round & 1;
            const uint32_t bar = bars + uint32_t(parity) * 8, phase = uint32_t(round >> 1) & 1u;
            bool here = dead;
            for (int k = 0; k < 32 && !here; ++k) here = tc::mbar_test_wait(bar, phase);  // soon, mostly
            if (!here && !tc::mbar_wait(bar, phase)) {
                dead = true;  // the results are wrong and the status says so; every later wait is skipped
                atomicOr(&g_scan_status, CONV_STATUS_SCAN);
            }
            if (!dead) arm(q, parity);  // of the round after the next
            // lane (seg, pair) takes rank seg's
            float2 a = both(1.f), h = both(0.f);
            if (q.seg < q.C) {
                const float4 v = tc::lds_f4(slots + uint32_t(((parity * q.C + q.seg) * SCAN_WARPS + q.warp) * 64 + q.pair * 16));
                a = make_float2(v.x, v.y);
                h = make_float2(v.z, v.w);
            }
            __syncwarp();  // read by all before the round after the next is announced
            const uint32_t theirs = RESET ? vote(q, a.x < 0.f) : 0u;
            if constexpr (RESET) join_all(a, h, theirs);
            else join_all<false>(a, h);
            const float2 s = enter<RESET>(a, h, theirs, state);
            if (q.rank > 0) in = shfl(s, (q.rank - 1) * 4 + q.pair);
            state = shfl(s, 28 + q.pair);
        } else {
            state = shfl(enter<RESET>(A, H, cuts, state), 28 + q.pair);
        }
        // what the stretches in front of this one make of it
        const float2 f = shfl_up(enter<RESET>(A, H, cuts, in), 4);
        return q.seg == 0 ? in : f;
    }
};

// The reset flags of a lane's stretch, a bit a step.  The four lanes of a stretch read a step each, a round ahead; what
// they read is looked at when it is needed.
template <int L, int DIR> struct ScanFlags {
    const uint8_t* row = nullptr;
    int len = 0;
    uint8_t next[L / 4];
    __device__ __forceinline__ void fetch(const ScanAt& q, int t0)
    {
#pragma unroll
        for (int k = 0; k < L / 4; ++k) {
            const int t = t0 + DIR * (q.pair + 4 * k);
            next[k] = 0;
            if (row && t >= 0 && t < len) next[k] = row[t];
        }
    }
    __device__ __forceinline__ uint32_t take(const ScanAt& q) const
    {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < L / 4; ++k) m |= next[k] != 0 ? 1u << (4 * k) : 0u;
        m <<= q.pair;
        m |= __shfl_xor_sync(0xFFFFFFFFu, m, 1);
        return m | __shfl_xor_sync(0xFFFFFFFFu, m, 2);
    }
};

__device__ __forceinline__ void scan_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void scan_arrived(int stages)
{
    if (stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
}

// Lengths of the block's batch rows, the exchange; returns the address of the stages.
__device__ __forceinline__ uint32_t scan_setup(const ScanPlan& p, const ScanAt& q, const int32_t* lengths, int* lens,
                                               uint32_t exchange, ScanExchange& ex)
{
    if (int(threadIdx.x) < 1 << p.by_log) {
        const int b = q.b0 + int(threadIdx.x);
        lens[threadIdx.x] = b < p.B ? scan_length(p, lengths, b) : 0;
    }
    ex.init(q, exchange);
    if (q.C > 1) {
        tc::cluster_sync();  // every block of the cluster is there
        ex.arm(q, 0);
        ex.arm(q, 1);
    } else {
        __syncthreads();
    }
    return exchange + (q.C > 1 ? SCAN_WARPS * 16 + 2 * q.C * SCAN_WARPS * 64 : 0);
}

__device__ __forceinline__ float2 scan_state(const ScanPlan& p, const ScanAt& q, const float* from)
{
    float2 s = both(0.f);
    if (from && q.b < p.B && q.c < p.D) {
        s.x = from[int64_t(q.b) * p.D + q.c];
        if (q.c + 1 < p.D) s.y = from[int64_t(q.b) * p.D + q.c + 1];
    }
    return s;
}
__device__ __forceinline__ void scan_store(const ScanPlan& p, const ScanAt& q, float* to, float2 s)
{
    if (to && q.rank == 0 && q.seg == 0 && q.b < p.B && q.c < p.D) {
        to[int64_t(q.b) * p.D + q.c] = s.x;
        if (q.c + 1 < p.D) to[int64_t(q.b) * p.D + q.c + 1] = s.y;
    }
}

// (A, H) of the pieces of time: [piece][batch row][channel], and behind them, as H, the state that enters the row (it
// may lie where the state behind it is written).
__device__ __forceinline__ int64_t scan_piece_at(const ScanPlan& p, const ScanAt& q, int piece)
{
    return (int64_t(piece) * p.B + q.b) * p.D + q.c;
}
// What the pieces in front of this one make of the state that enters the row: each of the warp's eight groups of
// lanes joins an eighth of them.
template <bool RESET>
__device__ __forceinline__ float2 scan_pieces(const ScanPlan& p, const ScanAt& q, const float2* pieces)
{
    float2 A = both(1.f), H = both(0.f), state = both(0.f);
    const int each = (q.piece + SCAN_SEGS - 1) / SCAN_SEGS, stop = min(q.piece, (q.seg + 1) * each);
    if (q.b < p.B && q.c < p.D) {
        const bool two = q.c + 1 < p.D;
#pragma unroll 4
        for (int k = q.seg * each; k < stop; ++k) {
            const float2* at = pieces + scan_piece_at(p, q, k);
            const float2 u = at[0], v = two ? at[1] : make_float2(1.f, 0.f);
            float2 a = make_float2(u.x, v.x), h = make_float2(u.y, v.y);
            scan_join<RESET>(a, h, A, H);
            A = a;
            H = h;
        }
        const float2* at = pieces + scan_piece_at(p, q, p.pieces);
        state = make_float2(at[0].y, two ? at[1].y : 0.f);
    }
    ScanExchange::join_all<RESET>(A, H);
    return shfl(scan_enter<RESET>(A, H, state), 28 + q.pair);
}

// (A, H) of each piece, forward from x and gate, backward (DIR = -1) from dh and gate.
template <typename T, int L, int CB, bool RESET, int DIR>
__global__ void __launch_bounds__(SCAN_THREADS, 3)
scan_part_totals(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const T* dh, const float* state,
                 const uint8_t* reset, const int32_t* lengths, float2* pieces)
{
    extern __shared__ __align__(128) uint8_t sm[];
    int* const lens = reinterpret_cast<int*>(sm);
    using Tile = ScanTile<T, L>;
    constexpr int STAGE = 2 * Tile::ARRAY;
    const ScanAt q(p);
    ScanExchange ex;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const uint32_t stages = scan_setup(p, q, lengths, lens, tc::smem_u32(sm) + SCAN_LENS, ex);
    const int len = lens[q.warp >> p.wx_log];
    using Copy = ScanCopy<T, L, CB, DIR>;
    const Copy copy(p, q, lens);
    const ScanLane<T, L> lane(q);
    constexpr int span = Tile::RT;
    const int begin = DIR > 0 ? 0 : p.T - 1;  // step u is begin + DIR * u
    typename Copy::Cursor ca = DIR > 0 ? copy.cursor(q, x, p.x, begin + q.begin, span)
                                       : copy.cursor(q, dh, p.dh, begin - q.begin, span);
    typename Copy::Cursor cg = copy.cursor(q, gate, p.gate, begin + DIR * q.begin, span);
    ScanFlags<L, DIR> flags;
    if (RESET && q.b < p.B) {
        flags.row = reset + int64_t(q.b) * p.T;
        flags.len = len;
        flags.fetch(q, begin + DIR * (q.begin + q.seg * L));
    }
    auto fill = [&](int slot, int base) {
        if (base < q.end) {
            copy.fill(ca, stages + slot * STAGE, begin + DIR * base, 0);
            copy.fill(cg, stages + slot * STAGE + Tile::ARRAY, begin + DIR * base, 0);
        }
        scan_commit();
    };
    fill(0, q.begin);
    float2 A = both(1.f), H = both(0.f);
    int now = 0;
    for (int base = q.begin; base < q.end; base += span, now ^= 1) {
        scan_arrived(2);
        fill(now ^ 1, base + span);
        const uint32_t stage = stages + now * STAGE;
        const int t0 = begin + DIR * (base + q.seg * L);
        uint32_t cut = 0;
        if (RESET) {
            cut = flags.take(q);
            flags.fetch(q, t0 + DIR * span);
        }
        float2 a = both(1.f), h = both(0.f);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int t = t0 + DIR * i;
            if (t < 0 || t >= len) continue;
            float2 e;
            const float2 z = scan_gate<T>(lane.read(stage, 1, i), e), keep = one_minus(z), v = lane.read(stage, 0, i);
            if (DIR > 0) {
                if (RESET && (cut >> i & 1u)) h = both(0.f);
                h = fma2(keep, h, mul2(z, v));
            } else {
                h = mul2(keep, add2(v, h));
                if (RESET && (cut >> i & 1u)) h = both(0.f);
            }
            a = mul2(a, keep);
        }
        if (RESET && cut != 0) a = both(-1.f);
        ScanExchange::join_all<RESET>(a, h);
        a = shfl(a, 28 + q.pair);
        h = shfl(h, 28 + q.pair);
        scan_join<RESET>(a, h, A, H);
        A = a;
        H = h;
    }
    if (q.seg == 0 && q.b < p.B && q.c < p.D) {
        float2* to = pieces + scan_piece_at(p, q, q.piece);
        to[0] = make_float2(A.x, H.x);
        if (q.c + 1 < p.D) to[1] = make_float2(A.y, H.y);
        if (q.piece == 0) {
            const float2 v = scan_state(p, q, state);
            to = pieces + scan_piece_at(p, q, p.pieces);
            to[0] = make_float2(0.f, v.x);
            if (q.c + 1 < p.D) to[1] = make_float2(0.f, v.y);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <typename T, int L, int CB, bool WINDOW, bool RESET>
__global__ void __launch_bounds__(SCAN_THREADS, sizeof(T) == 2 || WINDOW ? 2 : 3)
scan_part_fwd(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const float* h0, const uint8_t* reset,
              const int32_t* lengths, const float2* pieces, T* h, float* last)
{
    extern __shared__ __align__(128) uint8_t sm[];
    int* const lens = reinterpret_cast<int*>(sm);
    using Tile = ScanTile<T, L>;
    using Copy = ScanCopy<T, L, CB, 1>;
    using Window = ScanWindow<T, L, CB, 1>;
    using In = std::conditional_t<WINDOW, Window, Copy>;
    constexpr int ARRAY = WINDOW ? Window::ARRAY : Tile::ARRAY, STAGE = 2 * ARRAY;
    const ScanAt q(p);
    ScanExchange ex;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float2 state = p.pieces > 1 ? scan_pieces<RESET>(p, q, pieces) : scan_state(p, q, h0);
    const uint32_t stages = scan_setup(p, q, lengths, lens, tc::smem_u32(sm) + SCAN_LENS, ex);
    const int len = lens[q.warp >> p.wx_log];
    const Copy copy(p, q, lens);
    const In in_copy(p, q, lens);
    const ScanLane<T, L> lane(q);
    const int span = q.C * Tile::RT, rank0 = q.rank * Tile::RT;  // (T + span is below 2^31)
    typename In::Cursor cx = in_copy.cursor(q, x, p.x, q.begin + rank0, span);
    typename In::Cursor cg = in_copy.cursor(q, gate, p.gate, q.begin + rank0, span);
    typename Copy::Cursor ch = copy.cursor(q, h, p.h, q.begin + rank0, span);
    // Results wait in the places of x, or, where those are not a lane's own, behind the stages, two rounds in turn.
    const uint32_t results = stages + p.stages * STAGE;
    const uint32_t bx = WINDOW ? Window::begins(q, x, p.x, q.begin + rank0) : 0;
    const uint32_t bg = WINDOW ? Window::begins(q, gate, p.gate, q.begin + rank0) : 0;
    auto value = [&](uint32_t stage, int array, int i) {
        if constexpr (WINDOW)
            return Window::read(stage + Window::lane(q) + uint32_t(array * ARRAY + i * Window::PITCH),
                                array == 0 ? bx + uint32_t(i) * uint32_t(p.x.step * Tile::ES)
                                           : bg + uint32_t(i) * uint32_t(p.gate.step * Tile::ES));
        else
            return lane.read(stage, array, i);
    };
    ScanFlags<L, 1> flags;
    if (RESET && q.b < p.B) {
        flags.row = reset + int64_t(q.b) * p.T;
        flags.len = len;
        flags.fetch(q, q.begin + rank0 + q.seg * L);
    }
    auto fill = [&](int slot, int base) {
        if (base < q.end) {
            in_copy.fill(cx, stages + slot * STAGE, base + rank0, 0);
            in_copy.fill(cg, stages + slot * STAGE + ARRAY, base + rank0, 0);
        }
        scan_commit();
    };
    for (int k = 0; k < p.stages - 1; ++k) fill(k, q.begin + k * span);
    int now = 0, round = 0;
    for (int base = q.begin; base < q.end; base += span, ++round) {
        const int prev = now == 0 ? p.stages - 1 : now - 1;
        scan_arrived(p.stages);
        // The stage of a round ago, which nobody reads any more: its results go out, a later round comes in.  Between
        // send and receive, where the cluster's answers are waited for; loads that a thread waits for come first.
        auto turn = [&] {
            if (round > 0) copy.drain(ch, WINDOW ? results + ((round - 1) & 1) * Tile::ARRAY : stages + prev * STAGE, base - span + rank0, p.T);
            fill(prev, base + (p.stages - 1) * span);
        };
        if (CB == 2 && !WINDOW) turn();
        const uint32_t stage = stages + now * STAGE;
        const int t0 = base + rank0 + q.seg * L;
        uint32_t cut = 0;
        if (RESET) {
            cut = flags.take(q);
            flags.fetch(q, t0 + span);
        }
        // a step is h -> keep h + in; one that the row does not have keeps it as it is
        float2 keep[L], in[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float2 e;
            const float2 z = scan_gate<T>(value(stage, 1, i), e);
            keep[i] = one_minus(z);
            in[i] = mul2(z, value(stage, 0, i));
        }
        const bool full = t0 + L <= len;
        if (!full) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (t0 + i >= len) {
                    keep[i] = both(1.f);
                    in[i] = both(0.f);
                }
        }
        float2 A = both(1.f), H = both(0.f);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (RESET && (cut >> i & 1u)) H = both(0.f);
            H = fma2(keep[i], H, in[i]);
            A = mul2(A, keep[i]);
        }
        uint32_t cuts;
        ex.send<RESET>(q, round, A, H, cut != 0, cuts);
        if (CB != 2 || WINDOW) turn();
        float2 st = ex.receive<RESET>(q, round, A, H, cuts, state);
        const uint32_t out = WINDOW ? results + (round & 1) * Tile::ARRAY : stage;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (RESET && (cut >> i & 1u)) st = both(0.f);
            st = fma2(keep[i], st, in[i]);
            lane.write(out, 0, i, st);
        }
        if (!full) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (t0 + i >= len) lane.write(out, 0, i, both(0.f));
        }
        now = now + 1 == p.stages ? 0 : now + 1;
    }
    if (round > 0) {
        __syncthreads();
        copy.drain(ch, WINDOW ? results + ((round - 1) & 1) * Tile::ARRAY : stages + (now == 0 ? p.stages - 1 : now - 1) * STAGE,
                   q.begin + (round - 1) * span + rank0, p.T);
    }
    if (q.end == p.T) scan_store(p, q, last, state);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (q.C > 1) tc::cluster_sync();  // nothing is sent to a block that has ended
}

// Time runs backwards: a lane's stretch is the steps t = T - 1 - u, u = u0 .. u0 + L - 1, and the state is what
// flows from step t into t - 1, (1 - z[t]) s[t].
template <typename T, int L, int CB, bool WINDOW, bool RESET>
__global__ void __launch_bounds__(SCAN_THREADS, sizeof(T) == 2 || WINDOW ? 2 : 3)
scan_part_bwd(const __grid_constant__ ScanPlan p, const T* x, const T* gate, const T* h, const T* dh, const float* h0,
              const float* dlast, const uint8_t* reset, const int32_t* lengths, const float2* pieces, T* dx, T* dgate,
              float* dh0)
{
    extern __shared__ __align__(128) uint8_t sm[];
    int* const lens = reinterpret_cast<int*>(sm);
    using Tile = ScanTile<T, L>;
    using Copy = ScanCopy<T, L, CB, -1>;
    using Window = ScanWindow<T, L, CB, -1>;
    using In = std::conditional_t<WINDOW, Window, Copy>;
    constexpr int ARRAY = WINDOW ? Window::ARRAY : Tile::ARRAY, STAGE = 4 * ARRAY;
    const ScanAt q(p);
    ScanExchange ex;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    float2 state = p.pieces > 1 ? scan_pieces<RESET>(p, q, pieces) : scan_state(p, q, dlast);
    const uint32_t stages = scan_setup(p, q, lengths, lens, tc::smem_u32(sm) + SCAN_LENS, ex);
    const int len = lens[q.warp >> p.wx_log];
    const Copy copy(p, q, lens);
    const In in_copy(p, q, lens);
    const ScanLane<T, L> lane(q);
    const int span = q.C * Tile::RT, last0 = p.T - 1 - q.rank * Tile::RT;
    const int first = last0 - q.begin;
    typename In::Cursor cx = in_copy.cursor(q, x, p.x, first, span), cg = in_copy.cursor(q, gate, p.gate, first, span),
                        cd = in_copy.cursor(q, dh, p.dh, first, span), ch = in_copy.cursor(q, h, p.h, first - 1, span);
    typename Copy::Cursor ox = copy.cursor(q, dx, p.dx, first, span), og = copy.cursor(q, dgate, p.dgate, first, span);
    // (as in the forward)
    const uint32_t results = stages + p.stages * STAGE;
    const uint32_t bx = WINDOW ? Window::begins(q, x, p.x, first) : 0, bg = WINDOW ? Window::begins(q, gate, p.gate, first) : 0;
    const uint32_t bd = WINDOW ? Window::begins(q, dh, p.dh, first) : 0, bh = WINDOW ? Window::begins(q, h, p.h, first - 1) : 0;
    auto value = [&](uint32_t stage, int array, int i) {
        if constexpr (WINDOW) {
            const uint32_t n = uint32_t(i), es = Tile::ES;
            const uint32_t begin = array == 0   ? bx - n * uint32_t(p.x.step) * es
                                   : array == 1 ? bg - n * uint32_t(p.gate.step) * es
                                   : array == 2 ? bd - n * uint32_t(p.dh.step) * es
                                                : bh - n * uint32_t(p.h.step) * es;
            return Window::read(stage + Window::lane(q) + uint32_t(array * ARRAY + i * Window::PITCH), begin);
        } else {
            return lane.read(stage, array, i);
        }
    };
    ScanFlags<L, -1> flags;
    if (RESET && q.b < p.B) {
        flags.row = reset + int64_t(q.b) * p.T;
        flags.len = len;
        flags.fetch(q, last0 - q.begin - q.seg * L);
    }
    auto fill = [&](int slot, int base) {
        if (base < q.end) {
            const uint32_t to = stages + slot * STAGE;
            in_copy.fill(cx, to, last0 - base, 0);
            in_copy.fill(cg, to + ARRAY, last0 - base, 0);
            in_copy.fill(cd, to + 2 * ARRAY, last0 - base, 0);
            in_copy.fill(ch, to + 3 * ARRAY, last0 - base, 1);
        }
        scan_commit();
    };
    auto drain = [&](int slot, int round, int base) {
        const uint32_t from = WINDOW ? results + (round & 1) * 2 * Tile::ARRAY : stages + slot * STAGE;
        copy.drain(ox, from, last0 - base, p.T);
        copy.drain(og, from + Tile::ARRAY, last0 - base, p.T);
    };
    for (int k = 0; k < p.stages - 1; ++k) fill(k, q.begin + k * span);
    int now = 0, round = 0;
    for (int base = q.begin; base < q.end; base += span, ++round) {
        const int prev = now == 0 ? p.stages - 1 : now - 1;
        scan_arrived(p.stages);
        // The stage of a round ago, which nobody reads any more: its results go out, a later round comes in.  Between
        // send and receive, where the cluster's answers are waited for; loads that a thread waits for come first.
        auto turn = [&] {
            if (round > 0) drain(prev, round - 1, base - span);
            fill(prev, base + (p.stages - 1) * span);
        };
        if (CB == 2 && !WINDOW) turn();
        const uint32_t stage = stages + now * STAGE;
        const int t0 = last0 - base - q.seg * L;
        uint32_t cut = 0;
        if (RESET) {
            cut = flags.take(q);
            flags.fetch(q, t0 - span);
        }
        const bool full = t0 < len && t0 - L + 1 > 0;  // the row has all of the steps, and one before them
        // s = d + state, state -> (1 - z) s; dx = z s, dgate = w s
        float2 z[L], d[L], w[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            float2 e;
            z[i] = scan_gate<T>(value(stage, 1, i), e);
            d[i] = value(stage, 2, i);
            float2 before = value(stage, 3, i);
            if (RESET && (cut >> i & 1u)) before = both(0.f);
            w[i] = mul2(scan_slope(e, z[i]), fma2(before, both(-1.f), value(stage, 0, i)));
        }
        if (!full) {
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (t0 - i < 0 || t0 - i >= len) z[i] = d[i] = w[i] = both(0.f);
            // step 0 comes behind h0
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (t0 == i && len > 0) {
                    float2 e;
                    const float2 g = scan_gate<T>(value(stage, 1, i), e);
                    const float2 before = RESET && (cut >> i & 1u) ? both(0.f) : scan_state(p, q, h0);
                    w[i] = mul2(scan_slope(e, g), fma2(before, both(-1.f), value(stage, 0, i)));
                }
        }
        float2 A = both(1.f), H = both(0.f);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const float2 keep = one_minus(z[i]);
            H = mul2(keep, add2(d[i], H));
            if (RESET && (cut >> i & 1u)) H = both(0.f);
            A = mul2(A, keep);
        }
        uint32_t cuts;
        ex.send<RESET>(q, round, A, H, cut != 0, cuts);
        if (CB != 2 || WINDOW) turn();
        float2 st = ex.receive<RESET>(q, round, A, H, cuts, state);
        const uint32_t out = WINDOW ? results + (round & 1) * 2 * Tile::ARRAY : stage;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const float2 f = add2(d[i], st);
            float2 a = mul2(z[i], f), g = mul2(w[i], f);
            st = mul2(one_minus(z[i]), f);
            if (RESET && (cut >> i & 1u)) st = both(0.f);
            if (!full && t0 - i >= len) a = g = both(0.f);
            lane.write(out, 0, i, a);
            lane.write(out, 1, i, g);
        }
        now = now + 1 == p.stages ? 0 : now + 1;
    }
    if (round > 0) {
        __syncthreads();
        drain(now == 0 ? p.stages - 1 : now - 1, round - 1, q.begin + (round - 1) * span);
    }
    if (q.end == p.T) scan_store(p, q, dh0, state);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (q.C > 1) tc::cluster_sync();
}

int log2_up(int64_t n)
{
    int k = 0;
    while ((int64_t(1) << k) < n) ++k;
    return k;
}

}  // namespace

// `chunk`: bytes that every row begins at a multiple of, 16 at most.
ScanPlan scan_plan(const conv_scan_desc_t& e, const DevInfo& d, bool bwd, int chunk)
{
    ScanPlan p = {};
    const int es = e.dtype == CONV_F32 ? 4 : 2;
    p.B = e.B; p.T = e.T; p.D = e.D;
    p.x = e.x; p.gate = e.gate; p.h = e.h; p.dh = e.dh; p.dx = e.dx; p.dgate = e.dgate;
    const bool pairs = chunk >= 2 * es && e.D % 2 == 0;
    p.V = pairs ? 2 : 1;
    p.cols = (e.D + p.V - 1) / p.V;
    p.pieces = 1;
    p.piece = e.T;
    // Parts: rounds, and blocks without their number along time.
    p.CB = chunk >= 16 && e.D % (16 / es) == 0 ? 16 : es == 4 || (chunk >= 4 && e.D % 2 == 0) ? 4 : 2;
    p.L = es == 2 ? (bwd ? 8 : 16) : bwd ? 4 : 8;
    p.wx_log = std::min(3, log2_up((int64_t(e.D) + 7) / 8));
    p.by_log = 3 - p.wx_log;
    p.tiles = int((int64_t(e.D) + (8 << p.wx_log) - 1) / (8 << p.wx_log));
    const int64_t blocks = int64_t(p.tiles) * ((int64_t(e.B) + (1 << p.by_log) - 1) >> p.by_log);
    const int64_t rounds = (int64_t(e.T) + SCAN_SEGS * p.L - 1) / (SCAN_SEGS * p.L);
    // Pieces of time, as many as the GPU holds blocks for, of two rounds and more: each is read twice, and a second launch
    // comes on top, which is worth it where a cluster's blocks have some eight rounds more than that.
    // (The number of pieces, and so the workspace, does not go by where rows begin.)
    const int64_t most = std::min<int64_t>(int64_t(d.sms) * 2 / std::max<int64_t>(1, blocks), rounds / 2);
    const bool pieces = most > 8 && rounds >> 3 > 2 * ((rounds + most - 1) / most) + 8;
    // Whole pieces of memory or copies of what rows begin at multiples of, in us: fp32 forward 2 x 16384 x 1023 107 / 136,
    // 2 x 16384 x 1022 100 / 136, backward 5 x 2048 x 777 58 / 87, 2 x 16384 x 1022 293 / 326; bf16 forward 2 x 16384 x 1023 72 / 119,
    // 2 x 16384 x 1022 64 / 75; not the bf16 backward, which has no registers for it (2 x 16384 x 1023 431 / 239, 1022
    // 370 / 155), and not where time is cut into pieces of a few rounds (1 x 30001 x 333 fp32 79 / 67, but bf16 59 / 68).
    p.window = p.by_log == 0 && p.CB < 16 && !(es == 2 && bwd) && (!pieces || p.CB == 2);
    if (p.window && es == 4 && pairs) p.CB = 8;
    // Blocks along time: fewer rounds each, as far as the blocks fit the GPU.  A round takes 2.5 units with one block an SM,
    // 3.8 with two, 7.5 with three, a wave of blocks 5 us (the first 3) and with exchanges along a cluster 6.  The estimate
    // counts three fp32 blocks an SM where copies are of 16 or 4 bytes, for which the kernels are compiled (80 registers);
    // shared memory holds three only with two stages, one or two rounds a block, and with three stages two.  (bf16 backward, 1024
    // channels, clusters of 1, 2, 4, 8 blocks, us: 16 x 300 15 / 22 / 31 / 43, 16 x 2500 82 / 95 / 93 / 111, 8 x 1000 25 / 24 / 28 / 35,
    // 4 x 1000 23 / 17 / 15 / 18, 20 x 2500 132 / 122 / 117 / 137).
    const double unit = p.CB == 16 ? 0.44 : es == 4 ? 0.72 : p.CB == 4 ? 0.62 : bwd ? 1.8 : 0.9;
    const int fit = es == 2 || p.window ? 2 : 3;
    const double round_cost[] = {0, 2.5, 3.8, 7.5};
    const int64_t wave = int64_t(d.sms) * fit;
    int log_c = 0;
    double parts = 0;
    // (Where the backward takes whole pieces of memory, a cluster of 8 has no shared memory for a second block an SM.)
    const int most_c = p.window && bwd ? 2 : 3;
    for (int k = 0; k <= most_c && (k == 0 || (int64_t(1) << (k - 1)) < rounds); ++k) {
        const int64_t n = blocks << k, full = n / wave, rest = n % wave, each = (rounds + (int64_t(1) << k) - 1) >> k;
        const double one = double(full) * round_cost[fit] + round_cost[(rest + d.sms - 1) / d.sms];
        const double time = unit * one * double(each) + double(full + (rest > 0)) * (k == 0 ? 5 : 6) - 2;
        if (k == 0 || time < parts) {
            parts = time;
            log_c = k;
        }
    }
    // Or a walk, whose steps come one behind the other: a step's latency at least, with the steps to come in registers or
    // in shared memory (single bf16 values are none that an asynchronous copy takes), and its bytes.  In us, walk from
    // registers / from shared memory / parts:
    //   bf16 forward   64 x 300 x 328 31 / 18 / 15   48 x 300 x 1024 37 / 23 / 24   452 x 300 x 188 42 / 41 / 50
    //   bf16 backward  64 x 300 x 328 40 / 32 / 22   48 x 100 x 1024 17 / 17 / 20   452 x 300 x 188 64 / 64 / 77
    //   fp32 forward   16 x 300 x 1024 33 / 19 / 13  64 x 300 x 328 36 / 20 / 21    452 x 300 x 188 58 / 58 / 61
    //   fp32 backward  16 x 300 x 1024 47 / 36 / 23  28 x 300 x 1024 53 / 40 / 40   300 x 300 x 130 60 / 68 / 94
    const int64_t threads = int64_t(e.B) * p.cols;
    const bool ring = e.T > 8 && (es == 4 || pairs) && threads < int64_t(d.sms) * (bwd ? 128 : 256);
    // (fp32's expf: a second warp a scheduler doubles a step of the forward from shared memory)
    const double latency = !ring ? (!bwd ? 0.105 : es == 2 ? 0.13 : 0.145)
                           : bwd ? (es == 2 ? 0.098 : 0.113) : es == 4 && threads > int64_t(d.sms) * 128 ? 0.11 : 0.056;
    const double channel = es == 2 ? (bwd ? 2.65e-6 : 1.5e-6) : bwd ? 4e-6 : 2.15e-6;
    const double step = std::max(latency, channel * double(e.B) * double(e.D));
    p.walk = e.T <= 16 || (!pieces && step * e.T <= parts);
    if (p.walk) {
        p.ring = !ring ? 0 : es == 4 && !bwd ? 4 : 2;
        p.L = e.T > 4 ? 8 : e.T > 2 ? 4 : std::max(1, e.T);
        p.threads = WALK_THREADS;
        p.cluster = 1;
        p.blocks = (threads + WALK_THREADS - 1) / WALK_THREADS;
        return p;
    }
    p.cluster = 1 << log_c;
    p.threads = SCAN_THREADS;
    p.blocks = blocks << log_c;
    p.stages = !p.window && rounds > (int64_t(2) << log_c) ? 3 : 2;
    if (pieces) {
        const int64_t each = (rounds + most - 1) / most;
        p.cluster = 1;
        p.piece = int(each * SCAN_SEGS * p.L);
        p.pieces = int((rounds + each - 1) / each);
        p.blocks = blocks * p.pieces;
        p.stages = !p.window && each > 2 ? 3 : 2;
    }
    return p;
}

size_t scan_workspace(const conv_scan_desc_t& e, const DevInfo& d, bool bwd)
{
    const ScanPlan p = scan_plan(e, d, bwd, 16);  // (the pieces do not go by where rows begin)
    return p.pieces > 1 ? size_t(p.pieces + 1) * size_t(e.B) * size_t(e.D) * 8 : 0;
}

namespace {

int scan_smem(const ScanPlan& p, int es, bool bwd)
{
    if (p.walk) return p.ring * RING_STEPS * (bwd ? 4 : 2) * WALK_THREADS * p.V * es;
    const int rt = SCAN_SEGS * p.L, row = 64 * es, inputs = p.stages * (bwd ? 4 : 2), results = 2 * (bwd ? 2 : 1);
    const int skew = es == 2 ? 16 : p.L == 4 ? 96 : 32;  // (ScanWindow's)
    return SCAN_LENS + (p.cluster > 1 ? SCAN_WARPS * 16 + 2 * p.cluster * SCAN_WARPS * 64 : 0) +
           (p.window ? inputs * (rt * (row + 16) + SCAN_SEGS * skew) + results * rt * row : inputs * rt * row);
}

template <int N> using Int = std::integral_constant<int, N>;

// Calls f(T(), L, CB, WINDOW, RESET), the last four as types, for the plan of a call in parts, and g(T(), V, L, RESET) or
// ring(T(), V, RING, RESET) for one that walks.
template <bool BWD, class F, class G, class H>
cudaError_t scan_with(const ScanPlan& p, int dt, bool reset, F&& f, G&& g, H&& ring)
{
    auto parts = [&](auto t, auto r) {
        using L = Int<sizeof(t) == 2 ? (BWD ? 8 : 16) : BWD ? 4 : 8>;
        if (p.CB == 16) return f(t, L(), Int<16>(), std::false_type(), r);
        if constexpr (sizeof(t) == 4 || !BWD)
            if (p.window)
                return p.CB == sizeof(t) ? f(t, L(), Int<sizeof(t)>(), std::true_type(), r)
                                         : f(t, L(), Int<2 * sizeof(t)>(), std::true_type(), r);
        if constexpr (sizeof(t) == 2)
            if (p.CB == 2) return f(t, L(), Int<2>(), std::false_type(), r);
        return f(t, L(), Int<4>(), std::false_type(), r);
    };
    auto walk = [&](auto t, auto r) {
        auto steps = [&](auto v) {
            if constexpr (sizeof(t) == 4 || decltype(v)::value == 2) {
                using Ring = Int<sizeof(t) == 4 && !BWD ? 4 : 2>;
                if (p.ring > 0) return ring(t, v, Ring(), r);
            }
            return p.L == 1 ? g(t, v, Int<1>(), r) : p.L == 2 ? g(t, v, Int<2>(), r) : p.L == 4 ? g(t, v, Int<4>(), r)
                                                                                               : g(t, v, Int<8>(), r);
        };
        return p.V == 2 ? steps(Int<2>()) : steps(Int<1>());
    };
    auto on_reset = [&](auto t) {
        if (p.walk) return reset ? walk(t, std::true_type()) : walk(t, std::false_type());
        return reset ? parts(t, std::true_type()) : parts(t, std::false_type());
    };
    return dt == DT_F32 ? on_reset(float()) : on_reset(__nv_bfloat16());
}

// Time may be cut into pieces (scan_plan: with whole pieces of memory for single bf16 values alone).
constexpr bool scan_cuts(bool window, int CB) { return !window || CB == 2; }

template <typename T, int L, int CB, bool RESET, int DIR>
cudaError_t launch_totals(const ScanPlan& p, const T* x, const T* gate, const T* dh, const float* state,
                          const uint8_t* reset, const int32_t* lengths, float2* pieces, cudaStream_t s)
{
    constexpr auto kern = scan_part_totals<T, L, CB, RESET, DIR>;
    const int smem = SCAN_LENS + 4 * SCAN_SEGS * L * 64 * int(sizeof(T));  // two stages of two arrays
    const cudaError_t err = ensure_smem<kern>(smem);
    if (err != cudaSuccess) return err;
    return launch_ex(kern, dim3(unsigned(p.blocks)), dim3(p.threads), smem, s, 1, true, p, x, gate, dh, state, reset,
                     lengths, pieces);
}

// What every row of the array begins at a multiple of, in bytes: 16, 8, 4 or 2.
int rows_chunk(const void* p, const conv_rows_t& r, int es)
{
    const uint64_t all = reinterpret_cast<uintptr_t>(p) | uint64_t(r.batch) * es | uint64_t(r.step) * es;
    return all % 16 == 0 ? 16 : all % 8 == 0 ? 8 : all % 4 == 0 ? 4 : 2;
}

}  // namespace

cudaError_t run_scan_fwd(const conv_scan_desc_t& e, const DevInfo& d, const void* x, const void* gate, const float* h0,
                         const uint8_t* reset, const int32_t* lengths, void* h, float* last, void* ws, cudaStream_t s)
{
    const int es = e.dtype == CONV_F32 ? 4 : 2;
    const int chunk = std::min({rows_chunk(x, e.x, es), rows_chunk(gate, e.gate, es), rows_chunk(h, e.h, es)});
    const ScanPlan p = scan_plan(e, d, false, chunk);
    const int smem = scan_smem(p, es, false);
    float2* const pieces = static_cast<float2*>(ws);
    const dim3 grid(unsigned(p.blocks)), block(p.threads);
    return scan_with<false>(
        p, e.dtype, reset != nullptr,
        [&](auto t, auto l, auto cb, auto window, auto r) {
            using T = decltype(t);
            constexpr int L = decltype(l)::value, CB = decltype(cb)::value;
            constexpr bool WINDOW = decltype(window)::value, RESET = decltype(r)::value;
            const T *px = static_cast<const T*>(x), *pg = static_cast<const T*>(gate);
            if constexpr (scan_cuts(WINDOW, CB)) {
                cudaError_t err = cudaSuccess;
                if (p.pieces > 1) err = launch_totals<T, L, CB, RESET, 1>(p, px, pg, nullptr, h0, reset, lengths, pieces, s);
                if (err != cudaSuccess) return err;
            }
            constexpr auto kern = scan_part_fwd<T, L, CB, WINDOW, RESET>;
            const cudaError_t err = ensure_smem<kern>(smem);
            if (err != cudaSuccess) return err;
            return launch_ex(kern, grid, block, smem, s, p.cluster, true, p, px, pg, h0, reset, lengths,
                             static_cast<const float2*>(pieces), static_cast<T*>(h), last);
        },
        [&](auto t, auto v, auto l, auto r) {
            using T = decltype(t);
            return launch_ex(scan_walk_fwd<T, decltype(v)::value, decltype(l)::value, decltype(r)::value>, grid, block, 0, s,
                             1, true, p, static_cast<const T*>(x), static_cast<const T*>(gate), h0, reset, lengths,
                             static_cast<T*>(h), last);
        },
        [&](auto t, auto v, auto n, auto r) {
            using T = decltype(t);
            constexpr auto kern = scan_ring_fwd<T, decltype(v)::value, decltype(n)::value, decltype(r)::value>;
            const cudaError_t err = ensure_smem<kern>(smem);
            if (err != cudaSuccess) return err;
            return launch_ex(kern, grid, block, smem, s, 1, true, p, static_cast<const T*>(x), static_cast<const T*>(gate),
                             h0, reset, lengths, static_cast<T*>(h), last);
        });
}

cudaError_t run_scan_bwd(const conv_scan_desc_t& e, const DevInfo& d, const void* x, const void* gate, const void* h,
                         const void* dh, const float* h0, const float* dlast, const uint8_t* reset,
                         const int32_t* lengths, void* dx, void* dgate, float* dh0, void* ws, cudaStream_t s)
{
    const int es = e.dtype == CONV_F32 ? 4 : 2;
    const int chunk = std::min({rows_chunk(x, e.x, es), rows_chunk(gate, e.gate, es), rows_chunk(h, e.h, es),
                                rows_chunk(dh, e.dh, es), rows_chunk(dx, e.dx, es), rows_chunk(dgate, e.dgate, es)});
    const ScanPlan p = scan_plan(e, d, true, chunk);
    const int smem = scan_smem(p, es, true);
    float2* const pieces = static_cast<float2*>(ws);
    const dim3 grid(unsigned(p.blocks)), block(p.threads);
    return scan_with<true>(
        p, e.dtype, reset != nullptr,
        [&](auto t, auto l, auto cb, auto window, auto r) {
            using T = decltype(t);
            constexpr int L = decltype(l)::value, CB = decltype(cb)::value;
            constexpr bool WINDOW = decltype(window)::value, RESET = decltype(r)::value;
            const T *pg = static_cast<const T*>(gate), *pd = static_cast<const T*>(dh);
            if constexpr (scan_cuts(WINDOW, CB)) {
                cudaError_t err = cudaSuccess;
                if (p.pieces > 1) err = launch_totals<T, L, CB, RESET, -1>(p, nullptr, pg, pd, dlast, reset, lengths, pieces, s);
                if (err != cudaSuccess) return err;
            }
            constexpr auto kern = scan_part_bwd<T, L, CB, WINDOW, RESET>;
            const cudaError_t err = ensure_smem<kern>(smem);
            if (err != cudaSuccess) return err;
            return launch_ex(kern, grid, block, smem, s, p.cluster, true, p, static_cast<const T*>(x), pg,
                             static_cast<const T*>(h), pd, h0, dlast, reset, lengths, static_cast<const float2*>(pieces),
                             static_cast<T*>(dx), static_cast<T*>(dgate), dh0);
        },
        [&](auto t, auto v, auto l, auto r) {
            using T = decltype(t);
            return launch_ex(scan_walk_bwd<T, decltype(v)::value, decltype(l)::value, decltype(r)::value>, grid, block, 0, s,
                             1, true, p, static_cast<const T*>(x), static_cast<const T*>(gate), static_cast<const T*>(h),
                             static_cast<const T*>(dh), h0, dlast, reset, lengths, static_cast<T*>(dx),
                             static_cast<T*>(dgate), dh0);
        },
        [&](auto t, auto v, auto n, auto r) {
            using T = decltype(t);
            constexpr auto kern = scan_ring_bwd<T, decltype(v)::value, decltype(n)::value, decltype(r)::value>;
            const cudaError_t err = ensure_smem<kern>(smem);
            if (err != cudaSuccess) return err;
            return launch_ex(kern, grid, block, smem, s, 1, true, p, static_cast<const T*>(x), static_cast<const T*>(gate),
                             static_cast<const T*>(h), static_cast<const T*>(dh), h0, dlast, reset, lengths,
                             static_cast<T*>(dx), static_cast<T*>(dgate), dh0);
        });
}

cudaError_t scan_read_status(unsigned* out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_scan_status, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_scan_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace igc
