// kernels_distill.cu -- the loss of a row of logits z against a teacher's K named entries and its
// gradient.  With P = softmax(z / tau) over the vocabulary and p = softmax(teacher / tau) over the row's
// entries:
//   loss = tau^2 sum_k p_k (log p_k - log P[id_k])        dz = w tau (P - the p_k at their ids)
//
// One pass over a row keeps the running maximum m and the sum of exp((z - m) / tau); a row is one warp's
// (short ones), a block's, or that of a cluster of up to 8 blocks, each with a part of the vocabulary, whose
// (m, sum) travel through distributed shared memory.  The loss with its gradient reads z once: a block's part
// of the row comes to shared memory in a few large copies, waits there for the row's sum, and goes out as
// dz.  Rows begin anywhere: a row is taken by 16-byte vectors of memory, its first and last one by
// elements.
//
// One warp more than those that sweep works on the teacher's entries: their softmax, the student's logits at their
// ids, and which ids occur twice.  dz at the ids is written again, whole, behind the sweep's barrier, by
// one thread an id: no atomic adds, and a fixed order for an id that occurs twice.
//
// Floor: z once, and dz.  Measured, with the share of that floor at the measured copy's bandwidth: 1024 x 50021 fp32
// backward 69 us (87 %), 8192 x 50021 bf16 both at once 299 (81 %) and forward 131 (93 %), 24 x 131071 fp32 forward 6.0 (a launch
// and two trips along a cluster).  Bound by memory, bf16 both at once also by instructions (0.62 issued a slot); rows of a few
// hundred logits by the teacher's entries (32768 x 128 both at once, bf16 with 8 of them 27 against 2.8, fp32 with 100 of
// them 59 against 8.9).
#include <algorithm>

#include "gn_common.cuh"
#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

enum { DISTILL_FWD = 0, DISTILL_BWD = 1, DISTILL_GRAD = 2 };
constexpr int DISTILL_WARPS = 8;       // that sweep a row, where a block does
constexpr int DISTILL_UNROLL = 4;      // vectors a thread has on their way
constexpr int DISTILL_COPIES = 4;      // of a block's part of a row, one behind the other
// Vectors whose sums a thread adds to one another in one chain at most, where each addition may be off by half a step
// the same way.  CHAINS: a thread has more of them, and its chains (512 at most) are added to each other.  (In one
// kernel for both, the registers of the longer form cost rows of any length: 8192 x 50021 bf16 forward 131 us, 138 so.
// Rows of 10 million logits pay 4 %.  log sum exp over 2^30 - 1 logits, in one chain a thread, was off by 9e-4 in bf16 and
// 1.5e-3 in fp32.)
constexpr int DISTILL_CHAIN = 256;

__device__ unsigned g_distill_status = 0;  // CONV_STATUS_DISTILL: a bounded wait ran out

struct Stat { float m, s; };

// m: of both, or 0 while all values are -inf (so that nothing is subtracted from them).
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }
// Over groups of `lanes` lanes (a power of two): the largest m, and the sums brought to it.
__device__ __forceinline__ Stat stat_join(Stat a, int lanes, float k)
{
    float m = a.m;
    for (int o = lanes / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float s = a.s * fast_exp2((a.m - finite_base(m)) * k);
    for (int o = lanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return {m, s};
}

// A row's place: 16-byte vectors from `base` on; vector j holds the row's elements j * VE - off and on.
template <typename T> struct RowAt {
    static constexpr int VE = 16 / int(sizeof(T));
    int64_t first;    // element of the array that vector 0 begins with (may lie before the row)
    int off, V, vecs;
    __device__ __forceinline__ RowAt(const T* z, int64_t n, int64_t ld, int V_) : V(V_)
    {
        const int64_t at = n * ld;
        off = int((reinterpret_cast<uintptr_t>(z + at) & 15u) / sizeof(T));
        first = at - off;
        vecs = (off + V + VE - 1) / VE;
    }
    // Vectors that lie in the row with all their elements: [first_whole, end_whole).
    __device__ __forceinline__ int first_whole() const { return off > 0 ? 1 : 0; }
    __device__ __forceinline__ int end_whole() const { return (off + V) / VE; }
    __device__ __forceinline__ bool whole(int j) const { return j >= first_whole() && j < end_whole(); }
    __device__ __forceinline__ Vec<T, VE> load(const T* z, int j) const
    {
        Vec<T, VE> r;
        const T* p = z + first + int64_t(j) * VE;
        if (whole(j)) {
            r.load(p);
        } else {
            float f[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const int e = j * VE + i - off;
                f[i] = e >= 0 && e < V ? Elem<T>::ld(p + i) : -INFINITY;
            }
            r.set(f);
        }
        return r;
    }
    __device__ __forceinline__ void store(T* dz, int j, const Vec<T, VE>& r) const
    {
        T* p = dz + first + int64_t(j) * VE;
        if (whole(j)) {
            r.store(p);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const int e = j * VE + i - off;
                if (e >= 0 && e < V) Elem<T>::st(p + i, r.get(i));
            }
        }
    }
};

template <typename T, int VE> __device__ __forceinline__ float vec_max(const Vec<T, VE>& v)
{
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(v.r.w);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        return fmaxf(fmaxf(v.get(0), v.get(1)), fmaxf(v.get(2), v.get(3)));
    }
}
template <typename T, int VE> __device__ __forceinline__ float vec_sum(const Vec<T, VE>& v, float base, float k)
{
    float2 t[VE / 2];
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
        const float2 d = mul2(add2(make_float2(v.get(2 * i), v.get(2 * i + 1)), both(-base)), both(k));
        t[i] = make_float2(fast_exp2(d.x), fast_exp2(d.y));
    }
#pragma unroll
    for (int n = VE / 4; n > 0; n /= 2)
#pragma unroll
        for (int i = 0; i < n; ++i) t[i] = add2(t[i], t[i + n]);
    return t[0].x + t[0].y;
}

// The teacher's entries of a row, worked on by one warp.  ids: -1 where the entry names nothing; p: their
// probabilities; zk: the student's logits; total: what is taken off dz there, or -1 where another entry
// with the same id does it.
struct Teacher {
    int* id;
    float *p, *zk, *total;
    float top;       // the largest of the teacher's logits
    uint32_t* seen;  // two bitmaps
    int bits;        // of one, a power of two
    static __host__ __device__ int bytes(int K, int bits) { return 16 * K + bits / 4; }
    __device__ __forceinline__ Teacher(uint8_t* sm, int K, int bits_) : bits(bits_)
    {
        seen = reinterpret_cast<uint32_t*>(sm);
        id = reinterpret_cast<int*>(seen + bits / 16);
        p = reinterpret_cast<float*>(id + K);
        zk = p + K;
        total = zk + K;
    }
    // ids and the teacher's logits; false: the row names nothing.
    __device__ __forceinline__ bool entries(const DistillParams& a, int64_t n, int lane)
    {
        top = -INFINITY;
        bool nan = false;
        for (int k = lane; k < a.K; k += 32) {
            const int64_t at = n * a.K + k;
            const int64_t v = a.ids64 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
            float q = a.teacher_bf16 ? Elem<__nv_bfloat16>::ld(static_cast<const __nv_bfloat16*>(a.teacher) + at)
                                     : static_cast<const float*>(a.teacher)[at];
            const bool named = v >= 0 && v < a.V;
            if (!named) q = -INFINITY;
            id[k] = named ? int(v) : -1;
            p[k] = q;
            top = fmaxf(top, q);
            nan |= q != q;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        nan = __any_sync(0xFFFFFFFFu, nan);
        return !(top == -INFINITY && !nan);
    }
    __device__ __forceinline__ void probabilities(const DistillParams& a, int lane)
    {
        const float base = finite_base(top);
        float sum = 0.f;
        for (int k = lane; k < a.K; k += 32) {
            total[k] = (p[k] - base) * a.inv_tau;  // log p but for the sum, until it is needed no more
            const float e = expf(total[k]);
            p[k] = e;
            sum += e;
        }
        sum = warp_sum(sum);
        const float log_sum = logf(sum), over = __fdiv_rn(1.f, sum);
        for (int k = lane; k < a.K; k += 32) {
            p[k] *= over;
            total[k] -= log_sum;
        }
    }
    // The student's logits of the entries in [lo, hi).
    template <typename T> __device__ __forceinline__ void gather(const DistillParams& a, const T* row, int lo, int hi, int lane)
    {
        for (int k = lane; k < a.K; k += 32) zk[k] = id[k] >= lo && id[k] < hi ? Elem<T>::ld(row + id[k]) : 0.f;
    }
    __device__ __forceinline__ float loss(const DistillParams& a, float m, float log_s, int lane) const
    {
        float sum = 0.f;
        for (int k = lane; k < a.K; k += 32)
            if (!(p[k] == 0.f)) sum += p[k] * (total[k] - ((zk[k] - m) * a.inv_tau - log_s));
        return a.tau * a.tau * warp_sum(sum);
    }
    // total: the sum of p over the entries of an id, at the first of them.  Ids that share a bit of `seen` are
    // looked at one by one, in order.
    __device__ __forceinline__ void totals(const DistillParams& a, int lane)
    {
        if (a.K <= 32) {
            const int me = lane < a.K ? id[lane] : -1;
            const float mine = lane < a.K ? p[lane] : 0.f;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, me < 0 ? -1 - lane : me);
            float t = mine;
            if (__any_sync(0xFFFFFFFFu, (same & (same - 1)) != 0)) {
                t = 0.f;
                for (int j = 0; j < a.K; ++j) {
                    const float q = __shfl_sync(0xFFFFFFFFu, p[min(lane, a.K - 1)], j);
                    if (same >> j & 1u) t += q;
                }
                if (same & ((1u << lane) - 1u)) t = -1.f;
            }
            if (lane < a.K) total[lane] = t;
            return;
        }
        uint32_t* twice = seen + bits / 32;
        for (int i = lane; i < bits / 16; i += 32) seen[i] = 0;
        __syncwarp();
        for (int k = lane; k < a.K; k += 32) {
            if (id[k] < 0) continue;
            const int h = id[k] & (bits - 1);
            if (atomicOr(&seen[h >> 5], 1u << (h & 31)) >> (h & 31) & 1u) atomicOr(&twice[h >> 5], 1u << (h & 31));
        }
        __syncwarp();
        for (int k = lane; k < a.K; k += 32) {
            float t = p[k];
            const int me = id[k], h = me & (bits - 1);
            if (me >= 0 && (twice[h >> 5] >> (h & 31) & 1u)) {
                t = 0.f;
                for (int j = 0; j < a.K; ++j) {
                    if (id[j] != me) continue;
                    if (j < k) {
                        t = -1.f;
                        break;
                    }
                    t += p[j];
                }
            }
            total[k] = t;
        }
    }
};

// Blocks an SM for whose number of registers a kernel is compiled (0: the compiler's choice).
constexpr int distill_blocks(int mode, int NV)
{
    return NV == 0 || NV == 2 ? 5 : mode == DISTILL_BWD ? 0 : mode == DISTILL_GRAD && NV == 8 ? 3 : 4;
}

// NV > 0: a warp a row, which it keeps in registers, NV vectors a lane (but for the gradient alone, which reads it
// once anyway); else a block of `warps` warps, DISTILL_WARPS at most and a power of two, and one for the teacher,
// `cluster` blocks a row.
template <typename T, int MODE, int NV, bool CHAINS = false>
__global__ void __launch_bounds__(NV > 0 ? 256 : DISTILL_WARPS * 32 + 32, distill_blocks(MODE, NV))
distill_kernel(const __grid_constant__ DistillParams a, const T* z, const float* weight, float* zmax, float* zlog,
               float* loss, T* dz)
{
    constexpr bool WARP = NV > 0, HELD = WARP && MODE != DISTILL_BWD;
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ Stat parts[DISTILL_WARPS + 8];
    __shared__ int none;
    __shared__ __align__(8) uint64_t bars[DISTILL_COPIES];
    constexpr int VE = RowAt<T>::VE, U = DISTILL_UNROLL;
    const int lane = int(threadIdx.x) & 31, warp = int(threadIdx.x) >> 5;
    const int C = WARP ? 1 : a.cluster, rank = WARP ? 0 : int(blockIdx.x) % C;
    const int64_t n = WARP ? int64_t(blockIdx.x) * a.rows + warp : int64_t(blockIdx.x) / C;
    const int warps = a.warps, step = WARP ? 32 : warps * 32, me = WARP ? lane : int(threadIdx.x);
    const bool teaches = WARP || warp == warps, sweeps = WARP || !teaches;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (WARP && n >= a.N) return;
    if (!WARP && MODE != DISTILL_BWD && C > 1) tc::cluster_arrive();

    const RowAt<T> row(z, n, a.ld, a.V);
    const T* zrow = z + n * a.ld;
    const int per = (row.vecs + C - 1) / C, j0 = min(rank * per, row.vecs), j1 = min(j0 + per, row.vecs);
    const int lo = max(0, j0 * VE - row.off), hi = min(a.V, j1 * VE - row.off);  // the block's elements
    // whole vectors of the block's, and the one that this thread takes by elements (-1: none)
    const int w0 = max(j0, row.first_whole()), w1 = min(j1, row.end_whole());
    int edge = me == 0 ? 0 : me == 1 && row.vecs > 1 ? row.vecs - 1 : -1;
    if (edge >= 0 && (edge < j0 || edge >= j1 || row.whole(edge))) edge = -1;
    Teacher t(sm + (WARP ? warp * Teacher::bytes(a.K, a.bits) : 0), a.K, a.bits);
    uint8_t* const stage = sm + Teacher::bytes(a.K, a.bits);  // vector j - j0 at the thread that reads it
    const bool staged = !WARP && MODE == DISTILL_GRAD && a.stage_bytes > 0;
    // A block's part of the row comes in a few large copies; `copy` vectors each.
    const int copy = (max(0, w1 - w0) + DISTILL_COPIES * step - 1) / (DISTILL_COPIES * step) * step;
    if (!WARP && staged) {
        if (threadIdx.x == 0) {
            for (int k = 0; k < DISTILL_COPIES; ++k) tc::mbar_init(tc::smem_u32(&bars[k]), 1);
            tc::fence_mbar_init();
            for (int k = 0; k < DISTILL_COPIES; ++k) {
                const int from = w0 + k * copy, n = min(copy, w1 - from);
                if (n <= 0) break;
                tc::mbar_arrive_expect_tx(tc::smem_u32(&bars[k]), uint32_t(n) * 16u);
                tc::bulk_g2s(tc::smem_u32(stage) + uint32_t(from - j0) * 16u, z + row.first + int64_t(from) * VE,
                             uint32_t(n) * 16u, tc::smem_u32(&bars[k]));
            }
        }
        __syncthreads();
    }

    const uint32_t staged_at = tc::smem_u32(stage) - uint32_t(j0) * 16;
    auto waiting = [&](Vec<T, VE>& v, int j) {  // vector j, in shared memory
        const int4 q = tc::lds128(staged_at + uint32_t(j) * 16);
        v.r.w[0] = uint32_t(q.x); v.r.w[1] = uint32_t(q.y); v.r.w[2] = uint32_t(q.z); v.r.w[3] = uint32_t(q.w);
    };

    // A warp's row, all of it on its way beside the teacher's entries.
    Vec<T, VE> held[HELD ? NV : 1], ends;
    auto holds = [&](int u) { return lane + u * 32 >= w0 && lane + u * 32 < w1; };
    if constexpr (HELD) {
        const T* src = z + row.first + lane * VE;
#pragma unroll
        for (int u = 0; u < NV; ++u)
            if (holds(u)) held[u].load(src + u * 32 * VE);
        if (edge >= 0) ends = row.load(z, edge);
    }

    // ---- the teacher's entries, and what the first sweep finds
    bool empty = false;
    const float w = MODE != DISTILL_FWD && weight ? weight[n] : 1.f;
    float m, log_s;
    if (MODE == DISTILL_BWD) {
        m = zmax[n];
        log_s = zlog[n];
        const bool in_place = z == dz;
        if (teaches) {
            empty = !t.entries(a, n, lane);
            if (!WARP && lane == 0) none = empty;
            if (in_place && !empty) t.gather(a, zrow, lo, hi, lane);
        }
        if (WARP) __syncwarp();
        else __syncthreads();
        if (teaches && !empty) {
            t.probabilities(a, lane);
            if (!in_place) t.gather(a, zrow, lo, hi, lane);
        }
        if (WARP) __syncwarp();
    } else {
        if (teaches) {
            empty = !t.entries(a, n, lane);
            if (!WARP && lane == 0) none = empty;
            if (!empty) {
                t.probabilities(a, lane);
                t.gather(a, zrow, 0, a.V, lane);
            }
        }
        Stat st = {-INFINITY, 0.f};
        bool edged = false;  // the vector is one that no copy brought
        auto take = [&](auto& v, int j) {  // vectors j, j + step, ..
            constexpr int count = int(sizeof(v) / sizeof(v[0]));
            float top = st.m;
#pragma unroll
            for (int u = 0; u < count; ++u) {
                top = fmaxf(top, vec_max<T, VE>(v[u]));
                if (staged && edged) v[u].store(reinterpret_cast<T*>(stage + (j + u * step - j0) * 16));
            }
            const float base = finite_base(top);
            if (top > st.m) st.s *= fast_exp2((st.m - base) * a.k);
            st.m = top;
#pragma unroll
            for (int u = 0; u < count; ++u) st.s += vec_sum<T, VE>(v[u], base, a.k);
        };
        if constexpr (WARP) {
            if (edge >= 0) st.m = vec_max<T, VE>(ends);
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if (holds(u)) st.m = fmaxf(st.m, vec_max<T, VE>(held[u]));
            const float base = finite_base(st.m);
            if (edge >= 0) st.s = vec_sum<T, VE>(ends, base, a.k);
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if (holds(u)) st.s += vec_sum<T, VE>(held[u], base, a.k);
        } else if (sweeps) {
            Vec<T, VE> one[1];
            if (edge >= 0) {
                one[0] = row.load(z, edge);
                edged = true;
                take(one, edge);
                edged = false;
            }
            auto all = [&](int from, int to, auto&& read) {
                int j = from + me;
                for (; j + (U - 1) * step < to; j += U * step) {
                    Vec<T, VE> v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) read(v[u], j + u * step);
                    take(v, j);
                }
                for (; j < to; j += step) {
                    read(one[0], j);
                    take(one, j);
                }
            };
            if (staged) {
                for (int k = 0; k < DISTILL_COPIES && w0 + k * copy < w1; ++k) {
                    if (!tc::mbar_wait(tc::smem_u32(&bars[k]), 0u))
                        atomicOr(&g_distill_status, CONV_STATUS_DISTILL);  // the results are wrong, and the status says so
                    all(w0 + k * copy, min(w1, w0 + (k + 1) * copy), waiting);
                }
            } else {
                const T* src = z + row.first;
                auto read = [&](Vec<T, VE>& v, int j) { v.load(src + int64_t(j) * VE); };
                if constexpr (!CHAINS) {
                    all(w0, w1, read);
                } else {
                    float before = 0.f, m_before = -INFINITY;  // the chains so far
                    const int chain = DISTILL_CHAIN * step;
                    for (int from = w0; from < w1; from += chain) {
                        all(from, min(w1, from + chain), read);
                        before = before * fast_exp2((m_before - finite_base(st.m)) * a.k) + st.s;
                        m_before = st.m;
                        st.s = 0.f;
                    }
                    st.s = before;
                }
            }
        }
        st = stat_join(st, 32, a.k);
        if (!WARP) {
            if (lane == 0 && sweeps) parts[warp] = st;
            __syncthreads();
            st = stat_join(parts[lane & (warps - 1)], warps, a.k);
            if (C > 1) {
                tc::cluster_wait();  // every block of the cluster is there
                if (threadIdx.x < unsigned(C))
                    tc::st_dsmem_f2(tc::dsmem_addr(tc::smem_u32(&parts[DISTILL_WARPS + rank]), threadIdx.x), st.m, st.s);
                tc::cluster_sync();
                st = stat_join(parts[DISTILL_WARPS + (lane & (C - 1))], C, a.k);
            }
        }
        m = st.m;
        log_s = logf(st.s);
        if (teaches && rank == 0) {
            const float l = empty ? 0.f : t.loss(a, m, log_s, lane);
            if (lane == 0) {
                loss[n] = l;
                if (MODE == DISTILL_FWD) {
                    zmax[n] = m;
                    zlog[n] = log_s;
                }
            }
        }
    }
    if (MODE == DISTILL_FWD) return;

    // ---- the gradient
    if (!WARP) empty = none != 0;
    const float c = a.scale * a.tau * w, log2_s = log_s * kLog2e;
    const bool zeros = empty || w == 0.f;
    if (teaches && !zeros) t.totals(a, lane);
    if (sweeps) {
        auto give = [&](Vec<T, VE>& v) {
            float f[VE];
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
                const float2 d = fma2(add2(make_float2(v.get(i), v.get(i + 1)), both(-m)), both(a.k), both(-log2_s));
                const float2 e = mul2(make_float2(fast_exp2(d.x), fast_exp2(d.y)), both(c));
                f[i] = e.x;
                f[i + 1] = e.y;
            }
            v.set(f);
            if (zeros) v.zero();
        };
        if constexpr (HELD) {
            if (edge >= 0) {
                give(ends);
                row.store(dz, edge, ends);
            }
            T* dst = dz + row.first + lane * VE;
#pragma unroll
            for (int u = 0; u < NV; ++u)
                if (holds(u)) {
                    give(held[u]);
                    held[u].store(dst + u * 32 * VE);
                }
        }
        Vec<T, VE> one;
        if (!HELD && edge >= 0) {
            if (staged) one.load(reinterpret_cast<const T*>(stage + (edge - j0) * 16));
            else one = row.load(z, edge);
            give(one);
            row.store(dz, edge, one);
        }
        T* dst = dz + row.first + int64_t(w0 + me) * VE;
        auto sweep = [&](auto&& read) {  // read(v, j): vector j
            int j = w0 + me;
            for (; j + (U - 1) * step < w1; j += U * step, dst += U * step * VE) {
                Vec<T, VE> v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) read(v[u], j + u * step);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    give(v[u]);
                    v[u].store(dst + u * step * VE);
                }
            }
            for (; j < w1; j += step, dst += step * VE) {
                read(one, j);
                give(one);
                one.store(dst);
            }
        };
        if (staged) {
            sweep(waiting);
        } else if (!HELD) {
            const T* src = z + row.first;
            sweep([&](Vec<T, VE>& v, int j) { v.load(src + int64_t(j) * VE); });
        }
    }
    if (WARP) __syncwarp();
    else __syncthreads();
    if (zeros) return;
    for (int k = me; k < a.K; k += WARP ? 32 : int(blockDim.x)) {
        const int id = t.id[k];
        if (id < lo || id >= hi || t.total[k] == -1.f) continue;
        Elem<T>::st(dz + n * a.ld + id, c * (fast_exp2((t.zk[k] - m) * a.k - log2_s) - t.total[k]));
    }
}

}  // namespace

namespace {

DistillParams distill_params(const conv_distill_desc_t& e, const void* ids, const void* teacher, float scale)
{
    DistillParams a = {};
    a.N = e.N; a.V = e.V; a.K = e.K; a.ld = e.ld;
    a.ids = ids;
    a.ids64 = e.index_dtype == CONV_INDEX_I64;
    a.teacher = teacher;
    a.teacher_bf16 = e.teacher_dtype == CONV_BF16;
    a.tau = e.temperature;
    a.inv_tau = float(1.0 / double(e.temperature));
    a.k = float(1.4426950408889634 / double(e.temperature));
    a.scale = scale;
    return a;
}

}  // namespace

DistillPlan distill_plan(const conv_distill_desc_t& e, const DevInfo& d, int mode)
{
    DistillPlan p = {};
    const int es = e.dtype == CONV_F32 ? 4 : 2, ve = 16 / es;
    const int64_t vecs = (int64_t(e.V) + ve - 1) / ve + 1;
    const int64_t most = d.smem_optin - 2048;  // (and the static part)
    p.warp = vecs <= 256 && e.K <= 256;
    if (p.warp) {
        p.bits = 2048;
        // The row in registers or read by four vectors a lane, and again for dz, us: bf16 29605 x 1568 forward 35 / 40, at
        // once 51 / 57; 32768 x 128 at once 27 / 32; fp32 29639 x 618 forward 30.4 / 29.5, at once 43.8 / 44.7.  The gradient
        // alone has it no faster: fp32 29639 x 618 36 / 34.
        p.held = mode == DISTILL_BWD ? 4 : vecs <= 64 ? 2 : vecs <= 128 ? 4 : 8;
        const int64_t one = 16 * int64_t(e.K) + p.bits / 4;
        p.rows = int(std::max<int64_t>(1, std::min<int64_t>(8, 48 * 1024 / one)));
        p.cluster = 1;
        p.threads = p.rows * 32;
        p.smem = int(p.rows * one);
        p.blocks = (e.N + p.rows - 1) / p.rows;
        return p;
    }
    p.bits = 8192;
    p.rows = 1;
    const int64_t teacher = 16 * int64_t(e.K) + p.bits / 4;
    // A row's blocks: as many as give every SM four, while a thread has four vectors and more; and as many as keep a
    // block's part small enough for four on an SM.
    int C = 1;
    while (C < 8 && e.N * C < 4 * int64_t(d.sms) && vecs >= int64_t(C) * 2 * DISTILL_WARPS * 32 * 4) C *= 2;
    if (mode == DISTILL_GRAD) {
        while (C < 8 && (vecs + C - 1) / C * 16 + teacher > 55 * 1024) C *= 2;
        const int64_t bytes = (vecs + C - 1) / C * 16;
        p.stage_bytes = bytes + teacher <= most ? int(bytes) : 0;
    }
    // Warps that sweep: a thread has eight vectors and more (6319 x 8978 bf16 backward 88 us with 8 warps, 62 with 4; 20000 x
    // 3000 bf16 at once 136 with 8, 88 with 4, 59 with 2).
    const int64_t part = (vecs + C - 1) / C;
    p.warps = part > 2048 ? 8 : part > 512 ? 4 : 2;
    p.chains = part > DISTILL_CHAIN * p.warps * 32 && mode != DISTILL_BWD && p.stage_bytes == 0;
    p.threads = p.warps * 32 + 32;
    p.cluster = C;
    p.smem = int(teacher) + p.stage_bytes;
    p.blocks = e.N * C;
    return p;
}

namespace {

template <typename T, int MODE>
cudaError_t launch_distill(const DistillPlan& p, DistillParams a, const void* z, const float* weight, float* zmax,
                           float* zlog, float* loss, void* dz, cudaStream_t s)
{
    a.cluster = p.cluster;
    a.rows = p.rows;
    a.warps = p.warps;
    a.bits = p.bits;
    a.stage_bytes = p.stage_bytes;
    auto go = [&](auto kern) {
        return launch_ex(kern, dim3(unsigned(p.blocks)), dim3(p.threads), p.smem, s, p.cluster, true, a,
                         static_cast<const T*>(z), weight, zmax, zlog, loss, static_cast<T*>(dz));
    };
    const int room = p.smem + 1024;  // (the static part comes on top of the dynamic one)
    auto with = [&](auto held, auto chains) {
        constexpr auto kern = distill_kernel<T, MODE, decltype(held)::value, decltype(chains)::value>;
        const cudaError_t e = ensure_smem<kern>(room);
        return e != cudaSuccess ? e : go(kern);
    };
    const std::false_type one;
    if constexpr (MODE != DISTILL_BWD) {
        if (p.chains) return with(std::integral_constant<int, 0>(), std::true_type());
        if (p.warp && p.held == 2) return with(std::integral_constant<int, 2>(), one);
        if (p.warp && p.held == 8) return with(std::integral_constant<int, 8>(), one);
    }
    return p.warp ? with(std::integral_constant<int, 4>(), one) : with(std::integral_constant<int, 0>(), one);
}

template <int MODE>
cudaError_t run_distill(const conv_distill_desc_t& e, const DevInfo& d, const DistillParams& a, const void* z,
                        const float* weight, float* zmax, float* zlog, float* loss, void* dz, cudaStream_t s)
{
    const DistillPlan p = distill_plan(e, d, MODE);
    return e.dtype == CONV_F32 ? launch_distill<float, MODE>(p, a, z, weight, zmax, zlog, loss, dz, s)
                               : launch_distill<__nv_bfloat16, MODE>(p, a, z, weight, zmax, zlog, loss, dz, s);
}

}  // namespace

cudaError_t run_distill_fwd(const conv_distill_desc_t& e, const DevInfo& d, const void* z, const void* ids,
                            const void* teacher, float* loss, float* zmax, float* zlog, cudaStream_t s)
{
    return run_distill<DISTILL_FWD>(e, d, distill_params(e, ids, teacher, 1.f), z, nullptr, zmax, zlog, loss, nullptr, s);
}
cudaError_t run_distill_bwd(const conv_distill_desc_t& e, const DevInfo& d, const void* z, const void* ids,
                            const void* teacher, const float* zmax, const float* zlog, const float* weight, float scale,
                            void* dz, cudaStream_t s)
{
    return run_distill<DISTILL_BWD>(e, d, distill_params(e, ids, teacher, scale), z, weight, const_cast<float*>(zmax),
                                    const_cast<float*>(zlog), nullptr, dz, s);
}
cudaError_t run_distill_grad(const conv_distill_desc_t& e, const DevInfo& d, const void* z, const void* ids,
                             const void* teacher, const float* weight, float scale, float* loss, void* dz, cudaStream_t s)
{
    return run_distill<DISTILL_GRAD>(e, d, distill_params(e, ids, teacher, scale), z, weight, nullptr, nullptr, loss, dz,
                                     s);
}

cudaError_t distill_read_status(unsigned* out, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(out, g_distill_status, sizeof(unsigned));
    if (e == cudaSuccess && reset) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_distill_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace igc
