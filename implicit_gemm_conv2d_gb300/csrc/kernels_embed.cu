// kernels_embed.cu -- embedding lookup with scaling and its gradient:
//   y[t,:] = scale * table[idx[t],:],    dtable[v,:] = scale * sum_{t: idx[t] = v} dy[t,:].
//
// The lookup moves T*D values in and out with one multiply each: bound by memory.
//
// The gradient is a sum per row over the tokens that name it.  The tokens are sorted by row
// (least significant digit first, a stable counting sort a digit), so a row's tokens are one run
// of the sorted order in ascending t: dy is read once, row by row, and no atomic is needed.  The
// sorted order is cut into chunks of equal length, so a row that holds a large share of the
// tokens is spread over many thread groups; a run inside one chunk is written at once, a run
// that crosses chunks leaves fp32 partial sums that a second kernel adds in chunk order.
#include <algorithm>

#include "tc_ptx.cuh"
#include "train_internal.h"

namespace igc {

namespace {

constexpr int SORT_THREADS = 256;
constexpr int SORT_ITEMS = 8;                              // a thread
constexpr int SORT_TILE = SORT_THREADS * SORT_ITEMS;       // tokens a block sorts
constexpr int SORT_MAX_BITS = 9;                           // digit
constexpr int SORT_MAX_BINS = 1 << SORT_MAX_BITS;
constexpr int SUM_THREADS = 256;
constexpr int FIX_THREADS = 512;

struct EmbedPlan {
    int bits, passes, digit_bits;
    int tiles;
    int V;                // vector width of a row
    int nv;               // vectors a row
    int cols, wins;       // column vectors a block, windows
    int chunk, chunks;    // sorted tokens a thread group sums
    size_t off_keys[2], off_pos[2], off_counts, off_totals, off_part, bytes;
};

EmbedPlan embed_plan(const conv_embed_desc_t& e, const DevInfo& d)
{
    EmbedPlan q = {};
    while ((int64_t(1) << q.bits) <= e.V) ++q.bits;  // keys 0 .. V (V: no row)
    q.passes = std::max(1, ceil_div(q.bits, SORT_MAX_BITS));
    q.digit_bits = ceil_div(q.bits, q.passes);
    q.tiles = int((e.T + SORT_TILE - 1) / SORT_TILE);
    const int es = e.dtype == CONV_F32 ? 4 : 2;
    q.V = 16 / es;
    while (q.V > 1 && e.D % q.V != 0) q.V /= 2;
    q.nv = e.D / q.V;
    q.wins = ceil_div(q.nv, SUM_THREADS);
    q.cols = ceil_div(q.nv, q.wins);
    // Chunks: long enough that few runs cross a boundary, short enough to fill the SMs.
    const int64_t groups = std::max<int64_t>(1, int64_t(d.sms) * 2048 / std::max(1, q.nv));
    q.chunk = int(std::min<int64_t>(256, std::max<int64_t>(16, (e.T + groups - 1) / groups)));
    q.chunks = int((e.T + q.chunk - 1) / q.chunk);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    for (int i = 0; i < 2; ++i) {
        q.off_keys[i] = take(size_t(e.T) * 4);
        q.off_pos[i] = take(size_t(e.T) * 4);
    }
    q.off_counts = take(size_t(q.tiles) * SORT_MAX_BINS * 4);
    q.off_totals = take(SORT_MAX_BINS * 4);
    q.off_part = take(size_t(q.chunks) * 2 * e.D * 4);
    q.bytes = o;
    return q;
}

// ---- lookup ----------------------------------------------------------------------------------
template <typename I> __device__ __forceinline__ int token_row(const I* idx, int64_t t, int V, int padding)
{
    const int64_t i = int64_t(idx[t]);
    return i >= 0 && i < V && i != padding ? int(i) : -1;
}

// A block takes `tokens` consecutive tokens, its threads their vectors in order.
template <typename T, typename I, int V>
__global__ void __launch_bounds__(256) embed_fwd_kernel(int64_t n, int rows, int padding, FastDivmod nv, int tokens,
                                                        float scale, const I* idx, const T* table, T* y)
{
    __shared__ int row[1024];
    const int64_t t0 = int64_t(blockIdx.x) * tokens;
    const int cnt = int(n - t0 < tokens ? n - t0 : tokens);
    tc::grid_dep_wait();
    for (int i = threadIdx.x; i < cnt; i += blockDim.x) row[i] = token_row(idx, t0 + i, rows, padding);
    __syncthreads();
    const int total = cnt * int(nv.d);
    const int64_t D = int64_t(nv.d) * V;
    for (int i = threadIdx.x; i < total; i += blockDim.x) {
        uint32_t t, c;
        nv.divmod(uint32_t(i), t, c);
        const int r = row[t];
        Vec<T, V> v;
        if (r >= 0) {
            v.load(table + int64_t(r) * D + c * V);
            float f[V];
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = v.get(k) * scale;
            v.set(f);
        } else {
            v.zero();
        }
        v.store(y + (t0 + t) * D + c * V);
    }
}

// ---- sort ------------------------------------------------------------------------------------
// Counts of each digit in each tile: counts[bin][tile].
template <typename I>
__global__ void __launch_bounds__(SORT_THREADS) sort_count(int n, int rows, int padding, const I* idx,
                                                           const uint32_t* keys, int shift, int bins, int tiles,
                                                           uint32_t* counts)
{
    __shared__ uint32_t hist[SORT_MAX_BINS];
    for (int i = threadIdx.x; i < bins; i += SORT_THREADS) hist[i] = 0;
    __syncthreads();
    tc::grid_dep_wait();
    const int base = int(blockIdx.x) * SORT_TILE;
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i) {
        const int t = base + i * SORT_THREADS + int(threadIdx.x);
        if (t < n) {
            uint32_t k;
            if (idx) {
                const int r = token_row(idx, t, rows, padding);
                k = r >= 0 ? uint32_t(r) : uint32_t(rows);
            } else {
                k = keys[t];
            }
            atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += SORT_THREADS) counts[size_t(i) * tiles + blockIdx.x] = hist[i];
}

// Inclusive scan over a block's threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sm)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) sm[w] = v;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < w; ++i) before += sm[i];
    __syncthreads();
    return v + before;
}

// Block b: the exclusive scan of bin b's counts over the tiles, and the bin's total.
__global__ void __launch_bounds__(SORT_THREADS) sort_scan(int tiles, uint32_t* counts, uint32_t* totals)
{
    __shared__ uint32_t sm[SORT_THREADS / 32];
    uint32_t* row = counts + size_t(blockIdx.x) * tiles;
    uint32_t carry = 0;
    __shared__ uint32_t last;
    tc::grid_dep_wait();
    for (int i0 = 0; i0 < tiles; i0 += SORT_THREADS) {
        const int i = i0 + int(threadIdx.x);
        const uint32_t v = i < tiles ? row[i] : 0u;
        const uint32_t s = block_scan(v, sm);
        if (i < tiles) row[i] = carry + s - v;
        if (threadIdx.x == SORT_THREADS - 1) last = s;
        __syncthreads();
        carry += last;
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Stable scatter by one digit.  Warp w holds the tile's tokens [w*256, (w+1)*256), 32 at a time
// in order; lanes with equal digits find each other by a match, the lowest one advances the
// warp's counter of the digit.
template <typename I>
__global__ void __launch_bounds__(SORT_THREADS) sort_scatter(int n, int rows, int padding, const I* idx,
                                                             const uint32_t* keys, const uint32_t* pos, int shift,
                                                             int bins, int tiles, const uint32_t* counts,
                                                             const uint32_t* totals, uint32_t* keys_out,
                                                             uint32_t* pos_out)
{
    constexpr int WARPS = SORT_THREADS / 32;
    __shared__ uint32_t cnt[WARPS][SORT_MAX_BINS];
    __shared__ uint32_t base[SORT_MAX_BINS];
    __shared__ uint32_t sm[WARPS];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < WARPS * SORT_MAX_BINS; i += SORT_THREADS) (&cnt[0][0])[i] = 0;
    tc::grid_dep_wait();
    uint32_t carry = 0;
    for (int i0 = 0; i0 < bins; i0 += SORT_THREADS) {  // first position of each bin
        const int i = i0 + int(threadIdx.x);
        const uint32_t v = i < bins ? totals[i] : 0u;
        const uint32_t s = block_scan(v, sm);
        if (i < bins) base[i] = carry + s - v + counts[size_t(i) * tiles + blockIdx.x];
        __shared__ uint32_t last;
        if (threadIdx.x == SORT_THREADS - 1) last = s;
        __syncthreads();
        carry += last;
        __syncthreads();
    }
    const int t0 = int(blockIdx.x) * SORT_TILE + w * (32 * SORT_ITEMS) + lane;
    uint32_t key[SORT_ITEMS], p[SORT_ITEMS], rank[SORT_ITEMS];
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i) {
        const int t = t0 + i * 32;
        key[i] = 0xFFFFFFFFu;
        p[i] = uint32_t(t);
        if (t < n) {
            if (idx) {
                const int r = token_row(idx, t, rows, padding);
                key[i] = r >= 0 ? uint32_t(r) : uint32_t(rows);
            } else {
                key[i] = keys[t];
                p[i] = pos[t];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i) {
        const bool in = t0 + i * 32 < n;
        const uint32_t dg = in ? (key[i] >> shift) & uint32_t(bins - 1) : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, dg);
        const uint32_t before = in ? cnt[w][dg] : 0u;
        __syncwarp();
        rank[i] = before + __popc(same & ((1u << lane) - 1u));
        if (in && (same & ((1u << lane) - 1u)) == 0) cnt[w][dg] = before + __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += SORT_THREADS) {  // the warps' counts to first positions
        uint32_t at = base[i];
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            const uint32_t c = cnt[k][i];
            cnt[k][i] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i)
        if (t0 + i * 32 < n) {
            const uint32_t at = cnt[w][(key[i] >> shift) & uint32_t(bins - 1)] + rank[i];
            keys_out[at] = key[i];
            pos_out[at] = p[i];
        }
}

// ---- sums ------------------------------------------------------------------------------------
// A group of `cols` threads sums the chunk's sorted tokens, each thread one vector of the row.
// part[chunk][0]: the sum of a run that began in an earlier chunk; part[chunk][1]: of a run that
// begins here and goes on in the next chunk.
template <typename T, int V>
__global__ void __launch_bounds__(SUM_THREADS) embed_sum(int n, int rows, int D, int cols, int wins, int chunk,
                                                         int chunks, float scale, const uint32_t* keys,
                                                         const uint32_t* pos, const T* dy, T* dtable, float* part)
{
    constexpr int U = 8;
    const int per = SUM_THREADS / cols, sub = int(threadIdx.x) / cols;
    const int win = int(blockIdx.x % wins);
    const int64_t ch = int64_t(blockIdx.x / wins) * per + sub;
    const int c = (win * cols + int(threadIdx.x) - sub * cols) * V;
    tc::grid_dep_wait();
    if (sub >= per || ch >= chunks || c >= D) return;
    const int i0 = int(ch) * chunk, i1 = min(n, i0 + chunk);
    const uint32_t prev = i0 > 0 ? keys[i0 - 1] : 0xFFFFFFFFu, next = i1 < n ? keys[i1] : 0xFFFFFFFFu;
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    uint32_t cur = keys[i0];
    bool head = cur == prev;  // the running run began before this chunk
    auto flush = [&](bool goes_on) {
        if (cur >= uint32_t(rows)) return;
        if (head || goes_on) {
            float* o = part + (ch * 2 + (head ? 0 : 1)) * D + c;
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = acc[k];
        } else {
            float f[V];
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = acc[k] * scale;
            Vec<T, V> v;
            v.set(f);
            v.store(dtable + int64_t(cur) * D + c);
        }
    };
    for (int i = i0; i < i1; i += U) {
        uint32_t k[U];
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            k[u] = i + u < i1 ? keys[i + u] : 0xFFFFFFFFu;
            if (k[u] < uint32_t(rows)) v[u].load(dy + int64_t(pos[i + u]) * D + c);
            else v[u].zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < i1) {
                if (k[u] != cur) {
                    flush(false);
                    cur = k[u];
                    head = false;
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < V; ++j) acc[j] += v[u].get(j);
            }
    }
    flush(cur == next);
}

// Rows whose tokens cross chunks: block `ch` looks whether a run begins in chunk ch and goes on;
// if so it adds the run's partials: lanes take chunks round robin, then the lanes are added in
// order.
template <typename T, int V>
__global__ void __launch_bounds__(FIX_THREADS) embed_fix(int n, int rows, int D, int cols, int wins, int chunk,
                                                         int chunks, float scale, const uint32_t* keys, T* dtable,
                                                         const float* part)
{
    __shared__ float sm[FIX_THREADS * V];
    const int win = int(blockIdx.x % wins), ch = int(blockIdx.x / wins);
    const int lanes = FIX_THREADS / cols, lane = int(threadIdx.x) / cols, col = int(threadIdx.x) - lane * cols;
    const int c = (win * cols + col) * V;
    tc::grid_dep_wait();
    const int i0 = ch * chunk, i1 = min(n, i0 + chunk);
    if (i1 >= n) return;
    const uint32_t key = keys[i1 - 1];
    if (key >= uint32_t(rows) || keys[i1] != key) return;
    if (i0 > 0 && keys[i0 - 1] == key) return;  // began earlier
    // the last chunk that the run reaches, by bisection over the chunks' first keys
    int lo = ch + 1, hi = chunks - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (keys[mid * chunk] == key) lo = mid;
        else hi = mid - 1;
    }
    const int cnt = lo - ch;  // further chunks
    float acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = 0.f;
    if (lane < lanes && c < D)
#pragma unroll 4
        for (int j = lane; j <= cnt; j += lanes) {
            const float* s = part + (int64_t(ch + j) * 2 + (j == 0 ? 1 : 0)) * D + c;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += s[k];
        }
    if (lane < lanes)
#pragma unroll
        for (int k = 0; k < V; ++k) sm[(lane * cols + col) * V + k] = acc[k];
    __syncthreads();
    if (lane == 0 && c < D) {
        for (int l = 1; l < lanes; ++l)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] += sm[(l * cols + col) * V + k];
        Vec<T, V> v;
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] *= scale;
        v.set(acc);
        v.store(dtable + int64_t(key) * D + c);
    }
}

template <typename T, typename I>
cudaError_t fwd_t(const conv_embed_desc_t& e, const DevInfo& d, const I* idx, const T* table, T* y, cudaStream_t s)
{
    const int es = sizeof(T);
    int V = 16 / es;
    while (V > 1 && e.D % V != 0) V /= 2;
    const int nv = e.D / V;
    // about four vectors a thread, fewer when that leaves SMs without a block
    int64_t tokens = std::max(1, std::min(1024, 1024 / nv));
    tokens = std::max<int64_t>(1, std::min<int64_t>(tokens, (e.T + 2 * d.sms - 1) / (2 * d.sms)));
    const dim3 grid(unsigned((e.T + tokens - 1) / tokens));
    const FastDivmod dm{uint32_t(nv)};
    cudaError_t r = cudaSuccess;
#define EMB_CALL(V_)                                                                                             \
    r = launch_ex(embed_fwd_kernel<T, I, V_>, grid, dim3(256), 0, s, 1, true, e.T, e.V, e.padding_idx, dm,       \
                  int(tokens), e.scale, idx, table, y)
    if (V == 8) {
        if constexpr (sizeof(T) == 2) EMB_CALL(8);
    } else if (V == 4) EMB_CALL(4);
    else if (V == 2) EMB_CALL(2);
    else EMB_CALL(1);
#undef EMB_CALL
    return r != cudaSuccess ? r : cudaGetLastError();
}

template <typename I>
cudaError_t sort_tokens(const conv_embed_desc_t& e, const EmbedPlan& q, const I* idx, unsigned char* ws, int& where,
                        cudaStream_t s)
{
    const int n = int(e.T), bins = 1 << q.digit_bits;
    uint32_t* counts = reinterpret_cast<uint32_t*>(ws + q.off_counts);
    uint32_t* totals = reinterpret_cast<uint32_t*>(ws + q.off_totals);
    for (int pass = 0; pass < q.passes; ++pass) {
        const I* in = pass == 0 ? idx : nullptr;
        const uint32_t* kin = reinterpret_cast<const uint32_t*>(ws + q.off_keys[(pass + 1) & 1]);
        const uint32_t* pin = reinterpret_cast<const uint32_t*>(ws + q.off_pos[(pass + 1) & 1]);
        uint32_t* kout = reinterpret_cast<uint32_t*>(ws + q.off_keys[pass & 1]);
        uint32_t* pout = reinterpret_cast<uint32_t*>(ws + q.off_pos[pass & 1]);
        const int shift = pass * q.digit_bits;
        cudaError_t r = launch_ex(sort_count<I>, dim3(q.tiles), dim3(SORT_THREADS), 0, s, 1, true, n, e.V,
                                  e.padding_idx, in, kin, shift, bins, q.tiles, counts);
        if (r == cudaSuccess)
            r = launch_ex(sort_scan, dim3(bins), dim3(SORT_THREADS), 0, s, 1, true, q.tiles, counts, totals);
        if (r == cudaSuccess)
            r = launch_ex(sort_scatter<I>, dim3(q.tiles), dim3(SORT_THREADS), 0, s, 1, true, n, e.V, e.padding_idx, in,
                          kin, pin, shift, bins, q.tiles, static_cast<const uint32_t*>(counts),
                          static_cast<const uint32_t*>(totals), kout, pout);
        if (r != cudaSuccess) return r;
        where = pass & 1;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t sum_t(const conv_embed_desc_t& e, const EmbedPlan& q, const uint32_t* keys, const uint32_t* pos,
                  const T* dy, T* dtable, float* part, cudaStream_t s)
{
    const int n = int(e.T), per = SUM_THREADS / q.cols;
    const dim3 sgrid(unsigned(ceil_div(q.chunks, per)) * unsigned(q.wins)), fgrid(unsigned(q.chunks) * unsigned(q.wins));
    cudaError_t r = cudaSuccess;
    const float* cpart = part;
#define EMB_CALL(V_)                                                                                             \
    do {                                                                                                         \
        r = launch_ex(embed_sum<T, V_>, sgrid, dim3(SUM_THREADS), 0, s, 1, true, n, e.V, e.D, q.cols, q.wins,    \
                      q.chunk, q.chunks, e.scale, keys, pos, dy, dtable, part);                                  \
        if (r == cudaSuccess)                                                                                    \
            r = launch_ex(embed_fix<T, V_>, fgrid, dim3(FIX_THREADS), 0, s, 1, true, n, e.V, e.D, q.cols, q.wins,\
                          q.chunk, q.chunks, e.scale, keys, dtable, cpart);                                      \
    } while (0)
    if (q.V == 8) {
        if constexpr (sizeof(T) == 2) EMB_CALL(8);
    } else if (q.V == 4) EMB_CALL(4);
    else if (q.V == 2) EMB_CALL(2);
    else EMB_CALL(1);
#undef EMB_CALL
    return r != cudaSuccess ? r : cudaGetLastError();
}

}  // namespace

cudaError_t run_embed_fwd(const conv_embed_desc_t& e, const DevInfo& d, const void* idx, const void* table, void* y,
                          cudaStream_t s)
{
    using H = __nv_bfloat16;
    if (e.index_dtype == CONV_INDEX_I32)
        return e.dtype == CONV_F32 ? fwd_t(e, d, (const int32_t*)idx, (const float*)table, (float*)y, s)
                                   : fwd_t(e, d, (const int32_t*)idx, (const H*)table, (H*)y, s);
    return e.dtype == CONV_F32 ? fwd_t(e, d, (const int64_t*)idx, (const float*)table, (float*)y, s)
                               : fwd_t(e, d, (const int64_t*)idx, (const H*)table, (H*)y, s);
}

size_t embed_bwd_workspace(const conv_embed_desc_t& e, const DevInfo& d)
{
    return e.T == 0 ? 0 : embed_plan(e, d).bytes;
}

cudaError_t run_embed_bwd(const conv_embed_desc_t& e, const DevInfo& d, const void* idx, const void* dy, void* dtable,
                          void* ws_, cudaStream_t s)
{
    using H = __nv_bfloat16;
    unsigned char* ws = static_cast<unsigned char*>(ws_);
    cudaError_t r = cudaMemsetAsync(dtable, 0, size_t(e.V) * e.D * (e.dtype == CONV_F32 ? 4 : 2), s);
    if (r != cudaSuccess || e.T == 0) return r;
    const EmbedPlan q = embed_plan(e, d);
    int where = 0;
    r = e.index_dtype == CONV_INDEX_I32 ? sort_tokens(e, q, (const int32_t*)idx, ws, where, s)
                                        : sort_tokens(e, q, (const int64_t*)idx, ws, where, s);
    if (r != cudaSuccess) return r;
    const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + q.off_keys[where]);
    const uint32_t* pos = reinterpret_cast<const uint32_t*>(ws + q.off_pos[where]);
    float* part = reinterpret_cast<float*>(ws + q.off_part);
    return e.dtype == CONV_F32 ? sum_t(e, q, keys, pos, (const float*)dy, (float*)dtable, part, s)
                               : sum_t(e, q, keys, pos, (const H*)dy, (H*)dtable, part, s);
}

}  // namespace igc
