// kernels_embed.cu -- embedding lookup with scaling and its gradient:
//   y[t,:] = scale * table[idx[t],:],    dtable[v,:] = scale * sum_{t: idx[t] = v} dy[t,:].
//
// The lookup moves T*D values in and out with one multiply each: bound by memory.
//
// The gradient is a sum per row over the tokens that name it, in one of three ways:
//
// Few tokens: one launch, in which a block a token finds the others of its row.
//
// A table of few rows: half a warp keeps the sums of the whole table, a window of 32 columns, in its
// own part of shared memory (two columns a lane) and adds a contiguous share of the tokens to it,
// whose values are copied ahead as they lie.  The copies are added up at the end.
//
// Else the tokens are sorted by row (least significant digit first, a stable counting sort a
// digit), so a row's tokens are one run of the sorted order in ascending t: dy is read once, row
// by row, and no atomic is needed.  Up to 64 Ki tokens are sorted by one thread-block cluster in
// its shared memory, while the other blocks of the launch fill dtable with zeros.  The sorted
// order is cut into chunks; a run is summed by the group of the chunk it begins in, if it ends
// by the end of the next one.  A longer run -- a row that holds a large share of the tokens --
// leaves an fp32 partial sum in each chunk, which a last kernel adds in chunk order.
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
constexpr int SUM_THREADS = 256, SUM_BLOCKS_SM = 3;
constexpr int CHUNK_MAX = 256;                             // sorted tokens a group sums
constexpr int FIX_THREADS = 1024;
constexpr int FIX_MIN = 16, FIX_MAX = 256;                 // chunks a block of the last kernel looks at
constexpr int CS_THREADS = 1024, CS_ITEMS = 8;             // sort by one cluster: a block's threads, tokens a thread
constexpr int CS_TOKENS = CS_THREADS * CS_ITEMS;
constexpr int CS_WARPS = CS_THREADS / 32;
constexpr int TAB_COLS = 32;                               // columns of a table window: two a lane of half a warp
constexpr int TAB_STEP = 16, TAB_STAGES = 4;               // tokens copied at a time, copies under way and in use
constexpr int TAB_SMEM = 225 * 1024;
constexpr int TAB_GROUP = 4;                               // tokens added at a time
constexpr int TAB_TOKENS = 512 * TAB_GROUP;                // of a half warp's share at most: no chain of sums beyond 512
constexpr int FEW_THREADS = 256, FEW_WARPS = FEW_THREADS / 32;
constexpr int FEW_TOKENS = 512, FEW_BLOCKS = 4096, FEW_ROWS = 1024;              // tokens at most; rows a filling block takes at most
constexpr int TAB_MAX_UNITS = 32, TAB_MIN_UNITS = 4;       // half warps with a table each, a block (and SM)

struct EmbedPlan {
    bool few;             // few tokens: one launch
    bool table;           // sums of the whole table in shared memory
    int units, blocks;    // copies a block; blocks a window of columns (few: that fill)
    int smem;
    int cluster;          // blocks of the one-cluster sort, 0: sort by kernels
    int log_items;        // its tokens a thread: 2^log_items
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
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) / 256 * 256;
        return at;
    };
    const int es = e.dtype == CONV_F32 ? 4 : 2;
    q.V = 16 / es;
    while (q.V > 1 && e.D % q.V != 0) q.V /= 2;
    q.nv = e.D / q.V;
    // Few tokens: one launch beside three (us): 300 tokens, 696 x 16 fp32 6 / 17, 4410 x 1088 bf16 10 / 18;
    // 512 tokens, 60187 x 40 bf16 10 / 19, 20000 x 1024 fp32 (82 MB to write) 25 / 26.  Every block reads
    // all names: at 1024 tokens 20000 x 1024 takes 28 us either way.
    if (e.T <= FEW_TOKENS) {
        q.wins = ceil_div(q.nv, 32);
        q.cols = ceil_div(q.nv, q.wins);
        q.blocks = int(std::max<int64_t>(ceil_div(e.V, FEW_ROWS), std::min<int64_t>(e.V, 2 * d.sms)));
        if (e.T * q.wins <= FEW_BLOCKS) {
            q.few = true;
            return q;
        }
    }
    // Whole-table sums where the tokens outnumber by far the rows that every copy has to add up,
    // and an SM holds a few copies, whose reads ahead keep it busy.  Measured (Zipf tokens, us, whole
    // table against sort): 1540096 x 32 values, 128 rows, fp32 45 / 83; 60000 x 250 x 32 16 / 28;
    // 30000 x 16 x 1024 40 / 45; but 126925 x 102 x 504 98 / 87 (every window walks all tokens).
    // Shares of TAB_TOKENS take several waves of blocks for many tokens, each of which zeroes its copies
    // and adds them up: 4000000 x 128 x 32 fp32 106 / 214, 3000000 x 380 x 32 bf16 133 / 139 and 1000000
    // x 100 x 128 fp32 128 / 156, but with several windows of narrow values or few copies 1000000 x 200 x
    // 128 bf16 122 / 90, 1000000 x 380 x 128 bf16 176 / 93 and 19300 x 300 x 2500 fp32 104 / 78.
    const int64_t unit = (int64_t(e.V) + 1) * TAB_COLS * 4 +
                         TAB_STAGES * TAB_STEP * (TAB_COLS * (e.dtype == CONV_F32 ? 4 : 2) +
                                                  (e.index_dtype == CONV_INDEX_I32 ? 4 : 8));
    q.wins = ceil_div(e.D, TAB_COLS);
    q.units = int(std::min<int64_t>(TAB_MAX_UNITS, TAB_SMEM / unit / 2 * 2));
    const int64_t most = std::max(1, d.sms / q.wins), wave = std::max<int64_t>(1, most * q.units * TAB_TOKENS);
    const int64_t waves = (e.T + wave - 1) / wave;
    q.table = q.units >= TAB_MIN_UNITS && e.T >= int64_t(64) * e.V && e.T >= 8192 &&
              (e.D <= 256 || e.T <= int64_t(kMaxCluster) * CS_TOKENS) &&
              (waves == 1 || q.wins == 1 || (e.dtype == CONV_F32 && q.units >= 8));
    if (q.table) {
        q.smem = q.units * int(unit);
        q.blocks = int(waves > 1 ? waves * most
                                 : std::min<int64_t>(most, (e.T + q.units * 4 * TAB_STEP - 1) / (q.units * 4 * TAB_STEP)));
        q.off_part = take(size_t(q.blocks) * e.V * e.D * 4);
        q.bytes = o;
        return q;
    }
    while ((int64_t(1) << q.bits) <= e.V) ++q.bits;  // keys 0 .. V (V: no row)
    q.passes = std::max(1, ceil_div(q.bits, SORT_MAX_BITS));
    q.digit_bits = ceil_div(q.bits, q.passes);
    if (e.T <= int64_t(kMaxCluster) * CS_TOKENS) {  // as many blocks as have a token a thread
        q.cluster = 1;
        while (q.cluster < kMaxCluster && e.T > int64_t(q.cluster) * CS_THREADS) q.cluster *= 2;
        while (e.T > (int64_t(q.cluster) * CS_THREADS << q.log_items)) ++q.log_items;
    }
    q.tiles = int((e.T + SORT_TILE - 1) / SORT_TILE);
    const int each = ceil_div(q.nv, q.V * es >= 16 ? 1 : q.V * es == 8 ? 2 : 4);  // a thread's vectors: sum_vectors()
    q.wins = ceil_div(each, SUM_THREADS);
    q.cols = ceil_div(each, q.wins);
    // Chunks: long, so that few runs are cut, while the groups fill the SMs once; a run over two of
    // them is one chain of additions (512 and 1023 of equal values lose up to 8e-6 and 1.5e-5).
    const int64_t groups = std::max<int64_t>(1, int64_t(d.sms) * SUM_BLOCKS_SM * (SUM_THREADS / q.cols) / q.wins);
    q.chunk = int(std::min<int64_t>(CHUNK_MAX, std::max<int64_t>(16, (e.T + groups - 1) / groups)));
    q.chunks = int((e.T + q.chunk - 1) / q.chunk);
    for (int i = 0; i < (q.cluster ? 1 : 2); ++i) {
        q.off_keys[i] = take(size_t(e.T) * 4);
        q.off_pos[i] = take(size_t(e.T) * 4);
    }
    if (!q.cluster) {
        q.off_counts = take(size_t(q.tiles) * SORT_MAX_BINS * 4);
        q.off_totals = take(SORT_MAX_BINS * 4);
    }
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

// A block takes `tokens` consecutive tokens, its threads their vectors in order.  1540096 tokens,
// 128 x 32 bf16: 17 us, 6.1 TB/s of names in and values out, 91% of the measured copy's; 752
// tokens: 4 us, a launch.  Bound by memory (the table's rows come from L1 and L2).
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

// ---- few tokens --------------------------------------------------------------------------------
// One launch.  The first `fill` blocks write zeros to the rows that no token names.  Block (token,
// window) after those: looks for the other tokens of its token's row; the row's first token sums them
// all, groups of `cols` threads taking equal parts of them in order, the parts added in order.  6 to 12
// us for up to 512 tokens: a launch, the names, and a few rounds of reads.
template <typename T, typename I, int V>
__global__ void __launch_bounds__(FEW_THREADS) embed_few(int n, int rows, int padding, int D, int cols, int wins,
                                                         int fill, float scale, const I* idx, const T* dy, T* dtable)
{
    constexpr int U = 4;
    __shared__ __align__(16) float sm[FEW_THREADS * V];
    __shared__ int found[FEW_TOKENS], list[FEW_TOKENS], counts[FEW_WARPS];
    const int w = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
    tc::grid_dep_wait();
    if (int(blockIdx.x) < fill) {
        unsigned char* named = reinterpret_cast<unsigned char*>(sm);
        static_assert(FEW_ROWS <= int(sizeof(float)) * FEW_THREADS, "a byte a row");
        const int64_t f = blockIdx.x;
        const int r0 = int(f * rows / fill), cnt = int((f + 1) * rows / fill) - r0;
        for (int r = threadIdx.x; r < cnt; r += FEW_THREADS) named[r] = 0;
        __syncthreads();
        for (int t = threadIdx.x; t < n; t += FEW_THREADS) {
            const int r = token_row(idx, t, rows, padding) - r0;
            if (r >= 0 && r < cnt) named[r] = 1;
        }
        __syncthreads();
        Vec<T, V> zero;
        zero.zero();
        for (int r = w; r < cnt; r += FEW_WARPS)
            if (!named[r])
                for (int c = lane * V; c < D; c += 32 * V) zero.store(dtable + int64_t(r0 + r) * D + c);
        return;
    }
    const int t = (int(blockIdx.x) - fill) / wins, win = int(blockIdx.x) - fill - t * wins;
    const int row = token_row(idx, t, rows, padding);
    if (row < 0) return;
    // the row's tokens: each warp those of its share, then all in order
    const int share = (n + FEW_THREADS - 1) / FEW_THREADS * 32, t0 = w * share;
    int mine = 0;
    for (int i = t0; i < min(n, t0 + share); i += 32) {
        const bool is = i + lane < n && token_row(idx, i + lane, rows, padding) == row;
        const uint32_t m = __ballot_sync(0xFFFFFFFFu, is);
        if (is) found[t0 + mine + __popc(m & ((1u << lane) - 1))] = i + lane;
        mine += __popc(m);
    }
    if (lane == 0) counts[w] = mine;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < FEW_WARPS; ++i) {
        before += i < w ? counts[i] : 0;
        total += counts[i];
    }
    for (int i = lane; i < mine; i += 32) list[before + i] = found[t0 + i];
    __syncthreads();
    if (list[0] != t) return;  // an earlier token's block sums the row
    const int groups = FEW_THREADS / cols, g = int(threadIdx.x) / cols, col = int(threadIdx.x) - g * cols;
    const int c = (win * cols + col) * V;
    if (g < groups) {
        float acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        const int i1 = total * (g + 1) / groups;
        if (c < D)
            for (int i = total * g / groups; i < i1; i += U) {
                Vec<T, V> v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (i + u < i1) v[u].load(dy + int64_t(list[i + u]) * D + c);
                    else v[u].zero();
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] += v[u].get(k);
            }
#pragma unroll
        for (int k = 0; k < V; ++k) sm[k * FEW_THREADS + threadIdx.x] = acc[k];
    }
    __syncthreads();
    if (g == 0 && c < D) {
        float f[V];
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = sm[k * FEW_THREADS + col];
        for (int j = 1; j < groups; ++j)
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] += sm[k * FEW_THREADS + j * cols + col];
        Vec<T, V> v;
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] *= scale;
        v.set(f);
        v.store(dtable + int64_t(row) * D + c);
    }
}

// ---- sort ------------------------------------------------------------------------------------
// Three launches a digit for more tokens than a cluster holds: 887914 tokens, 13 bits in two digits:
// 41 us, each pass reading and writing keys and places once (count 7, scan 4, scatter 10 us).
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
    tc::grid_dep_launch();
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

__device__ __forceinline__ void st_dsmem(uint32_t addr, uint2 v)
{
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

// Inclusive scan over a block's threads (up to 32 warps).
__device__ __forceinline__ uint32_t warp_scan(uint32_t v)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if ((threadIdx.x & 31) >= unsigned(o)) v += u;
    }
    return v;
}
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sm)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    v = warp_scan(v);
    if (lane == 31) sm[w] = v;
    __syncthreads();
    const uint32_t t = warp_scan(lane < int(blockDim.x >> 5) ? sm[lane] : 0u);
    const uint32_t before = __shfl_sync(0xFFFFFFFFu, t, max(w, 1) - 1);
    __syncthreads();
    return w ? v + before : v;
}

// Block b: the exclusive scan of bin b's counts over the tiles, and the bin's total.
__global__ void __launch_bounds__(SORT_THREADS) sort_scan(int tiles, uint32_t* counts, uint32_t* totals)
{
    __shared__ uint32_t sm[SORT_THREADS / 32];
    uint32_t* row = counts + size_t(blockIdx.x) * tiles;
    uint32_t carry = 0;
    __shared__ uint32_t last;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
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
// warp's counter of the digit.  The tile is put in the digit's order in shared memory first, so
// that what goes to memory are runs of neighbours.
template <typename I>
__global__ void __launch_bounds__(SORT_THREADS) sort_scatter(int n, int rows, int padding, const I* idx,
                                                             const uint32_t* keys, const uint32_t* pos, int shift,
                                                             int bins, int tiles, const uint32_t* counts,
                                                             const uint32_t* totals, uint32_t* keys_out,
                                                             uint32_t* pos_out)
{
    constexpr int WARPS = SORT_THREADS / 32;
    __shared__ uint16_t cnt[WARPS][SORT_MAX_BINS];  // the warps' counts, then first places in the tile
    __shared__ uint32_t base[SORT_MAX_BINS];        // first place of the tile's tokens of a digit, less that in the tile
    __shared__ uint2 stage[SORT_TILE];
    __shared__ uint32_t sm[WARPS], last[2];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < WARPS * SORT_MAX_BINS / 2; i += SORT_THREADS)
        reinterpret_cast<uint32_t*>(&cnt[0][0])[i] = 0;
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    const int t0 = int(blockIdx.x) * SORT_TILE + w * (32 * SORT_ITEMS) + lane;
    const int here = min(SORT_TILE, n - int(blockIdx.x) * SORT_TILE);
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
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i) {
        const bool in = t0 + i * 32 < n;
        const uint32_t dg = in ? (key[i] >> shift) & uint32_t(bins - 1) : 0xFFFFFFFFu;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, dg), below = same & ((1u << lane) - 1u);
        const uint32_t before = in ? cnt[w][dg] : 0u;
        __syncwarp();
        rank[i] = before + __popc(below);
        if (in && below == 0) cnt[w][dg] = uint16_t(before + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    uint32_t carry = 0, local = 0;
    for (int i0 = 0; i0 < bins; i0 += SORT_THREADS) {  // first place of each digit, in all and in the tile
        const int i = i0 + int(threadIdx.x);
        uint32_t mine = 0;
        if (i < bins)
#pragma unroll
            for (int k = 0; k < WARPS; ++k) {
                const uint32_t c = cnt[k][i];
                cnt[k][i] = uint16_t(mine);
                mine += c;
            }
        const uint32_t v = i < bins ? totals[i] : 0u;
        const uint32_t s = block_scan(v, sm), m = block_scan(mine, sm);
        const uint32_t at = local + m - mine;
        if (i < bins) {
            base[i] = carry + s - v + counts[size_t(i) * tiles + blockIdx.x] - at;
#pragma unroll
            for (int k = 0; k < WARPS; ++k) cnt[k][i] = uint16_t(cnt[k][i] + at);
        }
        if (threadIdx.x == SORT_THREADS - 1) {
            last[0] = s;
            last[1] = m;
        }
        __syncthreads();
        carry += last[0];
        local += last[1];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i)
        if (t0 + i * 32 < n) stage[cnt[w][(key[i] >> shift) & uint32_t(bins - 1)] + rank[i]] = make_uint2(key[i], p[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < SORT_ITEMS; ++i) {
        const int s = i * SORT_THREADS + int(threadIdx.x);
        if (s < here) {
            const uint2 e = stage[s];
            const uint32_t at = base[(e.x >> shift) & uint32_t(bins - 1)] + uint32_t(s);
            keys_out[at] = e.x;
            pos_out[at] = e.y;
        }
    }
}

// The whole sort by one cluster of S blocks (blockIdx.x < S), which hold the tokens in order,
// up to CS_TOKENS a block; the other blocks write zeros to dtable meanwhile.  A pass ranks the
// tokens of a digit as sort_scatter does (16 bits hold a warp's counts), the blocks read each
// other's counts of each digit, and the tokens, put in the digit's order in the block first, go in
// runs to their places in the next order, in whichever block those lie.  16384 tokens, 50021 rows of
// 1024 bf16: 18 us, what the 102 MB of zeros take; the gradient as a whole takes 24 us less than with
// three launches a digit (65536 tokens, 50021 x 256: 7 us less; 4096 tokens, 1000 x 128 fp32: 6).
template <typename I>
__global__ void __launch_bounds__(CS_THREADS, 1)
sort_cluster(int n, int rows, int padding, int S, int log_items, int passes, int digit_bits, const I* idx,
             uint32_t* keys_out, uint32_t* pos_out, uint4* fill, int64_t fill_vecs, unsigned char* fill_tail,
             int fill_rest)
{
    extern __shared__ __align__(16) uint2 cs[];
    if (int(blockIdx.x) >= S) {
        const int64_t nb = int64_t(gridDim.x) - S, t = (int64_t(blockIdx.x) - S) * CS_THREADS + threadIdx.x;
        tc::grid_dep_wait();
        tc::grid_dep_launch();
#pragma unroll 4
        for (int64_t i = t; i < fill_vecs; i += nb * CS_THREADS) fill[i] = make_uint4(0, 0, 0, 0);
        if (t < fill_rest) fill_tail[t] = 0;
        return;
    }
    const int bins = 1 << digit_bits;
    uint2* stage = cs;                                           // the block's tokens (key, position) by digit
    uint2* next = cs + CS_TOKENS;                                // its part of the next order, written by all blocks
    uint32_t* hist = reinterpret_cast<uint32_t*>(next + CS_TOKENS);  // bins: the block's counts, read by the others
    uint32_t* base = hist + SORT_MAX_BINS;                       // bins: first place, less that in the block
    uint32_t* sm = base + SORT_MAX_BINS;                         // CS_WARPS
    uint16_t* cnt = reinterpret_cast<uint16_t*>(sm + CS_WARPS);  // warps x bins
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = S > 1 ? int(tc::cluster_rank()) : 0;
    const int log_cap = log_items + 10;  // tokens a block: 2^log_cap
    static_assert(CS_THREADS == 1 << 10, "a block's tokens");
    const int here = max(0, min(1 << log_cap, n - (rank << log_cap)));
    const int first = (w << (5 + log_items)) + lane;
    const int items = 1 << log_items;
    uint2 e[CS_ITEMS];  // key, position
    uint32_t rk[CS_ITEMS];
    tc::grid_dep_wait();
    tc::grid_dep_launch();
#pragma unroll
    for (int i = 0; i < CS_ITEMS; ++i) {
        const int t = first + i * 32;
        e[i] = make_uint2(0xFFFFFFFFu, uint32_t((rank << log_cap) + t));
        if (i < items && t < here) {
            const int r = token_row(idx, int64_t(e[i].y), rows, padding);
            e[i].x = r >= 0 ? uint32_t(r) : uint32_t(rows);
        }
    }
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * digit_bits;
        const bool last = pass + 1 == passes;
        for (int i = threadIdx.x; i < CS_WARPS * bins / 2; i += CS_THREADS) reinterpret_cast<uint32_t*>(cnt)[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CS_ITEMS; ++i) {
            if (i >= items) break;
            const bool in = first + i * 32 < here;
            const uint32_t dg = in ? (e[i].x >> shift) & uint32_t(bins - 1) : 0xFFFFFFFFu;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, dg), below = same & ((1u << lane) - 1u);
            const uint32_t before = in ? cnt[w * bins + dg] : 0u;
            __syncwarp();
            rk[i] = before + __popc(below);
            if (in && below == 0) cnt[w * bins + dg] = uint16_t(before + __popc(same));
            __syncwarp();
        }
        __syncthreads();
        // a digit's counts of the warps, and its total
        uint32_t total = 0;
        if (int(threadIdx.x) < bins) {
#pragma unroll 8
            for (int k = 0; k < CS_WARPS; ++k) {
                const uint32_t c = cnt[k * bins + threadIdx.x];
                cnt[k * bins + threadIdx.x] = uint16_t(total);
                total += c;
            }
            hist[threadIdx.x] = total;
        }
        uint32_t all = total, before = 0;
        if (S > 1) {
            __syncwarp();
            tc::cluster_sync();
            if (int(threadIdx.x) < bins) {
                uint32_t v[kMaxCluster];
                all = 0;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < S)
                        v[r] = __float_as_uint(
                            tc::ld_dsmem_f32(tc::dsmem_addr(tc::smem_u32(hist + threadIdx.x), uint32_t(r))));
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < S) {
                        all += v[r];
                        before += r < rank ? v[r] : 0u;
                    }
            }
        }
        // first place of each digit: in all (the digits below it, then the blocks below this one),
        // and in the block
        const uint32_t up = block_scan(all, sm), here_up = block_scan(total, sm);
        if (int(threadIdx.x) < bins) {
            const uint32_t at = here_up - total;
            base[threadIdx.x] = up - all + before - at;
#pragma unroll 8
            for (int k = 0; k < CS_WARPS; ++k) cnt[k * bins + threadIdx.x] += uint16_t(at);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < CS_ITEMS; ++i)
            if (i < items && first + i * 32 < here)
                stage[cnt[w * bins + ((e[i].x >> shift) & uint32_t(bins - 1))] + rk[i]] = e[i];
        __syncthreads();
        for (int s = threadIdx.x; s < here; s += CS_THREADS) {
            const uint2 v = stage[s];
            const uint32_t at = base[(v.x >> shift) & uint32_t(bins - 1)] + uint32_t(s);
            if (last) {
                keys_out[at] = v.x;
                pos_out[at] = v.y;
            } else if (S == 1) {
                next[at] = v;
            } else {
                st_dsmem(tc::dsmem_addr(tc::smem_u32(next + (at & ((1u << log_cap) - 1u))), at >> log_cap), v);
            }
        }
        if (last) break;
        if (S > 1) {
            __syncwarp();
            tc::cluster_sync();
        } else {
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < CS_ITEMS; ++i)
            if (i < items && first + i * 32 < here) e[i] = next[first + i * 32];
    }
    if (S > 1) {  // no block leaves while another still reads its counts
        __syncwarp();
        tc::cluster_sync();
    }
}

// ---- whole-table sums ------------------------------------------------------------------------
// Block (range, window), unit u (half a warp): its own table of rows + 1 rows (the last one takes
// the tokens that name none) and a ring of TAB_STAGES tiles of TAB_STEP tokens.  Four tokens are
// added at a time: their table rows are read together; where a row comes again among the four, its
// values are added to each other first, and the last of them stores the row.  A row thus gets one
// addition in four tokens at most where it holds most of them, and a unit's share is at most
// TAB_TOKENS: no chain of additions is longer than 512, which equal values keep within 8e-6 of their
// sum (a chain of 4825, which one block a window had, lost 7e-5).  Eight tokens at a time are bound by
// the comparisons: 1540096 tokens, 128 x 32 bf16 53 us against 47.
// 1540096 tokens, 128 x 32 fp32: 41 us with the copies' sum, 4.9 TB/s, 74% of the measured copy's.
// Bound by shared memory's latency: a step's sums wait for the step's before.
template <int BYTES> __device__ __forceinline__ void tab_copy(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

template <typename T, typename I, int V>
__global__ void __launch_bounds__(TAB_MAX_UNITS * 16, 1)
embed_table(int n, int rows, int padding, int D, int blocks, int units, const I* idx, const T* dy, float* part)
{
    constexpr int COPIES = TAB_COLS / V, TILE = TAB_STEP * TAB_COLS;  // copies a token; values a tile
    extern __shared__ __align__(16) unsigned char dynt[];
    const int lane = threadIdx.x & 15, u = threadIdx.x >> 4;
    float* tab = reinterpret_cast<float*>(dynt);            // units x (rows + 1) x TAB_COLS
    const int size = (rows + 1) * TAB_COLS;
    float2* my = reinterpret_cast<float2*>(tab + size_t(u) * size) + lane;
    T* tiles = reinterpret_cast<T*>(tab + size_t(units) * size);
    T* tile = tiles + u * (TAB_STAGES * TILE);
    I* names = reinterpret_cast<I*>(tiles + units * (TAB_STAGES * TILE)) + u * (TAB_STAGES * TAB_STEP);
    const int range = int(blockIdx.x) % blocks, c0 = int(blockIdx.x) / blocks * TAB_COLS;
    const int width = min(TAB_COLS, D - c0);
    const int64_t parts = int64_t(blocks) * units, at = int64_t(range) * units + u;
    const int t0 = int(int64_t(n) * at / parts), t1 = int(int64_t(n) * (at + 1) / parts);
    // (both halves of a warp walk as many steps)
    const int other = __shfl_xor_sync(0xFFFFFFFFu, t1 - t0, 16);
    const int steps = (max(t1 - t0, other) + TAB_STEP - 1) / TAB_STEP;
    for (int i = lane * 4; i < size; i += 64)
        *reinterpret_cast<float4*>(tab + size_t(u) * size + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = lane; i < TAB_STAGES * TILE; i += 16) Elem<T>::st(tile + i, 0.f);
    __syncwarp();
    // This lane's part of a step's copies: one in AT_ONCE tokens where a token is less than 16
    // copies, else a sixteenth of every token.
    constexpr int AT_ONCE = COPIES <= 16 ? 16 / COPIES : 1, EACH = COPIES <= 16 ? 1 : COPIES / 16;
    const int tok0 = COPIES <= 16 ? lane / COPIES : 0, col0 = lane % (COPIES <= 16 ? COPIES : 16) * V;
    const T* src0 = dy + int64_t(t0 + tok0) * D + c0 + col0;
    auto load = [&](int step, int stage) {  // as far as there is such a step
        const int left = t1 - t0 - step * TAB_STEP;
        if (lane < left)
            tab_copy<int(sizeof(I))>(tc::smem_u32(names + stage * TAB_STEP + lane), idx + t0 + step * TAB_STEP + lane);
        const T* src = src0;
        T* dst = tile + stage * TILE + tok0 * TAB_COLS + col0;
        src0 += int64_t(TAB_STEP) * D;
#pragma unroll
        for (int i = 0; i < TAB_STEP; i += AT_ONCE, src += int64_t(AT_ONCE) * D, dst += AT_ONCE * TAB_COLS)
#pragma unroll
            for (int k = 0; k < EACH; ++k)
                if (i + tok0 < left && col0 + 16 * k < width) {
                    if constexpr (sizeof(T) * V >= 4) tab_copy<int(sizeof(T)) * V>(tc::smem_u32(dst + 16 * k), src + 16 * k);
                    else dst[16 * k] = src[16 * k];
                }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    tc::grid_dep_wait();
#pragma unroll
    for (int k = 0; k + 1 < TAB_STAGES; ++k) load(k, k);
    int stage = 0;
    for (int k = 0; k < steps; ++k, stage = (stage + 1) % TAB_STAGES) {
        load(k + TAB_STAGES - 1, (stage + TAB_STAGES - 1) % TAB_STAGES);
        asm volatile("cp.async.wait_group %0;" ::"n"(TAB_STAGES - 1) : "memory");
        __syncwarp();  // every lane's copies have arrived
        const I name = t0 + k * TAB_STEP + lane < t1 ? names[stage * TAB_STEP + lane] : I(-1);
        const int row = (name >= 0 && name < rows && name != padding ? int(name) : rows) * (TAB_COLS / 2);
        const T* v = tile + stage * TILE + 2 * lane;
#pragma unroll
        for (int g = 0; g < TAB_STEP; g += TAB_GROUP) {
            int r[TAB_GROUP];
            float2 f[TAB_GROUP], s[TAB_GROUP];  // values, with those before them of the same row; the table's
#pragma unroll
            for (int j = 0; j < TAB_GROUP; ++j) {
                r[j] = __shfl_sync(0xFFFFFFFFu, row, g + j, 16);
                Vec<T, 2> e;
                e.load(v + (g + j) * TAB_COLS);
                f[j] = make_float2(e.get(0), e.get(1));
                s[j] = my[r[j]];
            }
#pragma unroll
            for (int j = 0; j < TAB_GROUP; ++j) {
                float2 b = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < j; ++i)
                    if (r[i] == r[j]) b = f[i];
                f[j] = make_float2(b.x + f[j].x, b.y + f[j].y);
                s[j] = make_float2(s[j].x + f[j].x, s[j].y + f[j].y);
            }
#pragma unroll
            for (int j = 0; j < TAB_GROUP; ++j) my[r[j]] = s[j];
        }
        __syncwarp();
    }
    __syncthreads();
    // the copies added in order, four columns at a time
    for (int i = int(threadIdx.x) * 4; i < rows * TAB_COLS; i += int(blockDim.x) * 4) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < units; ++k) {
            const float4 e = *reinterpret_cast<const float4*>(tab + size_t(k) * size + i);
            s = make_float4(s.x + e.x, s.y + e.y, s.z + e.z, s.w + e.w);
        }
        const int r = i / TAB_COLS, c = i % TAB_COLS;
        float* o = part + (int64_t(range) * rows + r) * D + c0 + c;
        if (D % 4 == 0) {
            if (c < width) *reinterpret_cast<float4*>(o) = s;
        } else {
            if (c < width) o[0] = s.x;
            if (c + 1 < width) o[1] = s.y;
            if (c + 2 < width) o[2] = s.z;
            if (c + 3 < width) o[3] = s.w;
        }
    }
}

// dtable = scale * the blocks' sums, added in order: eight lanes an element (an eighth of the
// blocks each, then a fixed butterfly).
template <typename T>
__global__ void __launch_bounds__(256) embed_table_sum(int64_t values, int blocks, float scale, const float* part,
                                                       T* dtable)
{
    __shared__ float sm[8][32];
    const int64_t e = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31);
    const int l = threadIdx.x >> 5;
    float s = 0.f;
    tc::grid_dep_wait();
    if (e < values)
        for (int b0 = l; b0 < blocks; b0 += 8 * 64) {  // 64 at a time, so that no chain is long
            float part_sum = 0.f;
            const int b1 = min(blocks, b0 + 8 * 64);
#pragma unroll 8
            for (int b = b0; b < b1; b += 8) part_sum += part[int64_t(b) * values + e];
            s += part_sum;
        }
    sm[l][threadIdx.x & 31] = s;
    __syncthreads();
    if (l == 0 && e < values) {
        s = 0.f;
        for (int k = 0; k < 8; ++k) s += sm[k][threadIdx.x];
        Elem<T>::st(dtable + e, s * scale);
    }
}

// ---- sums ------------------------------------------------------------------------------------
// A group of `cols` threads sums the runs that begin in its chunk of the sorted tokens, each
// thread one vector of the row.  A run that goes on in the next chunk and ends there is summed to
// its end.  A longer one leaves partial sums: part[chunk][1] where it begins, part[chunk][0] in
// each chunk that it enters from before.
// 16384 tokens, rows of 1024 bf16: 13 us, 2.6 TB/s, bound by instructions (0.66 issued a slot: adds
// and conversions at a few tokens a chunk); 887914 tokens, rows of 72 fp32: 74 us, 3.5 TB/s, by the
// latency of rows that lie anywhere.
struct ChunkRuns {
    bool skip;       // the run that enters from before is another group's
    bool head;       // it is a long one: its part of this chunk is a partial sum
    int end;         // where the group stops
    bool tail;       // the run at the end is a long one
    __device__ __forceinline__ ChunkRuns(const uint32_t* keys, int n, int chunk, int i0, int i1)
    {
        const uint32_t k0 = keys[i0], k1 = keys[i1 - 1];
        const bool enters = i0 > 0 && keys[i0 - 1] == k0, leaves = i1 < n && keys[i1] == k1;
        const bool from_last = enters && (i0 - chunk <= 0 || keys[i0 - chunk - 1] != k0);  // began in the chunk before
        skip = from_last && !(leaves && k0 == k1);
        head = enters && !skip;
        const bool one = enters && k0 == k1;  // a single run from before
        const int i2 = min(n, i1 + chunk);
        const bool ends_next = i2 >= n || keys[i2] != k1;
        tail = leaves && !one && !ends_next;
        end = leaves && !one && ends_next ? i2 : i1;
    }
};

// Vectors of a thread: narrow ones (rows that are not a multiple of 16 bytes) share a token's
// bookkeeping, 16 bytes of a row together (626078 tokens, 184423 rows of 37 fp32, bound by
// instructions: 74 us with one of 4 bytes, 48 with four).
template <typename T, int V> constexpr int sum_vectors()
{
    return int(sizeof(T)) * V >= 16 ? 1 : int(sizeof(T)) * V == 8 ? 2 : 4;
}

template <typename T, int V>
__global__ void __launch_bounds__(SUM_THREADS, SUM_BLOCKS_SM) embed_sum(int n, int rows, int D, int cols, int wins, int chunk,
                                                         int chunks, float scale, const uint32_t* keys,
                                                         const uint32_t* pos, const T* dy, T* dtable, float* part)
{
    constexpr int U = 4, E = sum_vectors<T, V>();
    const int per = SUM_THREADS / cols, sub = int(threadIdx.x) / cols;
    const int win = int(blockIdx.x % wins);
    const int64_t ch = int64_t(blockIdx.x / wins) * per + sub;
    int c[E];
    bool in[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        c[e] = ((win * E + e) * cols + int(threadIdx.x) - sub * cols) * V;
        in[e] = c[e] < D;
    }
    tc::grid_dep_wait();
    tc::grid_dep_launch();
    if (sub >= per || ch >= chunks || !in[0]) return;
    const int i0 = int(ch) * chunk, i1 = min(n, i0 + chunk);
    const ChunkRuns run(keys, n, chunk, i0, i1);
    float acc[E][V];
    auto clear = [&]() {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int k = 0; k < V; ++k) acc[e][k] = 0.f;
    };
    clear();
    uint32_t cur = keys[i0];
    const uint32_t last = keys[i1 - 1];
    bool head = run.head, skip = run.skip;
    auto flush = [&](bool tail) {
        if (cur >= uint32_t(rows) || skip) return;
        if (head || tail) {
            float* o = part + (ch * 2 + (head ? 0 : 1)) * D;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (in[e])
#pragma unroll
                    for (int k = 0; k < V; ++k) o[c[e] + k] = acc[e][k];
        } else {
            T* o = dtable + int64_t(cur) * D;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float f[V];
#pragma unroll
                for (int k = 0; k < V; ++k) f[k] = acc[e][k] * scale;
                Vec<T, V> v;
                v.set(f);
                if (in[e]) v.store(o + c[e]);
            }
        }
    };
    // Two steps ahead a token's name is read, one step ahead its value, and neither is looked at
    // before its step.  Beyond the chunk only the run at its end counts.
    uint32_t k[U], p[U], kn[U], kc[U];
    Vec<T, V> v[U][E], vn[U][E];
    auto names = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            k[u] = i + u < run.end ? keys[i + u] : 0xFFFFFFFFu;
            p[u] = i + u < run.end ? pos[i + u] : 0u;
        }
    };
    auto values = [&](int i) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kn[u] = i + u < i1 || k[u] == last ? k[u] : 0xFFFFFFFFu;
            const T* from = dy + int64_t(p[u]) * D;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (in[e] && kn[u] < uint32_t(rows)) vn[u][e].load(from + c[e]);
                else vn[u][e].zero();
            }
        }
    };
    names(i0);
    values(i0);
    names(i0 + U);
    for (int i = i0; i < run.end; i += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            kc[u] = kn[u];
#pragma unroll
            for (int e = 0; e < E; ++e) v[u][e] = vn[u][e];
        }
        values(i + U);
        names(i + 2 * U);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < i1 || kc[u] == last) {
                if (kc[u] != cur) {
                    flush(false);
                    cur = kc[u];
                    head = skip = false;
                    clear();
                }
#pragma unroll
                for (int e = 0; e < E; ++e)
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[e][j] += v[u][e].get(j);
            }
    }
    flush(run.tail);
}

// The long runs: a block looks at `look` chunks, and for each that a long run begins in adds the
// run's partials, V <= 4 values a thread: lanes take chunks round robin while those go on with the
// run, then the lanes are added in order.  So many chunks that the blocks are resident at once.  A
// chain of latencies (a run's keys and partials are read together, eight of a lane's at a time).
template <typename T, int V>
__global__ void __launch_bounds__(FIX_THREADS) embed_fix(int n, int rows, int D, int cols, int wins, int chunk,
                                                         int chunks, int look, float scale, const uint32_t* keys,
                                                         T* dtable, const float* part)
{
    constexpr int U = 8;
    __shared__ __align__(16) float sm[FIX_THREADS][V];
    __shared__ int begins[FIX_MAX];  // chunk that a long run begins in
    __shared__ uint32_t name[FIX_MAX], sums[FIX_THREADS / 32];
    const int win = int(blockIdx.x % wins), ch0 = int(blockIdx.x / wins) * look;
    const int lanes = FIX_THREADS / cols, lane = int(threadIdx.x) / cols, col = int(threadIdx.x) - lane * cols;
    const int c = (win * cols + col) * V;
    // The keys, too, are read behind the wait: they are the sort's, which is done when any block of the
    // kernel before runs on, but only the wait makes what earlier kernels wrote visible here.
    static_assert(FIX_THREADS >= FIX_MAX, "a thread a chunk");
    int active;
    tc::grid_dep_wait();
    {
        const int ch = ch0 + int(threadIdx.x);
        uint32_t key = 0;
        bool is = false;
        if (int(threadIdx.x) < look && ch < chunks) {
            const int i0 = ch * chunk, i1 = min(n, i0 + chunk), i2 = min(n, i1 + chunk);
            // one round of reads: a run that goes on beyond the next chunk, and began in this one
            const uint32_t before = i0 > 0 ? keys[i0 - 1] : 0xFFFFFFFFu, first = keys[i0];
            const uint32_t after = i1 < n ? keys[i1] : 0xFFFFFFFFu, beyond = i2 < n ? keys[i2] : 0xFFFFFFFFu;
            key = keys[i1 - 1];
            is = key < uint32_t(rows) && after == key && beyond == key && !(before == first && first == key);
        }
        const int at = int(block_scan(is, sums));
        if (is) {
            begins[at - 1] = ch;
            name[at - 1] = key;
        }
        active = __syncthreads_count(is);
    }
    if (active == 0) return;
    // the block's long runs side by side, as many as it has lanes, each with `per` lanes
    const int per = max(1, min(32, lanes / active)), slots = lanes / per, slot = lane / per, sub = lane - slot * per;
    for (int done = 0; done < active; done += slots) {
        const int k = slot < slots && done + slot < active ? done + slot : -1;  // this lane's run
        float acc[V];
        float* mine = sm[min(lane, lanes - 1) * cols + col];  // this lane's sum
#pragma unroll
        for (int i = 0; i < V; ++i) {
            acc[i] = 0.f;
            if (lane < lanes) mine[i] = 0.f;
        }
        if (k >= 0 && c < D) {
            const int ch = begins[k];
            const uint32_t key = name[k];
            bool on = true;
            int stop = sub + 256 * per;  // 256 chunks at a time, so that no chain is long
            for (int j = sub; on; j += per * U) {
                uint32_t q[U];
                Vec<float, V> v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int at = ch + j + u * per;
                    const bool in = at < chunks;
                    q[u] = !in ? 0xFFFFFFFFu : at == ch ? key : keys[int64_t(at) * chunk];
                    if (in) v[u].load(part + (int64_t(at) * 2 + (at == ch ? 1 : 0)) * D + c);
                    else v[u].zero();
                }
                if (j == stop) {
                    stop += 256 * per;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        mine[i] += acc[i];
                        acc[i] = 0.f;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    on = q[u] == key;  // beyond the run a partial is another's, or nothing
                    if (on)
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[i] += v[u].get(i);
                }
            }
        }
        if (lane < lanes)
#pragma unroll
            for (int i = 0; i < V; ++i) mine[i] += acc[i];
        __syncthreads();
        if (k >= 0 && sub == 0 && c < D) {
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = mine[i];
            for (int l = 1; l < per; ++l)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += sm[(lane + l) * cols + col][i];
            Vec<T, V> v;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] *= scale;
            v.set(acc);
            v.store(dtable + int64_t(name[k]) * D + c);
        }
        __syncthreads();
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
cudaError_t sort_tokens(const conv_embed_desc_t& e, const EmbedPlan& q, const DevInfo& d, const I* idx,
                        unsigned char* ws, void* dtable, int& where, cudaStream_t s)
{
    const int n = int(e.T), bins = 1 << q.digit_bits;
    const size_t bytes = size_t(e.V) * e.D * (e.dtype == CONV_F32 ? 4 : 2);
    if (q.cluster) {
        const int S = q.cluster;
        constexpr int smem = 4 * (4 * CS_TOKENS + 2 * SORT_MAX_BINS + CS_WARPS) + 2 * CS_WARPS * SORT_MAX_BINS;
        cudaError_t r = ensure_smem<sort_cluster<I>>(smem);
        if (r != cudaSuccess) return r;
        const int64_t vecs = int64_t(bytes / 16);
        // the sorting cluster, and blocks to fill with (whole clusters)
        const int64_t want = (vecs + int64_t(CS_THREADS) * 8 - 1) / (int64_t(CS_THREADS) * 8);
        // All resident at once: with a block an SM, 120 of the 152 SMs hold clusters of eight (the
        // GPCs leave a rest), and a second wave would begin when the first one's share is done.
        // 112 blocks fill at the memory's rate (16384 tokens, 50021 x 1024 bf16: 23 -> 18 us).
        const int more = round_up(int(std::min<int64_t>(std::max<int64_t>(1, want), d.sms * 3 / 4 - kMaxCluster + 1)), S);
        where = 0;
        return launch_ex(sort_cluster<I>, dim3(S + more), dim3(CS_THREADS), smem, s, S, true, n, e.V, e.padding_idx, S,
                         q.log_items, q.passes, q.digit_bits, idx, reinterpret_cast<uint32_t*>(ws + q.off_keys[0]),
                         reinterpret_cast<uint32_t*>(ws + q.off_pos[0]), static_cast<uint4*>(dtable), vecs,
                         static_cast<unsigned char*>(dtable) + vecs * 16, int(bytes - vecs * 16));
    }
    cudaError_t z = cudaMemsetAsync(dtable, 0, bytes, s);
    if (z != cudaSuccess) return z;
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

template <typename T, typename I, int V>
cudaError_t table_v(const conv_embed_desc_t& e, const EmbedPlan& q, const I* idx, const T* dy, float* part,
                    cudaStream_t s)
{
    const cudaError_t r = ensure_smem<embed_table<T, I, V>>(q.smem);
    if (r != cudaSuccess) return r;
    return launch_ex(embed_table<T, I, V>, dim3(unsigned(q.blocks) * unsigned(q.wins)), dim3(q.units * 16), q.smem, s,
                     1, true, int(e.T), e.V, e.padding_idx, e.D, q.blocks, q.units, idx, dy, part);
}

template <typename T, typename I>
cudaError_t few_t(const conv_embed_desc_t& e, const EmbedPlan& q, const I* idx, const T* dy, T* dtable, cudaStream_t s)
{
    const dim3 grid(unsigned(e.T * q.wins + q.blocks));
    cudaError_t r = cudaSuccess;
#define EMB_CALL(V_)                                                                                              \
    r = launch_ex(embed_few<T, I, V_>, grid, dim3(FEW_THREADS), 0, s, 1, true, int(e.T), e.V, e.padding_idx, e.D, \
                  q.cols, q.wins, q.blocks, e.scale, idx, dy, dtable)
    if (q.V == 8) {
        if constexpr (sizeof(T) == 2) EMB_CALL(8);
    } else if (q.V == 4) EMB_CALL(4);
    else if (q.V == 2) EMB_CALL(2);
    else EMB_CALL(1);
#undef EMB_CALL
    return r != cudaSuccess ? r : cudaGetLastError();
}

template <typename T, typename I>
cudaError_t table_t(const conv_embed_desc_t& e, const EmbedPlan& q, const I* idx, const T* dy, T* dtable, float* part,
                    cudaStream_t s)
{
    // copies of 16 bytes, or of 4 (bf16 of an odd width: 2) where the rows are not aligned for them
    constexpr int W = 16 / int(sizeof(T)), N = 4 / int(sizeof(T));
    cudaError_t r = e.D % W == 0   ? table_v<T, I, W>(e, q, idx, dy, part, s)
                    : e.D % N == 0 ? table_v<T, I, N>(e, q, idx, dy, part, s)
                                   : table_v<T, I, 1>(e, q, idx, dy, part, s);
    if (r != cudaSuccess) return r;
    const int64_t values = int64_t(e.V) * e.D;
    const float* cpart = part;
    r = launch_ex(embed_table_sum<T>, dim3(unsigned((values + 31) / 32)), dim3(256), 0, s, 1, true, values, q.blocks,
                  e.scale, cpart, dtable);
    return r != cudaSuccess ? r : cudaGetLastError();
}

template <typename T>
cudaError_t sum_t(const conv_embed_desc_t& e, const EmbedPlan& q, const DevInfo& d, const uint32_t* keys,
                  const uint32_t* pos, const T* dy, T* dtable, float* part, cudaStream_t s)
{
    const int n = int(e.T), per = SUM_THREADS / q.cols;
    const dim3 sgrid(unsigned(ceil_div(q.chunks, per)) * unsigned(q.wins));
    // the last kernel's columns: vectors of at most four values
    const int nvf = e.D / std::min(q.V, 4), fwins = ceil_div(nvf, SUM_THREADS), fcols = ceil_div(nvf, fwins);
    const int look = std::min(FIX_MAX, std::max(FIX_MIN, ceil_div(q.chunks, std::max(1, d.sms / fwins))));
    const dim3 fgrid(unsigned(ceil_div(q.chunks, look)) * unsigned(fwins));
    cudaError_t r = cudaSuccess;
    const float* cpart = part;
#define EMB_CALL(V_)                                                                                             \
    do {                                                                                                         \
        r = launch_ex(embed_sum<T, V_>, sgrid, dim3(SUM_THREADS), 0, s, 1, true, n, e.V, e.D, q.cols, q.wins,    \
                      q.chunk, q.chunks, e.scale, keys, pos, dy, dtable, part);                                  \
        if (r == cudaSuccess) {                                                                                  \
            constexpr int VF = V_ < 4 ? V_ : 4;                                                                  \
            r = launch_ex(embed_fix<T, VF>, fgrid, dim3(FIX_THREADS), 0, s, 1, true, n, e.V, e.D,                \
                          fcols, fwins, q.chunk, q.chunks, look, e.scale, keys, dtable, cpart);                  \
        }                                                                                                        \
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
    if (e.T == 0) return cudaMemsetAsync(dtable, 0, size_t(e.V) * e.D * (e.dtype == CONV_F32 ? 4 : 2), s);
    const EmbedPlan q = embed_plan(e, d);
    float* part = reinterpret_cast<float*>(ws + q.off_part);
    if (q.few) {
        if (e.dtype == CONV_F32)
            return e.index_dtype == CONV_INDEX_I32
                       ? few_t(e, q, (const int32_t*)idx, (const float*)dy, (float*)dtable, s)
                       : few_t(e, q, (const int64_t*)idx, (const float*)dy, (float*)dtable, s);
        return e.index_dtype == CONV_INDEX_I32 ? few_t(e, q, (const int32_t*)idx, (const H*)dy, (H*)dtable, s)
                                               : few_t(e, q, (const int64_t*)idx, (const H*)dy, (H*)dtable, s);
    }
    if (q.table) {
        if (e.dtype == CONV_F32)
            return e.index_dtype == CONV_INDEX_I32
                       ? table_t(e, q, (const int32_t*)idx, (const float*)dy, (float*)dtable, part, s)
                       : table_t(e, q, (const int64_t*)idx, (const float*)dy, (float*)dtable, part, s);
        return e.index_dtype == CONV_INDEX_I32 ? table_t(e, q, (const int32_t*)idx, (const H*)dy, (H*)dtable, part, s)
                                               : table_t(e, q, (const int64_t*)idx, (const H*)dy, (H*)dtable, part, s);
    }
    int where = 0;
    const cudaError_t r = e.index_dtype == CONV_INDEX_I32
                              ? sort_tokens(e, q, d, (const int32_t*)idx, ws, dtable, where, s)
                              : sort_tokens(e, q, d, (const int64_t*)idx, ws, dtable, where, s);
    if (r != cudaSuccess) return r;
    const uint32_t* keys = reinterpret_cast<const uint32_t*>(ws + q.off_keys[where]);
    const uint32_t* pos = reinterpret_cast<const uint32_t*>(ws + q.off_pos[where]);
    return e.dtype == CONV_F32 ? sum_t(e, q, d, keys, pos, (const float*)dy, (float*)dtable, part, s)
                               : sum_t(e, q, d, keys, pos, (const H*)dy, (H*)dtable, part, s);
}

}  // namespace igc
