// Type embedding: rows of a table gathered and scaled, and the gradient of the
// table summed over the nodes of each type in node order.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "eqc_elem.cuh"
#include "eqc_layers.h"

namespace cg = cooperative_groups;

namespace eqc {

void count_launch();

namespace {

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <class ID>
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t i) {
    return (int64_t)__ldg(reinterpret_cast<const ID*>(ids) + i);
}

// y[i, :] = scale * T[id_i, :].  Bound by memory: N C elements written and the
// rows read once (repeats of a row hit L2).  A block is LX lanes across the
// channels x 256 / LX rows; every thread keeps kRows rows in flight.  500009
// nodes of 95 types x 128 fp32 channels: 51 us (5.0 TB/s); 65536 rows of a
// 32000 x 2048 bf16 table: 84 us (4.8 TB/s).  Rows that no 16 bytes divide move
// 4 or 2 bytes a lane: 65536 x 896, 900 and 901 bf16 channels take 32, 57 and
// 80 us.  32768 x 128 fp32 take 5 us, less than the host's call (10 us).
constexpr int kRows = 4;

template <class T, class O, int VE, class ID>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void* ids, int64_t N, int64_t V, int C, const T* table,
                                                        int64_t ldt, float scale, O* y, int64_t ldy, int lx_log2,
                                                        unsigned* status) {
    const int lx = 1 << lx_log2, x = threadIdx.x & (lx - 1), r = threadIdx.x >> lx_log2, ly = 256 >> lx_log2;
    const int64_t row0 = (int64_t)blockIdx.x * ly * kRows + r;
    int64_t id[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t i = row0 + (int64_t)k * ly;
        id[k] = i < N ? id_at<ID>(ids, i) : 0;
    }
    bool bad = false;
#pragma unroll
    for (int k = 0; k < kRows; ++k)
        if ((uint64_t)id[k] >= (uint64_t)V) {
            id[k] = -1;
            bad = true;
        }
    if (bad && x == 0) atomicOr(status, 1u);
    for (int c = (blockIdx.y * lx + x) * VE; c < C; c += gridDim.y * lx * VE) {
        Pack<T, VE> in[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (id[k] >= 0) in[k].load(table + id[k] * ldt + c);
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t i = row0 + (int64_t)k * ly;
            if (i >= N) continue;
            Pack<O, VE> out;
#pragma unroll
            for (int e = 0; e < VE; ++e) out.set(e, id[k] >= 0 ? in[k].get(e) * scale : 0.f);
            out.store(y + i * ldy + c);
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient of the table.  The nodes are ordered by type (stable), and tiles of
// R ordered nodes are summed in that order.  A type whose nodes lie inside one
// tile is finished there; a type that reaches over tile ends leaves one partial
// row per tile, which a second kernel adds in tile order.  Ids that give no
// gradient (padding, out of range) get the key V and come last.

// Keys of K nodes, `first` + k `step` below `end`: from the ids, or (FIRST
// false) as an earlier pass left them.  All loads go out together; bad ids are
// looked for afterwards.
template <class ID, bool FIRST, int K>
__device__ __forceinline__ void load_keys(const void* in, int64_t first, int step, int64_t end, int64_t V,
                                          int64_t padding, unsigned* status, int (&key)[K]) {
    if constexpr (FIRST) {
        int64_t id[K];
#pragma unroll
        for (int k = 0; k < K; ++k) id[k] = first + k * step < end ? id_at<ID>(in, first + k * step) : 0;
        bool bad = false;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool ok = (uint64_t)id[k] < (uint64_t)V;
            bad |= !ok;
            key[k] = ok && id[k] != padding ? (int)id[k] : (int)V;
        }
        if (bad) atomicOr(status, 1u);
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) key[k] = first + k * step < end ? static_cast<const int*>(in)[first + k * step] : 0;
    }
}

constexpr int kDigitBits = 9;                 // radix of one sorting pass: at most 512
constexpr int kRadix = 1 << kDigitBits;

// The lanes that hold the same digit (by one vote per bit), among the valid.
__device__ __forceinline__ unsigned same_digit(int d, int bits, bool valid) {
    unsigned peers = __ballot_sync(0xffffffffu, valid);
    for (int b = 0; b < bits; ++b) {
        const bool one = (d >> b) & 1;
        const unsigned m = __ballot_sync(0xffffffffu, one);
        peers &= one ? m : ~m;
    }
    return peers;
}

// Ranks a warp's 32 keys of one round by digit, stably, behind the keys that
// the warp ranked in earlier rounds (counted in h[digit]).
__device__ __forceinline__ int warp_rank(int* h, int d, int bits, bool valid) {
    const int lane = threadIdx.x & 31;
    const unsigned peers = same_digit(d, bits, valid);
    const int before = __popc(peers & ((1u << lane) - 1u));
    const int rank = valid ? h[d] + before : 0;
    __syncwarp();
    if (valid && before == 0) h[d] += __popc(peers);
    __syncwarp();
    return rank;
}

// Sum of v over the lower-ranked threads of the block (THREADS of them).
template <int THREADS>
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    // every warp adds up the sums of the warps before it
    int before = lane < warp ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    return before + inc - v;
}

// Sort of up to 8 x 8192 nodes (sort_few) in one launch by one cluster: keys and node
// numbers stay in the CTAs' shared memory between passes and are scattered
// into each other's over the cluster (least significant digit first).  Bound
// by latency (16384 nodes, 65536 types, two passes: 19 us; 1503 nodes, one
// pass: 6 us); the launches it saves are worth more than its idle SMs.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCap = kSortThreads * 8;
constexpr int kMaxCluster = 8;

// ROUNDS (1, 2, 4, 8): nodes a thread.
template <int ROUNDS>
struct SortSmem {
    int key[2][kSortThreads * ROUNDS];
    int idx[2][kSortThreads * ROUNDS];
    int hist[kSortWarps][kRadix];
    int total[kRadix];
    int base[kRadix];
    int warp_sums[kSortWarps];
};

template <class ID, int ROUNDS>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const void* ids, int N, int64_t V, int64_t padding,
                                                                  int digit_bits, int passes, int* keys, int* perm,
                                                                  uint4* zero, int64_t zeros, unsigned* status) {
    let_next_start();
    extern __shared__ __align__(16) unsigned char smem_raw[];
    SortSmem<ROUNDS>& s = *reinterpret_cast<SortSmem<ROUNDS>*>(smem_raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    if ((int)blockIdx.x >= ctas) {
        // the other SMs write zeros to the first rows of the table meanwhile
        for (int64_t i = (int64_t)(blockIdx.x - ctas) * kSortThreads + threadIdx.x; i < zeros;
             i += (int64_t)(gridDim.x - ctas) * kSortThreads)
            zero[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int cap = kSortThreads * ROUNDS;
    const int radix = 1 << digit_bits;
    const int first = warp * 32 * ROUNDS + lane;       // this thread's items: first + 32 k
    {
        int key[ROUNDS];
        load_keys<ID, true>(ids, rank * cap + first, 32, N, V, padding, status, key);
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            s.key[0][first + 32 * k] = key[k];
            s.idx[0][first + 32 * k] = rank * cap + first + 32 * k;
        }
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * digit_bits, cur = p & 1;
        int key[ROUNDS], at[ROUNDS];
        for (int d = lane; d < radix; d += 32) s.hist[warp][d] = 0;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const int j = first + 32 * k;
            const bool valid = rank * cap + j < N;
            key[k] = valid ? s.key[cur][j] : 0;
            at[k] = warp_rank(s.hist[warp], (key[k] >> shift) & (radix - 1), digit_bits, valid);
        }
        __syncthreads();
        // the warps' counts of a digit become their first ranks: two threads a digit, half of the warps each
        const int half = tid >> kDigitBits, d0 = tid & (kRadix - 1);
        int count[kSortWarps / 2], sum = 0;
        if (d0 < radix) {
#pragma unroll
            for (int w = 0; w < kSortWarps / 2; ++w) count[w] = s.hist[half * (kSortWarps / 2) + w][d0];
#pragma unroll
            for (int w = 0; w < kSortWarps / 2; ++w) {
                const int c = count[w];
                count[w] = sum;
                sum += c;
            }
            if (half == 0) s.base[d0] = sum;
        }
        __syncthreads();
        if (d0 < radix) {
            const int off = half ? s.base[d0] : 0;
#pragma unroll
            for (int w = 0; w < kSortWarps / 2; ++w) s.hist[half * (kSortWarps / 2) + w][d0] = off + count[w];
            if (half) s.total[d0] = off + sum;
        }
        cluster.sync();
        int all = 0, below = 0;
        if (tid < radix) {
            int c[kMaxCluster];
#pragma unroll
            for (int q = 0; q < kMaxCluster; ++q)
                c[q] = q < ctas ? *cluster.map_shared_rank(&s.total[tid], q) : 0;
#pragma unroll
            for (int q = 0; q < kMaxCluster; ++q) {
                all += c[q];
                if (q < rank) below += c[q];
            }
        }
        const int excl = block_exclusive<kSortThreads>(all, s.warp_sums);
        if (tid < radix) s.base[tid] = excl + below;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const int j = first + 32 * k;
            if (rank * cap + j >= N) continue;
            const int d = (key[k] >> shift) & (radix - 1);
            const int pos = s.base[d] + s.hist[warp][d] + at[k], idx = s.idx[cur][j];
            if (p == passes - 1) {
                keys[pos] = key[k];
                perm[pos] = idx;
            } else {
                const int q = pos / cap, o = pos % cap;
                *cluster.map_shared_rank(&s.key[cur ^ 1][o], q) = key[k];
                *cluster.map_shared_rank(&s.idx[cur ^ 1][o], q) = idx;
            }
        }
        cluster.sync();
    }
}

// Sort of more nodes: per pass a histogram of every tile of 2048 nodes, a scan
// over the tiles by digit, and a stable scatter.  500009 nodes, one pass: 4 + 2
// + 9 us, most of it the latency of loads, votes and scattered stores.
constexpr int kLsdThreads = 512;
constexpr int kLsdRounds = 4;
constexpr int kLsdTile = kLsdThreads * kLsdRounds;
static_assert(kLsdThreads == kRadix && kSortThreads == 2 * kRadix, "one and two threads per digit");

template <class ID, bool FIRST>
__global__ void __launch_bounds__(kLsdThreads) embed_hist_kernel(const void* in, int N, int64_t V, int64_t padding,
                                                                 int shift, int mask, int* hist, int tiles,
                                                                 unsigned* status) {
    wait_for_last();
    let_next_start();
    __shared__ int h[kRadix];
    h[threadIdx.x] = 0;
    __syncthreads();
    const int64_t i0 = (int64_t)blockIdx.x * kLsdTile + threadIdx.x;
    int key[kLsdRounds];
    load_keys<ID, FIRST>(in, i0, kLsdThreads, N, V, padding, status, key);
#pragma unroll
    for (int k = 0; k < kLsdRounds; ++k) {
        const bool valid = i0 + k * kLsdThreads < N;
        const int d = (key[k] >> shift) & mask;
        // lanes with one digit count it once: a table of few types would serialise on it
        const unsigned peers = same_digit(d, 32 - __clz(mask), valid);
        if (valid && __ffs(peers) - 1 == (int)(threadIdx.x & 31)) atomicAdd(&h[d], __popc(peers));
    }
    __syncthreads();
    if ((int)threadIdx.x <= mask) hist[(int64_t)threadIdx.x * tiles + blockIdx.x] = h[threadIdx.x];
}

// hist[d][*] becomes its exclusive scan over the tiles, total[d] its sum: one warp per digit.
__global__ void embed_scan_kernel(int* hist, int tiles, int radix, int* total) {
    wait_for_last();
    let_next_start();
    const int d = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (d >= radix) return;
    int* h = hist + (int64_t)d * tiles;
    int run = 0;
    for (int t = 0; t < tiles; t += 32) {
        const int v = t + lane < tiles ? h[t + lane] : 0;
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (t + lane < tiles) h[t + lane] = run + inc - v;
        run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) total[d] = run;
}

template <class ID, bool FIRST>
__global__ void __launch_bounds__(kLsdThreads) embed_scatter_kernel(const void* in, const int* idx_in, int N,
                                                                    int64_t V, int64_t padding, int shift, int mask,
                                                                    const int* hist, const int* total, int tiles,
                                                                    int* keys_out, int* idx_out, unsigned* status) {
    wait_for_last();
    let_next_start();
    __shared__ int wh[kLsdThreads / 32][kRadix];
    __shared__ int base[kRadix];
    __shared__ int sums[kLsdThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int d = lane; d <= mask; d += 32) wh[warp][d] = 0;
    const int excl = block_exclusive<kLsdThreads>(tid <= mask ? total[tid] : 0, sums);
    if (tid <= mask) base[tid] = excl + hist[(int64_t)tid * tiles + blockIdx.x];
    __syncwarp();
    const int64_t i0 = (int64_t)blockIdx.x * kLsdTile + warp * 32 * kLsdRounds + lane;
    int key[kLsdRounds], at[kLsdRounds];
    load_keys<ID, FIRST>(in, i0, 32, N, V, padding, status, key);
    int idx[kLsdRounds];
#pragma unroll
    for (int k = 0; k < kLsdRounds; ++k)
        idx[k] = FIRST ? (int)(i0 + 32 * k) : i0 + 32 * k < N ? idx_in[i0 + 32 * k] : 0;
#pragma unroll
    for (int k = 0; k < kLsdRounds; ++k) at[k] = warp_rank(wh[warp], (key[k] >> shift) & mask, 32 - __clz(mask), i0 + 32 * k < N);
    __syncthreads();
    if (tid <= mask) {
        int run = base[tid];
#pragma unroll
        for (int w = 0; w < kLsdThreads / 32; ++w) {
            const int c = wh[w][tid];
            wh[w][tid] = run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kLsdRounds; ++k) {
        const int64_t i = i0 + 32 * k;
        if (i >= N) continue;
        const int pos = wh[warp][(key[k] >> shift) & mask] + at[k];
        keys_out[pos] = key[k];
        idx_out[pos] = idx[k];
    }
}

// Rows of a block that writes zeros: 512 KB of them, so that the search takes
// little of its time, and at most one a thread.
constexpr int kZeroRows = 256, kZeroBytes = 512 * 1024;
constexpr int64_t kSortZeroBytes = 64 << 20;

struct SumParams {
    const int *keys, *perm;   // nodes in type order, as the kernel before left them
    int N, C, R, tiles, slabs, lx_log2;
    int sum_blocks, zero_rows;
    int64_t V, ldg, zero_from;     // rows up to zero_from are zeros already
    float scale;
    float* part;              // [tiles][2][C]: the type begun before the tile, the one that goes on behind it
};

// First position whose key is not below k.
__device__ __forceinline__ int lower_bound(const int* keys, int n, int k) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (int)(((unsigned)lo + (unsigned)hi) >> 1);
        if (keys[mid] < k) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Blocks up to sum_blocks: one worker (1 << lx_log2 lanes) per tile and slab of
// channels; the rest write zeros to the rows of types without nodes, which the
// ordered keys show by search.  Bound by memory: gy is read once, dT written
// once.  500009 rows of 128 fp32 channels, 95 types: 47 us (5.5 TB/s); a table
// of 65536 x 2048 fp32 with 16384 bf16 rows: 97 us (5.5 TB/s).
template <class T, class O, int VE>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumParams p, const O* gy, T* dtable) {
    wait_for_last();
    let_next_start();
    if ((int)blockIdx.x >= p.sum_blocks) {
        __shared__ bool empty[kZeroRows];
        const int64_t v0 = p.zero_from + (int64_t)(blockIdx.x - p.sum_blocks) * p.zero_rows;
        const int rows = (int)(p.V - v0 < p.zero_rows ? p.V - v0 : p.zero_rows);
        if ((int)threadIdx.x < rows) {
            const int v = (int)(v0 + threadIdx.x), at = lower_bound(p.keys, p.N, v);
            empty[threadIdx.x] = at >= p.N || p.keys[at] != v;
        }
        __syncthreads();
        Pack<T, VE> zero;
#pragma unroll
        for (int e = 0; e < VE; ++e) zero.set(e, 0.f);
        const int vecs = p.C / VE;
        for (int r = 0, c = threadIdx.x;; c += 256) {
            while (c >= vecs) {
                c -= vecs;
                ++r;
            }
            if (r >= rows) break;
            if (empty[r]) zero.store(dtable + (v0 + r) * p.C + (int64_t)c * VE);
        }
        return;
    }
    const int64_t worker = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> p.lx_log2;
    const int tile = (int)(worker / p.slabs), slab = (int)(worker % p.slabs);
    const int c = ((slab << p.lx_log2) + (threadIdx.x & ((1 << p.lx_log2) - 1))) * VE;
    if (tile >= p.tiles || c >= p.C) return;
    const int64_t q0 = (int64_t)tile * p.R;
    const int n = (int)(p.N - q0 < p.R ? p.N - q0 : p.R);
    const int *keys = p.keys + q0, *perm = p.perm + q0;
    const int none = (int)p.V;
    int cur = keys[0];
    bool begun_before = tile > 0 && keys[-1] == cur;
    float acc[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = 0.f;
    float* part = p.part + (int64_t)tile * 2 * p.C + c;
    const auto row = [&](int v) {
        Pack<T, VE> out;
#pragma unroll
        for (int e = 0; e < VE; ++e) out.set(e, acc[e] * p.scale);
        out.store(dtable + (int64_t)v * p.C + c);
    };
    const auto partial = [&](int which) {
        Pack<float, VE> out;
#pragma unroll
        for (int e = 0; e < VE; ++e) out.e[e] = acc[e];
        out.store(part + which * p.C);
    };
    // batches of 8 rows in flight; the next batch's keys and places are fetched while they are
    constexpr int kAhead = 8;
    int key[kAhead], at[kAhead];
    const auto fetch = [&](int j0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            key[u] = j0 + u < n ? keys[j0 + u] : none;
            at[u] = j0 + u < n ? perm[j0 + u] : 0;
        }
    };
    fetch(0);
    for (int j0 = 0; j0 < n; j0 += kAhead) {
        Pack<O, VE> in[kAhead];
        int now[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            now[u] = key[u];
            if (key[u] != none) in[u].load(gy + (int64_t)at[u] * p.ldg + c);
        }
        fetch(j0 + kAhead);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (j0 + u >= n) break;
            if (now[u] != cur) {
                if (begun_before) partial(0);
                else row(cur);
                begun_before = false;
                cur = now[u];
#pragma unroll
                for (int e = 0; e < VE; ++e) acc[e] = 0.f;
            }
            if (cur == none) break;
#pragma unroll
            for (int e = 0; e < VE; ++e) acc[e] += in[u].get(e);
        }
        if (cur == none) return;
    }
    if (begun_before) partial(0);
    else if (q0 + n < p.N && keys[n] == cur) partial(1);
    else row(cur);
}

// Types that reach over tile ends: the tile in which such a type begins adds
// its partial row and those of the tiles behind it, in tile order.  A worker
// (1 << lx_log2 lanes, one tile and slab) does that alone where the type ends
// within kAlone tiles; what is longer is done by the block together, shares of
// the tiles by worker and the workers' sums in order.
constexpr int kAlone = 8;

template <class T, int VE>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumParams p, T* dtable) {
    wait_for_last();
    __shared__ float sums[256 * VE];
    __shared__ int long_type[256];         // of each worker: the type that takes the whole block, or V
    const int lanes = 1 << p.lx_log2, workers = 256 >> p.lx_log2;
    const int x = threadIdx.x & (lanes - 1), w = threadIdx.x >> p.lx_log2;
    const unsigned worker0 = blockIdx.x * (unsigned)workers;
    // of a worker: its tile (a block's tiles follow one another: one of them at most begins a long type, or few), its
    // channels, and the type that begins in the tile and goes on behind it (V: none)
    const unsigned tiles = p.tiles - 1;
    const auto tile_of = [&](unsigned worker) { return (int)(worker % tiles); };
    const auto channel_of = [&](unsigned worker) { return (((int)(worker / tiles) << p.lx_log2) + x) * VE; };
    const auto type_of = [&](int tile) {
        const int64_t end = (int64_t)(tile + 1) * p.R;
        const int k = p.keys[end - 1], next = p.keys[end];
        const bool before = tile > 0 && p.keys[end - p.R - 1] == k;
        return next == k && !before ? k : (int)p.V;
    };
    const auto starts = [&](int64_t t, int k) { return t * p.R < p.N && p.keys[t * p.R] == k; };
    const auto add = [&](float (&acc)[VE], int64_t row, int c) {
        Pack<float, VE> v;
        v.load_rw(p.part + row * p.C + c);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += v.e[e];
    };
    const auto finish = [&](const float (&acc)[VE], int k, int c) {
        Pack<T, VE> out;
#pragma unroll
        for (int e = 0; e < VE; ++e) out.set(e, acc[e] * p.scale);
        out.store(dtable + (int64_t)k * p.C + c);
    };
    {
        const int tile = tile_of(worker0 + w), c = channel_of(worker0 + w);
        const int k = worker0 + w < tiles * p.slabs ? type_of(tile) : (int)p.V;
        int behind = 0;      // tiles behind the first, kAlone + 1: more
        if (k != (int)p.V) {
#pragma unroll
            for (int i = 1; i <= kAlone + 1; ++i) behind += starts(tile + i, k);
            if (behind <= kAlone && c < p.C) {
                float acc[VE];
#pragma unroll
                for (int e = 0; e < VE; ++e) acc[e] = 0.f;
                add(acc, (int64_t)tile * 2 + 1, c);
#pragma unroll
                for (int i = 1; i <= kAlone; ++i)
                    if (i <= behind) add(acc, (int64_t)(tile + i) * 2, c);
                finish(acc, k, c);
            }
        }
        if (x == 0) long_type[w] = behind > kAlone ? k : (int)p.V;
    }
    __syncthreads();
    for (int u = 0; u < workers; ++u) {
        const int k = long_type[u];
        if (k == (int)p.V) continue;
        const int tile = tile_of(worker0 + u), c = channel_of(worker0 + u);
        // tile of the type's last node: the tiles behind that begin with the type follow one another
        int last = tile;
        for (int more = 256; more == 256; last += more) more = __syncthreads_count(starts((int64_t)last + 1 + threadIdx.x, k));
        const int share = (last - tile + workers - 1) / workers;          // of the tiles behind the first
        const int t0 = tile + 1 + w * share, t1 = t0 + share < last + 1 ? t0 + share : last + 1;
        float acc[VE];
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] = 0.f;
        if (c < p.C) {
            if (w == 0) add(acc, (int64_t)tile * 2 + 1, c);
#pragma unroll 8
            for (int t = t0; t < t1; ++t) add(acc, (int64_t)t * 2, c);
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) sums[threadIdx.x * VE + e] = acc[e];
        __syncthreads();
        if (w == 0 && c < p.C) {
            for (int o = 1; o < workers; ++o)
#pragma unroll
                for (int e = 0; e < VE; ++e) acc[e] += sums[((o << p.lx_log2) + x) * VE + e];
            finish(acc, k, c);
        }
        __syncthreads();
    }
}

// Few nodes and a small table (embed_few): one launch without a sort.  A CTA owns a type
// and a slab of 32 vectors of channels; every warp looks through its run of the
// ids for the type and adds the rows it finds in node order, and the warps'
// sums are added in warp order.  Bound by latency: of three launches (sort,
// sums, joins) here, and of the ids and at most N / 32 rows a warp.
template <class T, class O, int VE, class ID>
__global__ void __launch_bounds__(1024) embed_few_kernel(const void* ids, int N, int64_t V, int64_t padding, int C,
                                                         const O* gy, int64_t ldg, float scale, T* dtable,
                                                         unsigned* status) {
    __shared__ float sums[32][32 * VE];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t v = blockIdx.x;
    const int c = (blockIdx.y * 32 + lane) * VE;
    const int share = (N + 1023) / 1024 * 32;      // ids of a warp, in whole rounds of 32
    float acc[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = 0.f;
    for (int i0 = warp * share; i0 < (warp + 1) * share && i0 < N; i0 += 32) {
        const int64_t id = i0 + lane < N ? id_at<ID>(ids, i0 + lane) : 0;
        if (v == 0 && blockIdx.y == 0 && i0 + lane < N && (uint64_t)id >= (uint64_t)V) atomicOr(status, 1u);
        unsigned found = __ballot_sync(0xffffffffu, i0 + lane < N && id == v && v != padding);
        while (found) {
            Pack<O, VE> in[8];
            int count = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!found) break;
                const int i = i0 + __ffs(found) - 1;
                found &= found - 1;
                if (c < C) in[u].load(gy + (int64_t)i * ldg + c);
                ++count;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < count && c < C)
#pragma unroll
                    for (int e = 0; e < VE; ++e) acc[e] += in[u].get(e);
        }
    }
#pragma unroll
    for (int e = 0; e < VE; ++e) sums[warp][lane * VE + e] = acc[e];
    __syncthreads();
    // thread t adds channel t of the slab
    const int at = blockIdx.y * 32 * VE + threadIdx.x;
    if ((int)threadIdx.x >= 32 * VE || at >= C) return;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) s += sums[w][threadIdx.x];
    dtable[v * C + at] = from_float<T>(s * scale);
}

// Calls f with the largest of 8 (16-bit outputs), 4, 2 and 1 elements a vector
// such that every row of both tensors starts on the vector's boundary (16
// bytes at most) and C is whole vectors.
template <class T, class O, class F>
cudaError_t with_width(int C, const void* a, int64_t lda, const void* b, int64_t ldb, F&& f) {
    const auto ok = [&](int ve) {
        const auto fits = [&](const void* p, int64_t ld, size_t es) {
            const size_t piece = ve * es < 16 ? ve * es : 16;
            return reinterpret_cast<uintptr_t>(p) % piece == 0 && (size_t)ld * es % piece == 0;
        };
        return C % ve == 0 && fits(a, lda, sizeof(T)) && fits(b, ldb, sizeof(O));
    };
    constexpr int kWide = sizeof(O) == 2 ? 8 : 4;
    if (ok(kWide)) return f(std::integral_constant<int, kWide>{});
    if (ok(2)) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}

}  // namespace

cudaError_t embed_forward(const EmbedArgs& a, const void* table, int64_t table_stride, void* y, int64_t y_stride,
                          cudaStream_t st) {
    if (a.N == 0) return cudaSuccess;
    return with_type(a.in_type, [&](auto tv) {
        using T = decltype(tv);
        return with_type(a.out_type, [&](auto ov) {
            using O = decltype(ov);
            return with_width<T, O>(a.C, table, table_stride, y, y_stride, [&](auto wv) {
                constexpr int VE = decltype(wv)::value;
                const int vecs = a.C / VE;
                int lg = 0;
                while (lg < 8 && (1 << lg) < vecs) ++lg;
                const int ly = 256 >> lg;
                const dim3 grid(cdiv(a.N, (int64_t)ly * kRows), 1);
                if (a.id_bits == 32)
                    embed_fwd_kernel<T, O, VE, int32_t><<<grid, 256, 0, st>>>(
                        a.ids, a.N, a.V, a.C, static_cast<const T*>(table), table_stride, a.scale, static_cast<O*>(y),
                        y_stride, lg, a.status);
                else
                    embed_fwd_kernel<T, O, VE, int64_t><<<grid, 256, 0, st>>>(
                        a.ids, a.N, a.V, a.C, static_cast<const T*>(table), table_stride, a.scale, static_cast<O*>(y),
                        y_stride, lg, a.status);
                count_launch();
                return cudaGetLastError();
            });
        });
    });
}

namespace {

// How the sum is cut for (N, C): slabs of 32 vectors (or one slab of fewer
// lanes), and tiles of R nodes so that about 16 warps run on every SM (as many
// as their registers allow), with whole batches of 8 rows in flight.
struct SumShape {
    int ve, lx_log2, slabs, R, tiles;
};
SumShape sum_shape(int64_t N, int C, int ve) {
    SumShape s{};
    s.ve = ve;
    const int vecs = C / ve;
    while (s.lx_log2 < 5 && (1 << s.lx_log2) < vecs) ++s.lx_log2;
    s.slabs = cdiv(vecs, 1 << s.lx_log2);
    const int64_t lanes = N * s.slabs << s.lx_log2;
    int64_t R = (lanes / (148 * 512) + 7) / 8 * 8;
    s.R = (int)(R < 8 ? 8 : R > 256 ? 256 : R);
    s.tiles = cdiv(N, s.R);
    return s;
}

int bit_length(int64_t v) {
    int b = 0;
    for (; v; v >>= 1) ++b;
    return b;
}

int sort_passes(int64_t V) { return cdiv(bit_length(V), kDigitBits); }

// Whether one cluster sorts: up to 65536 nodes in one pass; where there are
// more passes (V of 512 and more) up to 16384, its eight SMs being slower than
// all of them in three launches a pass (60000 nodes, 20000 types: 36 us in one
// cluster, 22 us in tiles; 16384 nodes, 65536 types: 18 and 20 us).
bool sort_few(int64_t V, int64_t N) { return N <= (sort_passes(V) == 1 ? kMaxCluster * kSortCap : 16384); }

struct EmbedWs {
    size_t keys, perm, keys2, perm2, hist, total, part, bytes;
};
// Space for any of the vector widths (the widest tiles come with width 1).
EmbedWs embed_layout(int64_t V, int C, int64_t N) {
    const auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
    EmbedWs w{};
    size_t o = 0;
    w.keys = o; o += up(4 * (size_t)N);
    w.perm = o; o += up(4 * (size_t)N);
    if (!sort_few(V, N)) {
        const size_t tiles = cdiv(N, kLsdTile);
        w.keys2 = o; o += up(4 * (size_t)N);
        w.perm2 = o; o += up(4 * (size_t)N);
        w.hist = o;  o += up(4 * tiles * kRadix);
        w.total = o; o += up(4 * kRadix);
    }
    size_t tiles = 0;
    for (const int ve : {1, 2, 4, 8}) {
        if (C % ve) continue;
        const size_t t = sum_shape(N, C, ve).tiles;
        if (t > tiles) tiles = t;
    }
    w.part = o; o += up(tiles * 2 * C * sizeof(float));
    w.bytes = o > 0 ? o : 16;
    return w;
}

template <class ID, int ROUNDS>
cudaError_t launch_sort(const EmbedArgs& a, int ctas, int digit_bits, int passes, int* keys, int* perm,
                        void* dtable, int64_t zeros, cudaStream_t st) {
    static bool done[64] = {};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        err = cudaFuncSetAttribute(embed_sort_kernel<ID, ROUNDS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)sizeof(SortSmem<ROUNDS>));
        if (err != cudaSuccess) return err;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(zeros ? 148 / ctas * ctas : ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sizeof(SortSmem<ROUNDS>);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, embed_sort_kernel<ID, ROUNDS>, a.ids, (int)a.N, a.V, a.padding, digit_bits, passes,
                             keys, perm, static_cast<uint4*>(dtable), zeros, a.status);
    count_launch();
    return err;
}

// One CTA up to 1024 nodes, clusters of 2, 4 and 8 up to 8192, then more nodes a thread.
template <class ID>
cudaError_t sort_in_cluster(const EmbedArgs& a, int digit_bits, int passes, int* keys, int* perm, void* dtable,
                            int64_t zeros, cudaStream_t st) {
    int ctas = 1;
    while (ctas < kMaxCluster && a.N > (int64_t)ctas * kSortThreads) ctas *= 2;
    const int64_t rounds = (a.N + (int64_t)ctas * kSortThreads - 1) / ((int64_t)ctas * kSortThreads);
    if (rounds <= 1) return launch_sort<ID, 1>(a, ctas, digit_bits, passes, keys, perm, dtable, zeros, st);
    if (rounds <= 2) return launch_sort<ID, 2>(a, ctas, digit_bits, passes, keys, perm, dtable, zeros, st);
    if (rounds <= 4) return launch_sort<ID, 4>(a, ctas, digit_bits, passes, keys, perm, dtable, zeros, st);
    return launch_sort<ID, 8>(a, ctas, digit_bits, passes, keys, perm, dtable, zeros, st);
}

template <class ID>
cudaError_t sort_in_tiles(const EmbedArgs& a, int digit_bits, int passes, char* base, const EmbedWs& w, int** keys,
                          int** perm, cudaStream_t st) {
    int* k[2] = {reinterpret_cast<int*>(base + w.keys), reinterpret_cast<int*>(base + w.keys2)};
    int* x[2] = {reinterpret_cast<int*>(base + w.perm), reinterpret_cast<int*>(base + w.perm2)};
    int* hist = reinterpret_cast<int*>(base + w.hist);
    int* total = reinterpret_cast<int*>(base + w.total);
    const int tiles = cdiv(a.N, kLsdTile), radix = 1 << digit_bits, N = (int)a.N;
    for (int p = 0; p < passes; ++p) {
        const int shift = p * digit_bits, o = p & 1;
        // (the first kernel of the call starts when all work before it has ended, as any launch does)
        cudaError_t err = cudaSuccess;
        if (p == 0)
            embed_hist_kernel<ID, true><<<tiles, kLsdThreads, 0, st>>>(a.ids, N, a.V, a.padding, shift, radix - 1,
                                                                       hist, tiles, a.status);
        else
            err = launch_after(embed_hist_kernel<ID, false>, tiles, kLsdThreads, st, k[o ^ 1], N, a.V, a.padding, shift,
                               radix - 1, hist, tiles, a.status);
        if (err == cudaSuccess) err = launch_after(embed_scan_kernel, cdiv(radix, 8), 256, st, hist, tiles, radix, total);
        if (err == cudaSuccess)
            err = p == 0 ? launch_after(embed_scatter_kernel<ID, true>, tiles, kLsdThreads, st, a.ids, nullptr, N, a.V,
                                        a.padding, shift, radix - 1, hist, total, tiles, k[o], x[o], a.status)
                         : launch_after(embed_scatter_kernel<ID, false>, tiles, kLsdThreads, st, k[o ^ 1], x[o ^ 1], N,
                                        a.V, a.padding, shift, radix - 1, hist, total, tiles, k[o], x[o], a.status);
        for (int i = 0; i < 3; ++i) count_launch();
        if (err == cudaSuccess) err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        *keys = k[o];
        *perm = x[o];
    }
    return cudaSuccess;
}

}  // namespace

// Whether the kernel for few nodes and small tables takes the case: where its
// CTAs run in one wave (two an SM) at the narrowest vectors, and no warp looks
// through more than 128 ids.  Water box (1503 nodes, 2 types, 128 channels):
// 6.9 us in one launch, 14.5 us in three.
static bool embed_few(int64_t V, int C, int64_t N) { return N <= 4096 && V * cdiv(C, 32) <= 2 * 148; }

size_t embed_workspace(int64_t V, int C, int64_t N) { return N == 0 || embed_few(V, C, N) ? 0 : embed_layout(V, C, N).bytes; }

cudaError_t embed_backward(const EmbedArgs& a, const void* gy, int64_t gy_stride, void* dtable, void* ws,
                           cudaStream_t st) {
    if (a.N == 0)
        return cudaMemsetAsync(dtable, 0, (size_t)a.V * a.C * type_bytes(a.in_type), st);
    if (embed_few(a.V, a.C, a.N))
        return with_type(a.in_type, [&](auto tv) {
            using T = decltype(tv);
            return with_type(a.out_type, [&](auto ov) {
                using O = decltype(ov);
                return with_width<T, O>(a.C, dtable, a.C, gy, gy_stride, [&](auto wv) {
                    constexpr int VE = decltype(wv)::value;
                    const dim3 grid((unsigned)a.V, cdiv(a.C, 32 * VE));
                    if (a.id_bits == 32)
                        embed_few_kernel<T, O, VE, int32_t><<<grid, 1024, 0, st>>>(
                            a.ids, (int)a.N, a.V, a.padding, a.C, static_cast<const O*>(gy), gy_stride, a.scale,
                            static_cast<T*>(dtable), a.status);
                    else
                        embed_few_kernel<T, O, VE, int64_t><<<grid, 1024, 0, st>>>(
                            a.ids, (int)a.N, a.V, a.padding, a.C, static_cast<const O*>(gy), gy_stride, a.scale,
                            static_cast<T*>(dtable), a.status);
                    count_launch();
                    return cudaGetLastError();
                });
            });
        });
    const EmbedWs w = embed_layout(a.V, a.C, a.N);
    char* base = static_cast<char*>(ws);
    int* keys = reinterpret_cast<int*>(base + w.keys);
    int* perm = reinterpret_cast<int*>(base + w.perm);
    // keys 0..V in equal digits of at most 9 bits
    const int bits = bit_length(a.V), passes = sort_passes(a.V), digit_bits = cdiv(bits, passes);
    cudaError_t err;
    // A sort of one cluster leaves the other SMs idle for some 10 us: they write zeros to the first rows meanwhile
    // (whole 16 bytes, up to 64 MB), and the sums overwrite those that have nodes.
    int64_t zero_to = 0;
    const int64_t row = (int64_t)a.C * type_bytes(a.in_type);
    if (sort_few(a.V, a.N)) {
        if (reinterpret_cast<uintptr_t>(dtable) % 16 == 0) {
            zero_to = kSortZeroBytes / row;
            zero_to = (zero_to < a.V ? zero_to : a.V) / 16 * 16;
        }
        const int64_t zeros = zero_to * row / 16;
        err = a.id_bits == 32 ? sort_in_cluster<int32_t>(a, digit_bits, passes, keys, perm, dtable, zeros, st)
                              : sort_in_cluster<int64_t>(a, digit_bits, passes, keys, perm, dtable, zeros, st);
    } else {
        err = a.id_bits == 32 ? sort_in_tiles<int32_t>(a, digit_bits, passes, base, w, &keys, &perm, st)
                              : sort_in_tiles<int64_t>(a, digit_bits, passes, base, w, &keys, &perm, st);
    }
    if (err != cudaSuccess) return err;
    return with_type(a.in_type, [&](auto tv) {
        using T = decltype(tv);
        return with_type(a.out_type, [&](auto ov) {
            using O = decltype(ov);
            return with_width<T, O>(a.C, dtable, a.C, gy, gy_stride, [&](auto wv) {
                constexpr int VE = decltype(wv)::value;
                const SumShape s = sum_shape(a.N, a.C, VE);
                SumParams p{};
                p.keys = keys;
                p.perm = perm;
                p.N = (int)a.N;
                p.C = a.C;
                p.R = s.R;
                p.tiles = s.tiles;
                p.slabs = s.slabs;
                p.lx_log2 = s.lx_log2;
                p.V = a.V;
                p.ldg = gy_stride;
                p.scale = a.scale;
                p.part = reinterpret_cast<float*>(base + w.part);
                p.sum_blocks = cdiv(((int64_t)s.tiles * s.slabs) << s.lx_log2, 256);
                const int64_t zr = kZeroBytes / row;
                p.zero_from = zero_to;
                p.zero_rows = (int)(zr < 1 ? 1 : zr > kZeroRows ? kZeroRows : zr);
                cudaError_t e = launch_after(embed_sum_kernel<T, O, VE>, p.sum_blocks + cdiv(a.V - zero_to, p.zero_rows),
                                             256, st, p, static_cast<const O*>(gy), static_cast<T*>(dtable));
                count_launch();
                if (e == cudaSuccess && s.tiles > 1) {
                    e = launch_after(embed_join_kernel<T, VE>,
                                     cdiv(((int64_t)(s.tiles - 1) * s.slabs) << s.lx_log2, 256), 256, st, p,
                                     static_cast<T*>(dtable));
                    count_launch();
                }
                return e;
            });
        });
    });
}

}  // namespace eqc
