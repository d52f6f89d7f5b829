// Token embedding lookup with scaling, and its gradient by sorted tokens
// (include/lora_embedding.h).
//
//   out[t] = bf16(scale E[id_t]),    dE[v] = scale sum_{t: id_t = v} dOut[t]
//
// Both passes only move bytes: the lookup reads a row and writes a row for
// each token; the gradient reads each token's row of dOut once and writes
// every row of dE once, most of them zeros (a 128K vocabulary against a few
// thousand tokens).  So that no row is read back to be added to, and no
// atomic's order shows in a sum, the tokens are sorted by id first (stable
// radix sort): the tokens of an id then lie next to each other, in token
// order, and whoever writes row v sums them in registers.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "vec8.cuh"

namespace lmlp {
namespace step {

// ----------------------------------------------------------------------------- lookup

constexpr int kEmbThreads = 256;

// A row is walked by `tpr` threads (a power of two, at most the block), 16
// bytes at a time; a block holds kEmbThreads / tpr rows.
struct EmbFwdArgs {
    const long long* ids;
    const __nv_bfloat16* E;
    __nv_bfloat16* out;
    long long N, V;
    int nv;        // 16-byte vectors of a row
    int log_tpr;
    float scale;
    int* status;
};

__global__ void __launch_bounds__(kEmbThreads) embed_fwd_kernel(const EmbFwdArgs a) {
    const int rows = kEmbThreads >> a.log_tpr;
    const int lane = threadIdx.x & ((1 << a.log_tpr) - 1);
    const long long t = static_cast<long long>(blockIdx.x) * rows + (threadIdx.x >> a.log_tpr);
    if (t >= a.N) return;
    const long long id = a.ids[t];
    uint4* o = reinterpret_cast<uint4*>(a.out) + t * a.nv;
    const int step = 1 << a.log_tpr;
    if (id < 0 || id >= a.V) {
        if (lane == 0) atomicExch(a.status, kStatusBad);
        for (int j = lane; j < a.nv; j += step) o[j] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        return;
    }
    const uint4* e = reinterpret_cast<const uint4*>(a.E) + id * a.nv;
    constexpr int U = 4;
    for (int j0 = lane; j0 < a.nv; j0 += U * step) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j0 + u * step < a.nv) v[u] = __ldg(e + j0 + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u * step >= a.nv) break;
            float f[8];
            widen8(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= a.scale;
            o[j0 + u * step] = round8(f);
        }
    }
}

// ----------------------------------------------------------------------------- sorting the tokens

// Stable least-significant-digit radix sort of (id, token), digits of up to 9
// bits: 2 passes for vocabularies up to 2^18 - 1.  The tokens that take no
// part (padding_idx, ids outside [0, V)) get the key V and end behind all
// rows.
constexpr int kSortMaxBits = 9;
constexpr int kSortMaxBins = 1 << kSortMaxBits;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortSmallItems = 8;                                  // one block sorts up to 8192 tokens
constexpr int kSortSmall = kSortThreads * kSortSmallItems;
constexpr int kSortTileItems = 4;                                   // a tile of the many-block sort
constexpr int kSortTile = kSortThreads * kSortTileItems;

struct SortArgs {
    const long long* ids;
    int N;
    int V;
    long long padding;  // < 0: none
    int bits;           // digit width
    int passes;
    int ntiles;
    uint32_t *key[2], *val[2];  // [N] each; the result is in key[passes & 1], val[passes & 1]
    uint32_t* hist;             // [passes][ntiles][bins]
    uint32_t* counters;         // zeroed here for the gradient kernel
    int ncounters;
    int* status;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, long long id) {
    if (id == a.padding && a.padding >= 0) return static_cast<uint32_t>(a.V);
    if (id < 0 || id >= a.V) {
        atomicExch(a.status, kStatusBad);
        return static_cast<uint32_t>(a.V);
    }
    return static_cast<uint32_t>(id);
}

struct SortShared {
    uint16_t warp_bin[kSortWarps][kSortMaxBins];  // counts, then each warp's start within its bin
    uint32_t bin_total[kSortMaxBins];
    uint32_t bin_start[kSortMaxBins];
    uint32_t scan[kSortWarps];
};

// Where each of a block's keys goes among the block's keys of the same digit
// (`rank`), and the block's count of each digit (s.bin_total).  Item k of
// lane l of warp w is key w * 32 * IPT + 32 k + l, and ranks follow that
// order: lanes with the same digit find one another by a warp match, the
// lowest of them adds their number to the warp's count.
template <int IPT>
__device__ __forceinline__ void block_ranks(SortShared& s, const uint32_t (&digit)[IPT], int bins,
                                            uint32_t (&rank)[IPT]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int b = lane; b < bins; b += 32) s.warp_bin[warp][b] = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const uint32_t same = __match_any_sync(0xffffffffu, digit[k]);
        const uint32_t before = s.warp_bin[warp][digit[k]];
        const int below = __popc(same & ((1u << lane) - 1u));
        rank[k] = before + below;
        __syncwarp();
        if (below == 0) s.warp_bin[warp][digit[k]] = static_cast<uint16_t>(before + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < bins) {
        uint32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = s.warp_bin[w][threadIdx.x];
            s.warp_bin[w][threadIdx.x] = static_cast<uint16_t>(sum);
            sum += c;
        }
        s.bin_total[threadIdx.x] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < IPT; ++k) rank[k] += s.warp_bin[warp][digit[k]];
}

// start[b] = sum of total[b'] over b' < b (bins <= kSortMaxBins <= the block).
__device__ __forceinline__ void bin_starts(SortShared& s, const uint32_t* total, uint32_t* start, int bins) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t mine = static_cast<int>(threadIdx.x) < bins ? total[threadIdx.x] : 0u;
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s.scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        uint32_t v = s.scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        s.scan[lane] = v;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < bins) start[threadIdx.x] = incl - mine + (warp > 0 ? s.scan[warp - 1] : 0u);
    __syncthreads();
}

// Up to kSortSmall tokens: one block, every pass in shared memory.  The
// gradient kernel may start at once: what it does before it waits for this
// one (zeroing rows) needs nothing from here.
__global__ void __launch_bounds__(kSortThreads) embed_sort_small_kernel(const SortArgs a) {
    let_next();
    extern __shared__ __align__(16) unsigned char raw[];
    SortShared& s = *reinterpret_cast<SortShared*>(raw);
    uint32_t* skey = reinterpret_cast<uint32_t*>(raw + sizeof(SortShared));
    uint32_t* sval = skey + kSortSmall;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < a.ncounters; i += kSortThreads) a.counters[i] = 0u;
    uint32_t key[kSortSmallItems], val[kSortSmallItems];
#pragma unroll
    for (int k = 0; k < kSortSmallItems; ++k) {
        const int i = warp * 32 * kSortSmallItems + 32 * k + lane;
        key[k] = i < a.N ? sort_key(a, a.ids[i]) : 0xFFFFFFFFu;  // past the end: sorts last
        val[k] = static_cast<uint32_t>(i);
    }
    const int bins = 1 << a.bits;
    for (int p = 0; p < a.passes; ++p) {
        uint32_t digit[kSortSmallItems], rank[kSortSmallItems];
#pragma unroll
        for (int k = 0; k < kSortSmallItems; ++k) digit[k] = (key[k] >> (p * a.bits)) & (bins - 1);
        block_ranks(s, digit, bins, rank);
        bin_starts(s, s.bin_total, s.bin_start, bins);
#pragma unroll
        for (int k = 0; k < kSortSmallItems; ++k) {
            const uint32_t at = s.bin_start[digit[k]] + rank[k];
            skey[at] = key[k];
            sval[at] = val[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSortSmallItems; ++k) {
            const int i = warp * 32 * kSortSmallItems + 32 * k + lane;
            key[k] = skey[i];
            val[k] = sval[i];
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kSortSmallItems; ++k) {
        const int i = warp * 32 * kSortSmallItems + 32 * k + lane;
        if (i < a.N) {
            (a.passes & 1 ? a.key[1] : a.key[0])[i] = key[k];
            (a.passes & 1 ? a.val[1] : a.val[0])[i] = val[k];
        }
    }
}

// More tokens: tiles of kSortTile.  First the digit counts of every tile for
// pass 0 (and zeros for the other passes), then one scatter a pass; a scatter
// counts the next pass's digits by the tile each key lands in (whole numbers:
// their order does not matter).
__global__ void __launch_bounds__(kSortThreads) embed_sort_count_kernel(const SortArgs a) {
    let_next();
    __shared__ uint32_t cnt[kSortMaxBins];
    const int bins = 1 << a.bits, tile = blockIdx.x;
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
        cnt[b] = 0u;
        for (int p = 1; p < a.passes; ++p) a.hist[(static_cast<size_t>(p) * a.ntiles + tile) * bins + b] = 0u;
    }
    for (int i = tile * kSortThreads + threadIdx.x; i < a.ncounters; i += gridDim.x * kSortThreads) a.counters[i] = 0u;
    __syncthreads();
    for (int k = 0; k < kSortTileItems; ++k) {
        const long long i = static_cast<long long>(tile) * kSortTile + k * kSortThreads + threadIdx.x;
        if (i < a.N) {
            const uint32_t key = sort_key(a, a.ids[i]);
            atomicAdd(&cnt[key & (bins - 1)], 1u);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) a.hist[static_cast<size_t>(tile) * bins + b] = cnt[b];
}

// Pass p: reads the ids (p = 0) or key/val[p & 1], writes key/val[(p + 1) & 1].
__global__ void __launch_bounds__(kSortThreads) embed_sort_scatter_kernel(const SortArgs a, int p) {
    extern __shared__ __align__(16) unsigned char raw[];
    SortShared& s = *reinterpret_cast<SortShared*>(raw);
    const int bins = 1 << a.bits, tile = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    let_next();
    wait_prior();
    const bool last = p == a.passes - 1;
    const uint32_t *skey = p & 1 ? a.key[1] : a.key[0], *sval = p & 1 ? a.val[1] : a.val[0];
    uint32_t *dkey = p & 1 ? a.key[0] : a.key[1], *dval = p & 1 ? a.val[0] : a.val[1];
    uint32_t key[kSortTileItems], val[kSortTileItems], digit[kSortTileItems], rank[kSortTileItems];
#pragma unroll
    for (int k = 0; k < kSortTileItems; ++k) {
        const long long i = static_cast<long long>(tile) * kSortTile + warp * 32 * kSortTileItems + 32 * k + lane;
        const bool in = i < a.N;
        if (p == 0) {
            key[k] = in ? sort_key(a, a.ids[i]) : 0xFFFFFFFFu;
            val[k] = static_cast<uint32_t>(i);
        } else {
            key[k] = in ? skey[i] : 0xFFFFFFFFu;
            val[k] = in ? sval[i] : 0u;
        }
        digit[k] = (key[k] >> (p * a.bits)) & (bins - 1);
    }
    // this tile's start in each bin, and the bins' totals
    uint32_t before = 0u, total = 0u;
    if (static_cast<int>(threadIdx.x) < bins) {
        const uint32_t* h = a.hist + static_cast<size_t>(p) * a.ntiles * bins + threadIdx.x;
#pragma unroll 8
        for (int t = 0; t < a.ntiles; ++t) {
            const uint32_t c = h[static_cast<size_t>(t) * bins];
            if (t < tile) before += c;
            total += c;
        }
        s.bin_total[threadIdx.x] = total;
    }
    __syncthreads();
    bin_starts(s, s.bin_total, s.bin_start, bins);
    if (static_cast<int>(threadIdx.x) < bins) s.bin_start[threadIdx.x] += before;
    __syncthreads();
    block_ranks(s, digit, bins, rank);
#pragma unroll
    for (int k = 0; k < kSortTileItems; ++k) {
        const long long i = static_cast<long long>(tile) * kSortTile + warp * 32 * kSortTileItems + 32 * k + lane;
        if (i >= a.N) continue;
        const uint32_t at = s.bin_start[digit[k]] + rank[k];
        dkey[at] = key[k];
        dval[at] = val[k];
        if (!last)
            atomicAdd(a.hist + (static_cast<size_t>(p + 1) * a.ntiles + at / kSortTile) * bins +
                          ((key[k] >> ((p + 1) * a.bits)) & (bins - 1)),
                      1u);
    }
}

// ----------------------------------------------------------------------------- the gradient

// A "worker" is kEmbThreads threads or, where a row has fewer 16-byte vectors,
// as many warps as it has 32s of them; it writes `rows_w` consecutive rows of
// dE.  It finds its rows' tokens by a search of the sorted ids, writes zeros
// up to the next id that occurs, and sums that id's tokens in registers.
//
// An id that takes many tokens (padding, a space) would keep one worker busy
// long after the others: the sorted tokens are therefore also cut into chunks
// of kEmbChunk, and a chunk that lies wholly within one id is summed by a
// block of its own into `part`.  Whoever is last of an id's chunk blocks and
// its row's worker (a counter for each slice of columns) adds up the tokens
// before the first whole chunk, the chunks' sums and the tokens behind the
// last one, in that order: the same sum whoever is last.
//
// The first `first_wave` row blocks write zeros over all their rows before
// they wait for the sort, which keeps the memory busy while one block sorts;
// the few rows with tokens are written a second time.
constexpr int kEmbChunk = 64;
constexpr int kEmbBlockBytes = 65536;  // of dE a row block writes
constexpr int kEmbBlocksPerSm = 4;     // row blocks of the first wave

struct EmbBwdArgs {
    const uint32_t* key;  // sorted ids [N], V for tokens that take no part
    const uint32_t* val;  // their tokens
    const __nv_bfloat16* dOut;
    void* dE;
    float* part;         // [N / kEmbChunk][8 nv]
    uint32_t* counters;  // [N / kEmbChunk][slices], zero
    int N, V, nv;
    int slices;      // of kEmbThreads vectors
    int log_worker;  // threads of a worker: 32 .. kEmbThreads
    int rows_w;
    int first_wave;
    float scale;
};

// The first place in sorted key[lo, hi) that is not below x: each step, the 32
// lanes of the warp probe the range at once.
__device__ __forceinline__ int lower_bound(const uint32_t* key, int lo, int hi, uint32_t x) {
    const int lane = threadIdx.x & 31;
    while (hi - lo > 32) {
        const int step = (hi - lo + 31) >> 5;
        const int at = lo + (lane + 1) * step - 1;  // N is at most 2^30
        const unsigned below = __ballot_sync(0xffffffffu, at < hi && key[at] < x);
        lo += __popc(below) * step;
        hi = min(lo + step, hi);
    }
    return lo + __popc(__ballot_sync(0xffffffffu, lo + lane < hi && key[lo + lane] < x));
}

// acc += the rows of tokens val[from, to), vector j of each.
__device__ __forceinline__ void add_tokens(const EmbBwdArgs& a, int from, int to, int j, float (&acc)[8]) {
    constexpr int U = 4;
    const uint4* d = reinterpret_cast<const uint4*>(a.dOut) + j;
#pragma unroll 1
    for (int p = from; p < to; p += U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = p + u < to ? load_once(d + static_cast<long long>(a.val[p + u]) * a.nv) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[8];
            widen8(v[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += f[i];
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store_grad(const EmbBwdArgs& a, long long row, int j, float (&acc)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= a.scale;
    const long long at = row * a.nv + j;
    if (F32) {
        float4* o = reinterpret_cast<float4*>(a.dE) + 2 * at;
        o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    } else {
        reinterpret_cast<uint4*>(a.dE)[at] = round8(acc);
    }
}

// Slice `sl` of the row of an id with tokens [s, e) and whole chunks [c0, c1).
template <bool F32>
__device__ __noinline__ void finish_slice(const EmbBwdArgs& a, uint32_t row, int s, int e, int c0, int c1, int sl,
                                             int tid, int threads) {
    const int end = min(a.nv, (sl + 1) * kEmbThreads);
    for (int j = sl * kEmbThreads + tid; j < end; j += threads) {
        float acc[8] = {};
        add_tokens(a, s, c0 * kEmbChunk, j, acc);
        const float4* p = reinterpret_cast<const float4*>(a.part) + 2 * (static_cast<long long>(c0) * a.nv + j);
        constexpr int U = 4;
#pragma unroll 1
        for (int c = c0; c < c1; c += U) {
            float4 v[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4* q = p + 2 * static_cast<long long>(c - c0 + u) * a.nv;
                v[u][0] = c + u < c1 ? __ldcg(q) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                v[u][1] = c + u < c1 ? __ldcg(q + 1) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                acc[0] += v[u][0].x, acc[1] += v[u][0].y, acc[2] += v[u][0].z, acc[3] += v[u][0].w;
                acc[4] += v[u][1].x, acc[5] += v[u][1].y, acc[6] += v[u][1].z, acc[7] += v[u][1].w;
            }
        }
        add_tokens(a, c1 * kEmbChunk, e, j, acc);
        store_grad<F32>(a, row, j, acc);
    }
}

// One chunk and slice of columns: its sum, and the row if it comes last.
template <bool F32>
__device__ void chunk_block(const EmbBwdArgs& a, int chunk, int sl) {
    const int from = chunk * kEmbChunk;
    const uint32_t id = a.key[from];
    if (id >= static_cast<uint32_t>(a.V) || a.key[from + kEmbChunk - 1] != id) return;
    const int j = sl * kEmbThreads + threadIdx.x;
    if (j < a.nv) {
        float acc[8] = {};
        add_tokens(a, from, from + kEmbChunk, j, acc);
        float4* p = reinterpret_cast<float4*>(a.part) + 2 * (static_cast<long long>(chunk) * a.nv + j);
        __stcg(p, make_float4(acc[0], acc[1], acc[2], acc[3]));
        __stcg(p + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
    }
    const int s = lower_bound(a.key, 0, from, id), e = lower_bound(a.key, from, a.N, id + 1u);
    const int c0 = (s + kEmbChunk - 1) / kEmbChunk, c1 = e / kEmbChunk;
    __shared__ uint32_t arrived;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) arrived = atomicAdd(a.counters + static_cast<long long>(c0) * a.slices + sl, 1u);
    __syncthreads();
    if (arrived != static_cast<uint32_t>(c1 - c0)) return;  // c1 - c0 chunks and the row's worker
    __threadfence();
    finish_slice<F32>(a, id, s, e, c0, c1, sl, threadIdx.x, kEmbThreads);
}

template <bool F32>
__global__ void __launch_bounds__(kEmbThreads, kEmbBlocksPerSm) embed_bwd_kernel(const EmbBwdArgs a) {
    // block order: the first wave of row blocks, the chunks, the other row blocks
    const int nchunk_blocks = a.N / kEmbChunk * a.slices;
    int rb = blockIdx.x;
    if (rb >= a.first_wave) {
        rb -= a.first_wave;
        if (rb < nchunk_blocks) {
            wait_prior();
            chunk_block<F32>(a, rb / a.slices, rb % a.slices);
            return;
        }
        rb += a.first_wave - nchunk_blocks;
    }
    const int threads = 1 << a.log_worker, workers = kEmbThreads >> a.log_worker;
    const int tid = threadIdx.x & (threads - 1), w = threadIdx.x >> a.log_worker;
    const long long first = (static_cast<long long>(rb) * workers + w) * a.rows_w;
    const long long r0 = min(first, static_cast<long long>(a.V)), r1 = min(first + a.rows_w, static_cast<long long>(a.V));
    constexpr int kOut = F32 ? 2 : 1;  // 16-byte stores of a vector
    uint4* out = static_cast<uint4*>(a.dE);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool early = rb < a.first_wave;
    if (early)
        for (long long i = r0 * a.nv * kOut + tid; i < r1 * a.nv * kOut; i += threads) out[i] = zero;
    wait_prior();
    if (early) __threadfence();  // before this worker counts itself in at a row that others may write
    __syncthreads();
    if (r0 >= r1) return;
    int p = lower_bound(a.key, 0, a.N, static_cast<uint32_t>(r0));
    const int hi = lower_bound(a.key, p, a.N, static_cast<uint32_t>(r1));
    long long r = r0;
    while (r < r1) {
        const long long next = p < hi ? static_cast<long long>(a.key[p]) : r1;
        if (!early)
            for (long long i = r * a.nv * kOut + tid; i < next * a.nv * kOut; i += threads) out[i] = zero;
        if (next >= r1) break;
        const uint32_t id = static_cast<uint32_t>(next);
        const int s = p, e = lower_bound(a.key, p, hi, id + 1u);
        const int c0 = (s + kEmbChunk - 1) / kEmbChunk, c1 = e / kEmbChunk;
        if (c0 < c1) {
            // the chunks' blocks write this row, or this worker does if it comes last
            for (int sl = 0; sl < a.slices; ++sl) {
                __shared__ uint32_t seen[kEmbThreads / 32];  // the worker's threads learn one count
                asm volatile("bar.sync %0, %1;" ::"r"(w + 1), "r"(threads) : "memory");
                if (tid == 0) seen[w] = atomicAdd(a.counters + static_cast<long long>(c0) * a.slices + sl, 1u);
                asm volatile("bar.sync %0, %1;" ::"r"(w + 1), "r"(threads) : "memory");
                if (seen[w] == static_cast<uint32_t>(c1 - c0)) {
                    __threadfence();
                    finish_slice<F32>(a, id, s, e, c0, c1, sl, tid, threads);
                }
            }
        } else {
            for (int j = tid; j < a.nv; j += threads) {
                float acc[8] = {};
                add_tokens(a, s, e, j, acc);
                store_grad<F32>(a, next, j, acc);
            }
        }
        p = e;
        r = next + 1;
    }
}

}  // namespace step
}  // namespace lmlp
