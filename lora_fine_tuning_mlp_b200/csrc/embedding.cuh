// Token embedding lookup with scaling, and its gradient by sorted tokens
// (include/lora_embedding.h).
//
//   out[t] = bf16(scale E[id_t]),    dE[v] = scale sum_{t: id_t = v} dOut[t]
//
// Both passes only move bytes: the lookup reads a row and writes a row for
// each token; the gradient reads each token's row of dOut once and writes
// every row of dE, most of them zeros (a 128K vocabulary against a few
// thousand tokens).  So that no row is read back to be added to, and no
// atomic's order shows in a sum, the tokens are sorted by id first (stable
// radix sort): the tokens of an id then lie next to each other, in token
// order, and whoever writes row v sums them in registers.  The sort takes one
// multiprocessor or a few; zeros are written everywhere meanwhile, and the few
// rows with tokens a second time.
//
// On a B200: 32768 rows of 2048 looked up 31 us (8.6 TB/s of reads and writes,
// the frequent rows from L2); the gradient of 128256 x 4096 bf16 for 4096 tokens
// 167 us (141 of them the zeros), of 256000 x 2048 fp32 for 16001 tokens 320 us.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "vec8.cuh"

namespace lmlp {
namespace step {

// ----------------------------------------------------------------------------- lookup

constexpr int kEmbThreads = 256;

// A row is walked by `tpr` threads (a power of two, at most the block), 16
// bytes at a time, up to kEmbLoads of them in flight a thread (one made the
// lookup above 60 us); a block holds kEmbThreads / tpr rows.
constexpr int kEmbLoads = 4;
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
        if (lane == 0) atomicMin(a.status, kStatusBad);
        for (int j = lane; j < a.nv; j += step) o[j] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        return;
    }
    const uint4* e = reinterpret_cast<const uint4*>(a.E) + id * a.nv;
    constexpr int U = kEmbLoads;
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
            __stcs(o + j0 + u * step, round8(f));
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
constexpr int kSortSmall = kSortThreads * 8;  // tokens that one block sorts

struct SortArgs {
    const long long* ids;
    int N;
    int V;
    long long padding;  // < 0: none
    int bits;           // digit width
    int passes;
    int ntiles;
    int tile;           // tokens of a tile: kSortThreads, once or four times
    uint32_t *key[2], *val[2];  // [N] each; the result is in key[passes & 1], val[passes & 1]
    uint32_t* hist;             // [passes][ntiles][bins]
    uint32_t* counters;         // zeroed here for the gradient kernel
    int ncounters;
    int* status;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, long long id) {
    if (id == a.padding && a.padding >= 0) return static_cast<uint32_t>(a.V);
    if (id < 0 || id >= a.V) {
        atomicMin(a.status, kStatusBad);
        return static_cast<uint32_t>(a.V);
    }
    return static_cast<uint32_t>(id);
}

struct SortShared {
    uint16_t warp_bin[kSortWarps][kSortMaxBins];  // counts, then each warp's start within its bin
    uint32_t bin_total[kSortMaxBins];
    uint32_t bin_start[kSortMaxBins];
    uint32_t bin_before[kSortMaxBins];
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
template <int IPT>
__global__ void __launch_bounds__(kSortThreads) embed_sort_small_kernel(const SortArgs a) {
    let_next();
    extern __shared__ __align__(16) unsigned char raw[];
    SortShared& s = *reinterpret_cast<SortShared*>(raw);
    uint32_t* skey = reinterpret_cast<uint32_t*>(raw + sizeof(SortShared));
    uint32_t* sval = skey + kSortThreads * IPT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < a.ncounters; i += kSortThreads) a.counters[i] = 0u;
    uint32_t key[IPT], val[IPT];
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = warp * 32 * IPT + 32 * k + lane;
        key[k] = i < a.N ? sort_key(a, a.ids[i]) : 0xFFFFFFFFu;  // past the end: sorts last
        val[k] = static_cast<uint32_t>(i);
    }
    const int bins = 1 << a.bits;
    for (int p = 0; p < a.passes; ++p) {
        uint32_t digit[IPT], rank[IPT];
#pragma unroll
        for (int k = 0; k < IPT; ++k) digit[k] = (key[k] >> (p * a.bits)) & (bins - 1);
        block_ranks(s, digit, bins, rank);
        bin_starts(s, s.bin_total, s.bin_start, bins);
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const uint32_t at = s.bin_start[digit[k]] + rank[k];
            skey[at] = key[k];
            sval[at] = val[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < IPT; ++k) {
            const int i = warp * 32 * IPT + 32 * k + lane;
            key[k] = skey[i];
            val[k] = sval[i];
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const int i = warp * 32 * IPT + 32 * k + lane;
        if (i < a.N) {
            (a.passes & 1 ? a.key[1] : a.key[0])[i] = key[k];
            (a.passes & 1 ? a.val[1] : a.val[0])[i] = val[k];
        }
    }
}

// More tokens: tiles, one to a block.  First the digit counts of every tile for
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
    for (int k = threadIdx.x; k < a.tile; k += kSortThreads) {
        const long long i = static_cast<long long>(tile) * a.tile + k;
        if (i < a.N) {
            const uint32_t key = sort_key(a, a.ids[i]);
            atomicAdd(&cnt[key & (bins - 1)], 1u);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) a.hist[static_cast<size_t>(tile) * bins + b] = cnt[b];
}

// Pass p: reads the ids (p = 0) or key/val[p & 1], writes key/val[(p + 1) & 1].
template <int IPT>
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
    uint32_t key[IPT], val[IPT], digit[IPT], rank[IPT];
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const long long i = static_cast<long long>(tile) * (kSortThreads * IPT) + warp * 32 * IPT + 32 * k + lane;
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
    // this tile's start in each bin, and the bins' totals; the halves of the
    // block take every other tile
    const int bin = threadIdx.x & (kSortMaxBins - 1), half = threadIdx.x / kSortMaxBins;
    uint32_t before = 0u, total = 0u;
    if (bin < bins) {
        const uint32_t* h = a.hist + static_cast<size_t>(p) * a.ntiles * bins + bin;
#pragma unroll 16
        for (int t = half; t < a.ntiles; t += 2) {
            const uint32_t c = h[static_cast<size_t>(t) * bins];
            if (t < tile) before += c;
            total += c;
        }
        if (half == 1) s.bin_total[bin] = total, s.bin_before[bin] = before;
    }
    __syncthreads();
    if (half == 0 && bin < bins) s.bin_total[bin] += total;
    __syncthreads();
    bin_starts(s, s.bin_total, s.bin_start, bins);
    if (half == 0 && bin < bins) s.bin_start[bin] += before + s.bin_before[bin];
    __syncthreads();
    block_ranks(s, digit, bins, rank);
#pragma unroll
    for (int k = 0; k < IPT; ++k) {
        const long long i = static_cast<long long>(tile) * (kSortThreads * IPT) + warp * 32 * IPT + 32 * k + lane;
        if (i >= a.N) continue;
        const uint32_t at = s.bin_start[digit[k]] + rank[k];
        dkey[at] = key[k];
        dval[at] = val[k];
        if (!last)
            atomicAdd(a.hist + (static_cast<size_t>(p + 1) * a.ntiles + at / (kSortThreads * IPT)) * bins +
                          ((key[k] >> ((p + 1) * a.bits)) & (bins - 1)),
                      1u);
    }
}

// ----------------------------------------------------------------------------- the gradient

// Zeros for all of dE, while the tokens are sorted: many small blocks, which
// the hardware starts in the order of their addresses, write 7.4 TB/s; blocks
// that stay and take several parts, wherever these lie, 6.3.
constexpr int kZeroThreads = 256;
constexpr int kZeroStores = 4;  // of 16 bytes, a thread
constexpr int kZeroBlock = kZeroThreads * kZeroStores;

__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(uint4* out, long long n) {
    let_next();
    const long long i = static_cast<long long>(blockIdx.x) * kZeroBlock + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kZeroStores; ++k)
        if (i + k * kZeroThreads < n) __stcs(out + i + k * kZeroThreads, make_uint4(0u, 0u, 0u, 0u));
    // nothing here needs the sort, but who waits for this kernel relies on it
    if (blockIdx.x == gridDim.x - 1) wait_prior();
}

// A "worker" is the power of two of threads, 32 .. kEmbThreads, that has two
// vectors of a row each, at most (or as often as the row asks for it).  Worker
// p looks at place p of the sorted tokens.  Where an id begins, it sums that
// id's tokens in registers and writes the row.
//
// An id that takes many tokens (padding, a space) would keep one worker busy
// long after the others: the sorted tokens are therefore also cut into chunks
// of kEmbChunk, and a chunk that lies wholly within one id is summed into
// `part`, a block for each slice of the row: groups of its threads, two vectors
// a thread, take a share of the tokens each and the shares are added up in
// order.  Whichever of an id's chunks is last (a counter for each slice) adds up
// the tokens before the first whole chunk, the chunks' sums and the tokens
// behind the last one, shared out in the same way: the same sum whichever is
// last.
constexpr int kEmbChunk = 32;

struct EmbBwdArgs {
    const uint32_t* key;  // sorted ids [N], V for tokens that take no part
    const uint32_t* val;  // their tokens
    const __nv_bfloat16* dOut;
    void* dE;
    float* part;         // [N / kEmbChunk][8 nv]
    uint32_t* counters;  // [N / kEmbChunk][slices], zero
    int N, V, nv;
    int slices;
    int log_group;   // threads of a group: half a slice's vectors
    int log_worker;
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

// acc[h] += the rows of tokens val[from, to), vector j + h * step of each.
__device__ __forceinline__ void add_tokens(const EmbBwdArgs& a, int from, int to, int j, int step,
                                           float (&acc)[2][8]) {
    constexpr int U = 4;
    const uint4* d = reinterpret_cast<const uint4*>(a.dOut) + j;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool first = j < a.nv, second = j + step < a.nv;
#pragma unroll 1
    for (int p = from; p < to; p += U) {
        uint4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint4* row = d + static_cast<long long>(p + u < to ? a.val[p + u] : 0u) * a.nv;
            v[u][0] = p + u < to && first ? load_once(row) : zero;
            v[u][1] = p + u < to && second ? load_once(row + step) : zero;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[8];
                widen8(v[u][h], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[h][i] += f[i];
            }
    }
}

template <bool F32>
__device__ __forceinline__ void store_grad(const EmbBwdArgs& a, uint32_t row, int j, int step, float (&acc)[2][8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (j + h * step >= a.nv) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[h][i] *= a.scale;
        const long long at = static_cast<long long>(row) * a.nv + j + h * step;
        if (F32) {
            float4* o = reinterpret_cast<float4*>(a.dE) + 2 * at;
            __stcs(o, make_float4(acc[h][0], acc[h][1], acc[h][2], acc[h][3]));
            __stcs(o + 1, make_float4(acc[h][4], acc[h][5], acc[h][6], acc[h][7]));
        } else {
            __stcs(reinterpret_cast<uint4*>(a.dE) + at, round8(acc[h]));
        }
    }
}

// The groups' shares, added up in order by the first.
__device__ __forceinline__ void join_shares(int group, float (&acc)[2][8]) {
    __shared__ float shares[2][8][kEmbThreads];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) shares[h][i][threadIdx.x] = acc[h][i];
    __syncthreads();
    if (static_cast<int>(threadIdx.x) >= group) return;
    for (int t = threadIdx.x + group; t < kEmbThreads; t += group)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[h][i] += shares[h][i][t];
}

// One chunk and slice: its sum, and the row's if it comes last.
template <bool F32>
__device__ void chunk_block(const EmbBwdArgs& a, int chunk, int sl) {
    const int from = chunk * kEmbChunk;
    const uint32_t id = a.key[from];
    if (id >= static_cast<uint32_t>(a.V) || a.key[from + kEmbChunk - 1] != id) return;
    const int group = 1 << a.log_group, groups = kEmbThreads >> a.log_group, share = kEmbChunk / groups;
    const int g = threadIdx.x >> a.log_group;
    const int j = sl * 2 * group + (threadIdx.x & (group - 1));
    float acc[2][8] = {};
    add_tokens(a, from + g * share, from + (g + 1) * share, j, group, acc);
    join_shares(group, acc);
    if (g == 0)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (j + h * group < a.nv) {
                float4* p = reinterpret_cast<float4*>(a.part) + 2 * (static_cast<long long>(chunk) * a.nv + j + h * group);
                __stcg(p, make_float4(acc[h][0], acc[h][1], acc[h][2], acc[h][3]));
                __stcg(p + 1, make_float4(acc[h][4], acc[h][5], acc[h][6], acc[h][7]));
            }
    const int s = lower_bound(a.key, 0, from, id), e = lower_bound(a.key, from, a.N, id + 1u);
    const int c0 = (s + kEmbChunk - 1) / kEmbChunk, c1 = e / kEmbChunk;
    __shared__ uint32_t arrived;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) arrived = atomicAdd(a.counters + static_cast<long long>(c0) * a.slices + sl, 1u);
    __syncthreads();
    if (arrived != static_cast<uint32_t>(c1 - c0 - 1)) return;
    __threadfence();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[h][i] = 0.0f;
    const int before = c0 * kEmbChunk, behind = c1 * kEmbChunk;
    add_tokens(a, min(s + g * share, before), min(s + (g + 1) * share, before), j, group, acc);
    const int each = (c1 - c0 + groups - 1) / groups;
    const int first = min(c0 + g * each, c1), last = min(first + each, c1);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    constexpr int U = 2;
#pragma unroll 1
    for (int c = first; c < last; c += U) {
        float4 v[U][2][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool in = c + u < last && j + h * group < a.nv;
                const float4* q =
                    reinterpret_cast<const float4*>(a.part) + 2 * (static_cast<long long>(c + u) * a.nv + j + h * group);
                v[u][h][0] = in ? __ldcg(q) : zero;
                v[u][h][1] = in ? __ldcg(q + 1) : zero;
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    acc[h][4 * k] += v[u][h][k].x, acc[h][4 * k + 1] += v[u][h][k].y;
                    acc[h][4 * k + 2] += v[u][h][k].z, acc[h][4 * k + 3] += v[u][h][k].w;
                }
    }
    add_tokens(a, min(behind + g * share, e), min(behind + (g + 1) * share, e), j, group, acc);
    join_shares(group, acc);
    if (g == 0) store_grad<F32>(a, id, j, group, acc);
}

template <bool F32>
__global__ void __launch_bounds__(kEmbThreads, 4) embed_bwd_kernel(const EmbBwdArgs a) {
    wait_prior();
    const int chunk_blocks = a.N / kEmbChunk * a.slices;
    if (static_cast<int>(blockIdx.x) < chunk_blocks) {
        chunk_block<F32>(a, blockIdx.x / a.slices, blockIdx.x % a.slices);
        return;
    }
    const int threads = 1 << a.log_worker, lane = threadIdx.x & 31;
    const long long p = (static_cast<long long>(blockIdx.x - chunk_blocks) << (8 - a.log_worker)) +
                        (threadIdx.x >> a.log_worker);
    static_assert(kEmbThreads == 1 << 8, "the workers of a block");
    if (p >= a.N) return;
    const int s = static_cast<int>(p);
    const uint32_t id = a.key[s];
    if (id >= static_cast<uint32_t>(a.V) || (s > 0 && a.key[s - 1] == id)) return;
    // the id's end, as far as it can lie without a whole chunk
    int n = 0;
    for (; n < 2 * kEmbChunk; n += 32) {
        const unsigned same = __ballot_sync(0xffffffffu, s + n + lane < a.N && a.key[min(s + n + lane, a.N - 1)] == id);
        if (same != 0xffffffffu) {
            n += __ffs(~same) - 1;
            break;
        }
    }
    const int e = s + n;
    if ((s + kEmbChunk - 1) / kEmbChunk < e / kEmbChunk) return;  // its chunks' blocks write the row
    for (int j = threadIdx.x & (threads - 1); j < a.nv; j += 2 * threads) {
        float acc[2][8] = {};
        add_tokens(a, s, e, j, threads, acc);
        store_grad<F32>(a, id, j, threads, acc);
    }
}

}  // namespace step
}  // namespace lmlp
