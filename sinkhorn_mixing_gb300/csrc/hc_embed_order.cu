// hc_embed_order.cu -- tokens in order of their ids, those of one id by position, and
// where each id's tokens are.  Two ways to the same order, by the number of tokens:
//   up to 4,096     k_rank: each token counts the tokens before it, one launch
//   above           a radix sort: k_sort_count and k_sort_move for each digit, then
//                   k_embed_places
// Both are latency: a few hundred KB that stay in L2.
#include "hc_common.cuh"
#include "hc_embed_order.h"

namespace hc {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kTile = 1024;  // tokens a block of the radix sort has at a time
constexpr int kItems = kTile / kSortThreads;
constexpr int kSortBlocks = 304;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;  // as many as kSortThreads

constexpr int kRankTokens = 4096;
constexpr int kRankRows = 8192;  // table rows whose presence a block of k_rank notes
constexpr int kRankThreads = 1024;
constexpr int kRankWarps = kRankThreads / 32;

int bits_of(int64_t v) {  // of the numbers 0 .. v
    int b = 1;
    while ((v >> b) != 0) ++b;
    return b;
}

// An id as it is ordered: those outside the table come behind it, as `vocab`.
template <typename ID>
__device__ __forceinline__ uint32_t row_of(const ID *ids, int64_t i, int64_t vocab) {
    const int64_t id = (int64_t)__ldg(ids + i);
    return (uint32_t)(id >= 0 && id < vocab ? id : vocab);
}

// Few tokens: a token's place is the number of tokens with a smaller id, and of those
// before it with its own.  A block has 32 of them, one a lane, and all ids in shared
// memory; its warps share the comparisons.  64 tokens into 32,768 rows of 5120: 109 us
// for the whole call, with the sort below 118; 1,500 of 1 x 1000 34 and 44; at 8,192
// tokens the n^2 comparisons lose, 48 and 40.  A block also notes which of kRankRows
// rows of the table are present.
template <typename ID>
__global__ void __launch_bounds__(kRankThreads)
    k_rank(int n, int64_t vocab, const ID *__restrict__ ids, uint2 *__restrict__ sorted,
           uint32_t *__restrict__ longs_count, uint32_t *__restrict__ present,
           uint32_t *__restrict__ start, uint32_t *__restrict__ end) {
    __shared__ __align__(16) uint32_t id[kRankTokens];
    __shared__ uint32_t bits[kRankRows / 32], count[kRankWarps][3][32];
    griddep_wait_then_release();
    if (blockIdx.x == 0 && threadIdx.x == 0) *longs_count = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * kRankRows;
    for (int i = threadIdx.x; i < kRankRows / 32; i += kRankThreads) bits[i] = 0;
    __syncthreads();
    const int padded = (n + 31) & ~31;  // places behind the last token: no id is larger
    uint32_t own[kRankTokens / kRankThreads];
#pragma unroll
    for (int k = 0; k < kRankTokens / kRankThreads; ++k) {
        const int i = threadIdx.x + k * kRankThreads;
        own[k] = i < n ? row_of(ids, i, vocab) : 0xFFFFFFFFu;
    }
#pragma unroll
    for (int k = 0; k < kRankTokens / kRankThreads; ++k) {
        const int i = threadIdx.x + k * kRankThreads;
        if (i < padded) id[i] = own[k];
        if (own[k] < vocab && own[k] >= row0 && own[k] < row0 + kRankRows)
            atomicOr(&bits[(own[k] - row0) >> 5], 1u << (own[k] & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kRankRows / 32; i += kRankThreads)
        if (row0 + i * 32 < vocab) present[row0 / 32 + i] = bits[i];
    if ((int64_t)blockIdx.x * 32 >= n) return;
    const int t0 = blockIdx.x * 32, t = t0 + lane;
    const uint32_t mine = id[t];
    // groups of 32 tokens, the block's own among them
    uint32_t less = 0, same = 0, before = 0;
    for (int g = warp * 32; g < padded; g += kRankThreads) {
        uint32_t here = 0;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            const uint4 o = *reinterpret_cast<const uint4 *>(&id[g + k]);
            less += (o.x < mine) + (o.y < mine) + (o.z < mine) + (o.w < mine);
            here += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
        }
        same += here;
        if (g < t0) before += here;
        if (g == t0)
            for (int k = 0; k < lane; ++k) before += id[g + k] == mine;
    }
    count[warp][0][lane] = less, count[warp][1][lane] = same, count[warp][2][lane] = before;
    __syncthreads();
    if (warp != 0 || t >= n) return;
#pragma unroll
    for (int w = 1; w < kRankWarps; ++w)
        less += count[w][0][lane], same += count[w][1][lane], before += count[w][2][lane];
    sorted[less + before] = make_uint2(mine, (uint32_t)t);
    if (mine < vocab && before == 0) {
        start[mine] = less;
        end[mine] = less + same;
    }
}

// The place of each lane's token among the warp's with the same digit: `cnt` holds the
// warp's tokens with each digit so far, and takes the new ones in.
__device__ __forceinline__ uint32_t rank_in_warp(bool in, uint32_t digit, uint32_t *cnt) {
    const int lane = threadIdx.x & 31;
    // lanes without a token have a group of their own
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, in ? digit : 0xFFFFFFFFu);
    const uint32_t below = same & ((1u << lane) - 1u);
    const uint32_t had = in ? cnt[digit] : 0;
    __syncwarp();
    if (in && below == 0) cnt[digit] = had + __popc(same);
    __syncwarp();
    return had + __popc(below);
}

// Exclusive sums of v over the block's threads.
__device__ __forceinline__ uint32_t exclusive_sum(uint32_t v, uint32_t *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, s, off);
        if (lane >= off) s += o;
    }
    if (lane == 31) red[warp] = s;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) before += w < warp ? red[w] : 0;
    return before + s - v;
}

// Where a pass of the radix sort reads: the ids themselves, or the pass before.
template <typename ID>
struct FromIds {
    const ID *ids;
    int64_t vocab;
    __device__ __forceinline__ uint2 get(int64_t i) const {
        return make_uint2(row_of(ids, i, vocab), (uint32_t)i);
    }
};
struct FromPairs {
    const uint2 *pairs;
    __device__ __forceinline__ uint2 get(int64_t i) const { return pairs[i]; }
};

// A block's tokens in a pass: whole tiles, in order.
__device__ __forceinline__ int64_t first_token(int64_t n, int blocks, int b) {
    const int64_t tiles = (n + kTile - 1) / kTile, per = (tiles + blocks - 1) / blocks;
    const int64_t at = (int64_t)b * per * kTile;
    return at < n ? at : n;
}

// How many of a block's tokens have each digit.  The first pass also clears what
// k_embed_places adds to.  (Counting the next digit while the tokens are moved saves
// this launch, but its atomics cost as much: no size was faster.  Nor was a sort in
// the shared memory of one cluster of 16 blocks, one launch in place of five: 65,536
// tokens 53 us for the whole call, as here 45; 8,192 tokens 39 and 40.)
template <typename SRC>
__global__ void __launch_bounds__(kSortThreads)
    k_sort_count(int64_t n, SRC src, int shift, int bins, uint32_t *__restrict__ hist,
                 uint32_t *__restrict__ longs_count, uint32_t *__restrict__ present,
                 int64_t words) {
    __shared__ uint32_t cnt[kMaxBins];
    griddep_wait_then_release();
    cnt[threadIdx.x] = 0;
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < words;
         i += (int64_t)gridDim.x * kSortThreads)
        present[i] = 0;
    if (words != 0 && blockIdx.x == 0 && threadIdx.x == 0) *longs_count = 0;
    __syncthreads();
    const int64_t i1 = first_token(n, gridDim.x, blockIdx.x + 1);
    for (int64_t i = first_token(n, gridDim.x, blockIdx.x) + threadIdx.x; i < i1;
         i += kSortThreads)
        atomicAdd(&cnt[(src.get(i).x >> shift) & (bins - 1)], 1u);
    __syncthreads();
    if ((int)threadIdx.x < bins) hist[(int64_t)blockIdx.x * bins + threadIdx.x] = cnt[threadIdx.x];
}

// A block's tokens to their places in the digit's order.  A place: tokens with a
// smaller digit, then those of blocks, tiles, warps and lanes before this one.
template <typename SRC>
__global__ void __launch_bounds__(kSortThreads)
    k_sort_move(int64_t n, SRC src, int shift, int bins, const uint32_t *__restrict__ hist,
                uint2 *__restrict__ out) {
    __shared__ uint32_t cnt[kSortWarps][kMaxBins], red[kSortWarps];
    griddep_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = gridDim.x;
    const int mine = threadIdx.x;  // the digit whose places this thread counts
    uint32_t total = 0, before = 0;
    if (mine < bins) {
#pragma unroll 8
        for (int b = 0; b < blocks; ++b) {
            const uint32_t c = hist[(int64_t)b * bins + mine];
            total += c;
            before += b < (int)blockIdx.x ? c : 0;
        }
    }
    uint32_t base = exclusive_sum(total, red) + before;
    const int64_t i1 = first_token(n, blocks, blockIdx.x + 1);
    for (int64_t i0 = first_token(n, blocks, blockIdx.x); i0 < i1; i0 += kTile) {
        uint2 e[kItems];
        uint32_t rank[kItems];
        const int64_t first = i0 + warp * (32 * kItems) + lane;
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            e[k] = first + k * 32 < i1 ? src.get(first + k * 32) : make_uint2(0, 0);
        for (int i = threadIdx.x; i < kSortWarps * kMaxBins; i += kSortThreads)
            (&cnt[0][0])[i] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kItems; ++k)
            rank[k] = rank_in_warp(first + k * 32 < i1, (e[k].x >> shift) & (bins - 1), cnt[warp]);
        __syncthreads();
        if (mine < bins) {
            uint32_t c[kSortWarps];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) c[w] = cnt[w][mine];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                cnt[w][mine] = base;
                base += c[w];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            if (first + k * 32 < i1)
                out[cnt[warp][(e[k].x >> shift) & (bins - 1)] + rank[k]] = e[k];
        }
        __syncthreads();
    }
}

// First and last places of every id, and which ids are present.
__global__ void __launch_bounds__(256)
    k_embed_places(int64_t n, uint32_t vocab, const uint2 *__restrict__ sorted,
                   uint32_t *__restrict__ present, uint32_t *__restrict__ start,
                   uint32_t *__restrict__ end) {
    griddep_wait_then_release();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const uint32_t id = sorted[i].x;
    if (id == vocab) return;
    if (i == 0 || sorted[i - 1].x != id) {
        start[id] = (uint32_t)i;
        atomicOr(&present[id >> 5], 1u << (id & 31));
    }
    if (i + 1 == n || sorted[i + 1].x != id) end[id] = (uint32_t)i + 1;
}

template <typename SRC>
cudaError_t sort_pass(int64_t n, SRC src, int shift, int bins, const TokenOrder &o, uint2 *out,
                      int64_t clear_words, cudaStream_t s) {
    const int64_t tiles = (n + kTile - 1) / kTile;
    const dim3 grid((unsigned)(tiles < kSortBlocks ? tiles : kSortBlocks));
    cudaError_t e = launch_overlapped(&k_sort_count<SRC>, grid, dim3(kSortThreads), 0, s, n, src,
                                      shift, bins, o.hist, o.count, o.present, clear_words);
    if (e != cudaSuccess) return e;
    return launch_overlapped(&k_sort_move<SRC>, grid, dim3(kSortThreads), 0, s, n, src, shift, bins,
                             (const uint32_t *)o.hist, out);
}

template <typename ID>
cudaError_t order(int64_t n, int64_t vocab, const ID *ids, const TokenOrder &o, cudaStream_t s) {
    if (n <= kRankTokens) {
        const int64_t by_tokens = (n + 31) / 32, by_rows = (vocab + kRankRows - 1) / kRankRows;
        return launch_overlapped(&k_rank<ID>,
                                 dim3((unsigned)(by_tokens > by_rows ? by_tokens : by_rows)),
                                 dim3(kRankThreads), 0, s, (int)n, vocab, ids, o.sorted[0], o.count,
                                 o.present, o.start, o.end);
    }
    const int bits = bits_of(vocab), passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    const int digit = (bits + passes - 1) / passes, bins = 1 << digit;
    int to = (passes - 1) & 1;
    cudaError_t e = sort_pass(n, FromIds<ID>{ids, vocab}, 0, bins, o, o.sorted[to],
                              (vocab + 31) / 32, s);
    for (int i = 1; i < passes && e == cudaSuccess; ++i, to ^= 1)
        e = sort_pass(n, FromPairs{o.sorted[to]}, i * digit, bins, o, o.sorted[to ^ 1], 0, s);
    if (e != cudaSuccess) return e;
    return launch_overlapped(&k_embed_places, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, n,
                             (uint32_t)vocab, (const uint2 *)o.sorted[0], o.present, o.start,
                             o.end);
}

}  // namespace

size_t order_hist_bytes(int64_t n) {
    return n <= kRankTokens ? 0 : (size_t)kSortBlocks * kMaxBins * 4;
}

cudaError_t launch_order(int64_t n, int64_t vocab, int id_bytes, const void *ids,
                         const TokenOrder &o, cudaStream_t s) {
    return id_bytes == 4 ? order(n, vocab, static_cast<const int32_t *>(ids), o, s)
                         : order(n, vocab, static_cast<const int64_t *>(ids), o, s);
}

}  // namespace hc
