// hc_embed_bwd.cu -- the gradient of an embedding table:
//   dtable[v, :] (+)= scale * sum over the tokens t with id_t = v, over the copies j, of dx[t, j, :].
//
// Tokens are put in order of their ids, those of one id by position, so that a sum's
// order depends on nothing but the ids.  The ordered tokens are cut into windows of
// C places, and each id's tokens into pieces of C from its first one on; the block
// of a window sums the pieces that start in it.  An id with C tokens or fewer is
// one piece, and its sum is written to the table at once.  Longer ones leave a row of
// partial sums per piece, which k_embed_join adds up in order.  So every gradient
// is read once and a frequent id's sum is spread over the GPU.
#include <algorithm>

#include "hc_rows.cuh"

namespace hc {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kTile = 2048;  // tokens a block of the radix sort has at a time
constexpr int kItems = kTile / kSortThreads;
constexpr int kSortBlocks = 304;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;  // as many as threads
constexpr int kMaxPiece = 32;
constexpr int kRankTokens = 4096;  // up to which tokens are ranked by comparing them all
constexpr int kRankRows = 8192;    // table rows whose presence a block of k_rank notes
constexpr int kRankThreads = 1024;
constexpr int kRankWarps = kRankThreads / 32;

int bits_of(int64_t v) {  // of the numbers 0 .. v
    int b = 1;
    while ((v >> b) != 0) ++b;
    return b;
}

// Tokens a piece: 32, fewer where there are too few of them to fill the GPU (in
// pieces times slices of 1,024 channels).  4,096 tokens of 4 x 5120 into 32,768 rows:
// 101 us with 32 a piece, 106 with 16, 122 with 8 (the pieces' sums are written, read
// and joined); 1,537 of 8 x 1032 into 50,001: 47, 48 and 55.
int piece_tokens(int64_t n, int64_t d) {
    const int64_t slices = (d + 1023) / 1024;
    int c = kMaxPiece;
    while (c > 1 && n * slices < (int64_t)c * 608) c /= 2;
    return c;
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

struct Workspace {
    uint2 *sorted[2];   // (id, token): the last pass leaves them in [0]
    uint32_t *hist;     // [blocks, bins]
    uint32_t *count;    // of `longs`
    uint4 *longs;       // ids with more than C tokens: id, first window, pieces
    uint32_t *present;  // a bit for each row of the table: some token names it
    uint32_t *start;    // [vocab], first place of an id that is present
    uint32_t *end;      // [vocab], the place behind its last
    float *part;        // [windows, 2, d]
    size_t bytes;
};

// The parts of a workspace at `base`, and its size.
Workspace layout(uint8_t *base, int64_t n, int64_t d, int64_t vocab) {
    const int64_t c = piece_tokens(n, d), windows = (n + c - 1) / c;
    size_t at = 0;
    auto take = [&](size_t b) {
        const size_t here = at;
        at += align256(b);
        return base == nullptr ? nullptr : base + here;
    };
    Workspace w;
    w.sorted[0] = reinterpret_cast<uint2 *>(take((size_t)n * 8));
    w.sorted[1] = reinterpret_cast<uint2 *>(take((size_t)n * 8));
    w.hist = reinterpret_cast<uint32_t *>(take((size_t)kSortBlocks * kMaxBins * 4));
    w.count = reinterpret_cast<uint32_t *>(take(4));
    w.longs = reinterpret_cast<uint4 *>(take((size_t)windows * 16));
    w.present = reinterpret_cast<uint32_t *>(take((size_t)((vocab + 31) / 32) * 4));
    w.start = reinterpret_cast<uint32_t *>(take((size_t)vocab * 4));
    w.end = reinterpret_cast<uint32_t *>(take((size_t)vocab * 4));
    w.part = reinterpret_cast<float *>(take((size_t)windows * 2 * d * 4));
    w.bytes = at;
    return w;
}

// An id as it is ordered: those outside the table come behind it, as `vocab`.
template <typename ID>
__device__ __forceinline__ uint32_t row_of(const ID *ids, int64_t i, int64_t vocab) {
    const int64_t id = (int64_t)__ldg(ids + i);
    return (uint32_t)(id >= 0 && id < vocab ? id : vocab);
}

// Few tokens: a token's place is the number of tokens with a smaller id, and of those
// before it with its own.  A block has 32 of them, one a lane, and all ids in shared
// memory; its warps share the comparisons.  n^2 of them take 1.4 us at 4,096 tokens,
// where the passes of the sort below take 20.  A block also notes which of
// kRankRows rows of the table are present.
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
// k_embed_places adds to.
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
        for (int k = 0; k < kItems; ++k) {
            const bool in = first + k * 32 < i1;
            const uint32_t digit = (e[k].x >> shift) & (bins - 1);
            // lanes past the end have a group of their own
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, in ? digit : 0xFFFFFFFFu);
            const uint32_t below = same & ((1u << lane) - 1u);
            const uint32_t had = in ? cnt[warp][digit] : 0;
            __syncwarp();
            if (in && below == 0) cnt[warp][digit] = had + __popc(same);
            __syncwarp();
            rank[k] = had + __popc(below);
        }
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

// Eight channels of a row of the table's gradient: scale * a, written or added to
// what was there.
template <int DT>
struct Out {
    static constexpr int E = RowVec<DT>::E, Q = 8 / E;
    uint4 old[Q];
    __device__ __forceinline__ void load(const uint4 *table, int64_t at) {
#pragma unroll
        for (int q = 0; q < Q; ++q) old[q] = table[at * Q + q];
    }
    __device__ __forceinline__ void put(uint4 *table, int64_t at, const float a[8], float scale,
                                        bool accumulate) const {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            float f[E];
            if (accumulate) {
                RowVec<DT>::get(old[q], f);
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = fmaf(scale, a[q * E + e], f[e]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) f[e] = scale * a[q * E + e];
            }
            st_stream(table + at * Q + q, RowVec<DT>::set(f));
        }
    }
};

// Zeros to the rows that no token names.  A warp takes 32 rows (a word of `present`)
// and 4 KB of each of them at a time.
__device__ void clear_rows(int64_t vocab, int64_t row16, const uint32_t *present, uint4 *table,
                           int64_t warp, int64_t warps) {
    const int lane = threadIdx.x & 31;
    const int64_t parts = (row16 + 255) / 256, units = ((vocab + 31) / 32) * parts;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t u = warp; u < units; u += warps) {
        const int64_t word = u / parts, at = (u - word * parts) * 256 + lane;
        uint32_t absent = ~__ldg(present + word);
        if (word * 32 + 32 > vocab) absent &= (1u << (vocab - word * 32)) - 1u;
        while (absent != 0) {
            const int64_t row = word * 32 + __ffs(absent) - 1;
            absent &= absent - 1;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (at + k * 32 < row16) st_stream(table + row * row16 + at + k * 32, zero);
        }
    }
}

template <int HC>
constexpr int sum_stages() {
    return HC == 1 ? 16 : HC == 4 ? 5 : 3;  // tokens under way: 16 to 24 vectors a thread
}

// Sums of the pieces that start in a window of c ordered tokens, for the vectors of
// a slice (blockIdx.y).  The window's tokens follow one another, whatever ids they
// have; each thread copies its vector of the tokens to come to shared memory ahead of
// the sums.  Blocks behind the windows clear the rows that no token names.
template <int DT, int HC>
__global__ void __launch_bounds__(256)
    k_embed_sum(int64_t n, int64_t nv, int64_t windows, int c, int64_t vocab, float scale,
                bool accumulate, const uint2 *__restrict__ sorted,
                uint32_t *__restrict__ longs_count, uint4 *__restrict__ longs,
                const uint32_t *__restrict__ present, const uint32_t *__restrict__ start,
                const uint32_t *__restrict__ end, const uint4 *__restrict__ dx,
                uint4 *__restrict__ table, float4 *__restrict__ part) {
    constexpr int S = sum_stages<HC>();
    enum { kLast = 1, kWhole = 2, kFirst = 4 };
    extern __shared__ uint4 ring[];
    __shared__ uint32_t token[2 * kMaxPiece], ids[2 * kMaxPiece], flags[2 * kMaxPiece], from, count;
    griddep_wait_then_release();
    const int64_t w = blockIdx.x;
    if (w >= windows) {
        const int64_t wpb = blockDim.x >> 5;
        clear_rows(vocab, nv * 8 / RowVec<DT>::E, present, table,
                   ((w - windows) * gridDim.y + blockIdx.y) * wpb + (threadIdx.x >> 5),
                   (gridDim.x - windows) * gridDim.y * wpb);
        return;
    }
    if (threadIdx.x == 0) from = 2 * kMaxPiece, count = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * c; i += blockDim.x) {
        const int64_t p = w * c + i;
        if (p >= n) break;
        const uint2 e = sorted[p];
        if (e.x == (uint32_t)vocab) break;
        const uint32_t s = start[e.x], t = end[e.x];
        const int in_piece = (int)(((uint32_t)p - s) & (uint32_t)(c - 1));
        // pieces that start in this window, up to their ends in the next
        if (in_piece > i || i - in_piece >= c) continue;
        const bool whole = t - s <= (uint32_t)c, first = (uint32_t)p - s < (uint32_t)c;
        token[i] = e.y;
        ids[i] = e.x;
        flags[i] = (in_piece == c - 1 || p + 1 == t ? kLast : 0) | (whole ? kWhole : 0) |
                   (first ? kFirst : 0);
        atomicMin(&from, (uint32_t)i);
        atomicAdd(&count, 1u);
        if (p == s && !whole && blockIdx.y == 0)
            longs[atomicAdd(longs_count, 1u)] =
                make_uint4(e.x, (uint32_t)w, (t - s + (uint32_t)c - 1) / (uint32_t)c, 0);
    }
    __syncthreads();
    const int64_t v = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
    const int i0 = (int)from, i1 = i0 + (int)count;
    if (v >= nv || count == 0) return;
    auto slot = [&](int stage, int j) { return ring + (stage * HC + j) * blockDim.x + threadIdx.x; };
    auto copy = [&](int i, int stage) {
        if (i < i1) {
            const uint4 *g = dx + (int64_t)token[i] * HC * nv + v;
#pragma unroll
            for (int j = 0; j < HC; ++j) copy16_async(slot(stage, j), g + j * nv);
        }
        copies_commit();
    };
#pragma unroll
    for (int k = 0; k < S - 1; ++k) copy(i0 + k, k);
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = 0.0f;
    int at = 0;
    for (int i = i0; i < i1; ++i) {
        const uint32_t f = flags[i];
        const int64_t row = (int64_t)ids[i] * nv + v;
        Out<DT> out;
        if (accumulate && (f & (kLast | kWhole)) == (kLast | kWhole)) out.load(table, row);
        copies_wait<S - 2>();
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            float x[8];
            unpack8(*slot(at, j), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] += x[e];
        }
        copy(i + S - 1, at == 0 ? S - 1 : at - 1);
        at = at + 1 == S ? 0 : at + 1;
        if (f & kLast) {
            if (f & kWhole) {
                out.put(table, row, a, scale, accumulate);
            } else {
                float4 *p = part + ((w * 2 + (f & kFirst ? 1 : 0)) * nv + v) * 2;
                p[0] = make_float4(a[0], a[1], a[2], a[3]);
                p[1] = make_float4(a[4], a[5], a[6], a[7]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = 0.0f;
        }
    }
}

// The partial sums of an id with more than C tokens, in order: 8 warps take every
// eighth of them for 32 vectors, and their sums meet in shared memory.
template <int DT>
__global__ void __launch_bounds__(256)
    k_embed_join(int64_t nv, float scale, bool accumulate, const uint32_t *__restrict__ longs_count,
                 const uint4 *__restrict__ longs, const float4 *__restrict__ part,
                 uint4 *__restrict__ table) {
    __shared__ float red[8][32][9];
    griddep_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t count = *longs_count;
    for (uint32_t i = blockIdx.x; i < count; i += gridDim.x) {
        const uint4 entry = longs[i];
        const int64_t id = entry.x, w = entry.y, pieces = entry.z;
        for (int64_t v0 = (int64_t)blockIdx.y * 32; v0 < nv; v0 += (int64_t)gridDim.y * 32) {
            const int64_t v = v0 + lane;
            Out<DT> out;
            if (accumulate && warp == 0 && v < nv) out.load(table, id * nv + v);
            float a[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = 0.0f;
            if (v < nv) {
#pragma unroll 4
                for (int64_t k = warp; k < pieces; k += 8) {
                    const float4 *p = part + (((w + k) * 2 + (k == 0 ? 1 : 0)) * nv + v) * 2;
                    const float4 lo = p[0], hi = p[1];
                    a[0] += lo.x, a[1] += lo.y, a[2] += lo.z, a[3] += lo.w;
                    a[4] += hi.x, a[5] += hi.y, a[6] += hi.z, a[7] += hi.w;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) red[warp][lane][e] = a[e];
            __syncthreads();
            if (warp == 0 && v < nv) {
#pragma unroll
                for (int q = 1; q < 8; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) a[e] += red[q][lane][e];
                out.put(table, id * nv + v, a, scale, accumulate);
            }
            __syncthreads();
        }
    }
}

template <typename SRC>
cudaError_t sort_pass(int64_t n, SRC src, int shift, int bins, const Workspace &w, uint2 *out,
                      int64_t clear_words, cudaStream_t s) {
    const int64_t tiles = (n + kTile - 1) / kTile;
    const dim3 grid((unsigned)(tiles < kSortBlocks ? tiles : kSortBlocks));
    cudaError_t e = launch_overlapped(&k_sort_count<SRC>, grid, dim3(kSortThreads), 0, s, n, src,
                                      shift, bins, w.hist, w.count, w.present, clear_words);
    if (e != cudaSuccess) return e;
    return launch_overlapped(&k_sort_move<SRC>, grid, dim3(kSortThreads), 0, s, n, src, shift, bins,
                             (const uint32_t *)w.hist, out);
}

// Tokens in order of their ids, and each id's places.
template <typename ID>
cudaError_t order_tokens(const EmbedBackward &p, const Workspace &w, cudaStream_t s) {
    const ID *ids = static_cast<const ID *>(p.ids);
    if (p.n <= kRankTokens) {
        const int64_t by_tokens = (p.n + 31) / 32, by_rows = (p.vocab + kRankRows - 1) / kRankRows;
        return launch_overlapped(&k_rank<ID>,
                                 dim3((unsigned)(by_tokens > by_rows ? by_tokens : by_rows)),
                                 dim3(kRankThreads), 0, s, (int)p.n, p.vocab, ids, w.sorted[0], w.count,
                                 w.present, w.start, w.end);
    }
    const int bits = bits_of(p.vocab), passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    const int digit = (bits + passes - 1) / passes, bins = 1 << digit;
    int to = (passes - 1) & 1;
    cudaError_t e = sort_pass(p.n, FromIds<ID>{ids, p.vocab}, 0, bins, w, w.sorted[to],
                              (p.vocab + 31) / 32, s);
    for (int i = 1; i < passes && e == cudaSuccess; ++i, to ^= 1)
        e = sort_pass(p.n, FromPairs{w.sorted[to]}, i * digit, bins, w, w.sorted[to ^ 1], 0, s);
    if (e != cudaSuccess) return e;
    return launch_overlapped(&k_embed_places, dim3((unsigned)((p.n + 255) / 256)), dim3(256), 0, s,
                             p.n, (uint32_t)p.vocab, (const uint2 *)w.sorted[0], w.present, w.start,
                             w.end);
}

template <int DT, int HC>
cudaError_t launch(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    static SmemState smem;
    const Workspace w = layout(p.ws, p.n, p.d, p.vocab);
    const int c = piece_tokens(p.n, p.d);
    const int64_t nv = p.d / 8, windows = (p.n + c - 1) / c;
    cudaError_t e = p.id_bytes == 4 ? order_tokens<int32_t>(p, w, s) : order_tokens<int64_t>(p, w, s);
    if (e != cudaSuccess) return e;
    // slices of at most 256 vectors, as even as whole warps make them
    const int64_t slices = (nv + 255) / 256;
    const int threads = (int)(((nv + slices - 1) / slices + 31) & ~(int64_t)31);
    constexpr int per_thread = sum_stages<HC>() * HC * 16;
    auto *kernel = &k_embed_sum<DT, HC>;
    e = allow_smem(smem, reinterpret_cast<const void *>(kernel), per_thread * 256, di);
    if (e != cudaSuccess) return e;
    uint4 *table = static_cast<uint4 *>(p.dtable);
    const uint2 *sorted = w.sorted[0];
    // to clear rows: a few blocks an SM, no more than there is work for
    const int64_t work = (p.vocab * p.d + (1 << 16) - 1) >> 16;
    const int64_t clear = p.accumulate ? 0 : std::min(work, (int64_t)di.sms * 4);
    e = launch_overlapped(kernel, dim3((unsigned)(windows + clear), (unsigned)slices), dim3(threads),
                          (size_t)per_thread * threads, s, p.n, nv, windows, c, p.vocab, p.scale,
                          p.accumulate, sorted, w.count, w.longs, (const uint32_t *)w.present,
                          (const uint32_t *)w.start, (const uint32_t *)w.end,
                          reinterpret_cast<const uint4 *>(p.dx), table,
                          reinterpret_cast<float4 *>(w.part));
    if (e != cudaSuccess) return e;
    // ids with more than c tokens: no more than windows, and few of them as a rule
    const int64_t parts = std::min<int64_t>((nv + 31) / 32, 1024);
    const int64_t joins = std::min(windows, std::max<int64_t>(2432 / parts, 16));
    return launch_overlapped(&k_embed_join<DT>, dim3((unsigned)joins, (unsigned)parts), dim3(256), 0,
                             s, nv, p.scale, p.accumulate, (const uint32_t *)w.count,
                             (const uint4 *)w.longs, (const float4 *)w.part, table);
}

template <int DT>
cudaError_t launch(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.hc == 1   ? launch<DT, 1>(p, di, s)
           : p.hc == 4 ? launch<DT, 4>(p, di, s)
                       : launch<DT, 8>(p, di, s);
}

}  // namespace

size_t embed_backward_bytes(int64_t n, int64_t d, int64_t vocab) {
    return layout(nullptr, n, d, vocab).bytes;
}

cudaError_t launch_embed_backward(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    if (p.n == 0) {
        if (p.accumulate) return cudaSuccess;
        return cudaMemsetAsync(p.dtable, 0, (size_t)p.vocab * p.d * row_type_bytes(p.dtype), s);
    }
    return p.dtype == HC_BF16  ? launch<HC_BF16>(p, di, s)
           : p.dtype == HC_F16 ? launch<HC_F16>(p, di, s)
                               : launch<HC_F32>(p, di, s);
}

}  // namespace hc
