// hc_embed_bwd.cu -- the gradient of an embedding table:
//   dtable[v, :] (+)= scale * (sum over tokens t with id_t = v, over copies j, of dx[t, j, :]).
//
// Tokens are put in order of their ids, those of one id by position, so that a sum's
// order depends on nothing but the ids.  The ordered tokens are cut into windows of
// C places, and each id's tokens into pieces of C from its first one on; the block
// of a window sums the pieces that start in it.  An id with C tokens or fewer is
// one piece, and its sum is written to the table at once.  Longer ones leave a row of
// partial sums per piece, which k_embed_join adds up in order.  So every gradient
// is read once and a frequent id's sum is spread over the GPU.
//
// An HBM stream: 65,536 tokens of 4 x 5120 into 131,072 fp32 rows (5.37 GB) 826 us, 6.5 TB/s,
// 96% of a copy's rate; 16,384 497 us (6.8 TB/s); added to those rows 570 us (6.1 TB/s).
#include <algorithm>

#include "hc_embed_order.h"
#include "hc_rows.cuh"

namespace hc {
namespace {

constexpr int kMaxPiece = 32;

// Tokens a piece: 32, down to 4 where there are too few of them to fill the GPU (in
// pieces times slices of 1,024 channels): a block's tokens follow one another, but
// ids with more than a piece's tokens pay for a second launch's work.  In us, with
// 4, 8, 16 and 32 a piece: 300 tokens of 1 x 1000 8.6, 10, 13, 17; 1,500 into 1,000
// rows 15.7, 14.6, 13.7, 13.2 (21 with two); 4,096 of 4 x 5120 122, 106, 101 from 8 on.
int piece_tokens(int64_t n, int64_t d) {
    if (n <= 8) return 8;  // one piece holds them all: nothing to join
    const int64_t slices = (d + 1023) / 1024;
    int c = kMaxPiece;
    while (c > 4 && n * slices < (int64_t)c * 256) c /= 2;
    return c;
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

struct Workspace {
    TokenOrder order;
    uint4 *longs;  // ids with more than C tokens: id, first window, pieces
    float *part;   // [windows, 2, d]
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
    w.order.sorted[0] = reinterpret_cast<uint2 *>(take((size_t)n * 8));
    w.order.sorted[1] = reinterpret_cast<uint2 *>(take((size_t)n * 8));
    w.order.hist = reinterpret_cast<uint32_t *>(take(order_hist_bytes(n)));
    w.order.present = reinterpret_cast<uint32_t *>(take((size_t)((vocab + 31) / 32) * 4));
    w.order.start = reinterpret_cast<uint32_t *>(take((size_t)vocab * 4));
    w.order.end = reinterpret_cast<uint32_t *>(take((size_t)vocab * 4));
    w.order.count = reinterpret_cast<uint32_t *>(take(4));
    w.longs = reinterpret_cast<uint4 *>(take((size_t)windows * 16));
    w.part = reinterpret_cast<float *>(take((size_t)windows * 2 * d * 4));
    w.bytes = at;
    return w;
}

// Eight channels of a row of the table's gradient lie in so many 16-byte vectors.
template <int DT>
constexpr int kRow16 = 8 / RowVec<DT>::E;

// scale * a, or that and what was there (`old`), rounded once.
template <int DT, bool ADD>
__device__ __forceinline__ void put(uint4 *table, int64_t at, const float a[8], float scale,
                                    const uint4 old[kRow16<DT>]) {
    constexpr int E = RowVec<DT>::E;
#pragma unroll
    for (int q = 0; q < kRow16<DT>; ++q) {
        float f[E];
        if (ADD) {
            RowVec<DT>::get(old[q], f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = fmaf(scale, a[q * E + e], f[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = scale * a[q * E + e];
        }
        st_stream(table + at * kRow16<DT> + q, RowVec<DT>::set(f));
    }
}

// Zeros to the rows that no token names.  A warp takes a part of 32 rows at a time (a
// word of `present`): 8 KB of them as one run where rows are shorter than 4 KB, else
// 1 KB of each (64 tokens into 32,768 fp32 rows of 5120: 98 us, with 4 KB 108).
inline __host__ __device__ int64_t clear_parts(int64_t row16) {
    return row16 < 256 ? (32 * row16 + 511) / 512 : (row16 + 63) / 64;
}
__device__ void clear_rows(int64_t vocab, int64_t row16, const uint32_t *present, uint4 *table,
                           int64_t warp, int64_t warps) {
    const int lane = threadIdx.x & 31;
    const int64_t parts = clear_parts(row16), units = (vocab + 31) / 32 * parts;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t u = warp; u < units; u += warps) {
        const int64_t word = u / parts;
        const int part = (int)(u - word * parts);
        uint32_t absent = ~__ldg(present + word);
        if (word * 32 + 32 > vocab) absent &= (1u << (vocab - word * 32)) - 1u;
        uint4 *rows = table + word * 32 * row16;
        if (row16 < 256) {
            const uint32_t r16 = (uint32_t)row16, all = 32 * r16;
#pragma unroll 4
            for (int k = 0; k < 16; ++k) {
                const uint32_t i = part * 512 + k * 32 + lane;
                if (i < all && (absent >> (i / r16) & 1u)) st_stream(rows + i, zero);
            }
            continue;
        }
        const int64_t at = (int64_t)part * 64 + lane;
        while (absent != 0) {
            uint4 *row = rows + (__ffs(absent) - 1) * row16 + at;
            absent &= absent - 1;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (at + k * 32 < row16) st_stream(row + k * 32, zero);
        }
    }
}

// Tokens under way in k_embed_sum, 16 to 24 vectors a thread.
template <int HC>
constexpr int kSumStages = HC == 1 ? 16 : HC == 4 ? 5 : 3;

// Sums of the pieces that start in a window of c ordered tokens, for the vectors of
// a slice (blockIdx.y).  The window's tokens follow one another, whatever ids they
// have; each thread copies its vector of the tokens to come to shared memory ahead of
// the sums.  (What the sums are added to is read when they are due: copied ahead as
// well, 65,536 tokens took 614 us in place of 566.)  Blocks behind the windows clear
// the rows that no token names.
template <int DT, int HC, bool ADD>
__global__ void __launch_bounds__(256)
    k_embed_sum(int64_t n, int64_t nv, int64_t windows, int c, int64_t vocab, float scale,
                const uint2 *__restrict__ sorted, uint32_t *__restrict__ longs_count,
                uint4 *__restrict__ longs, const uint32_t *__restrict__ present,
                const uint32_t *__restrict__ start, const uint32_t *__restrict__ end,
                const uint4 *__restrict__ dx, uint4 *table, float4 *__restrict__ part) {
    constexpr int S = kSumStages<HC>, Q = kRow16<DT>;
    enum { kLast = 1, kWhole = 2, kFirst = 4, kRow = kLast | kWhole };
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
    auto slot = [&](int stage, int j) {
        return ring + (stage * HC + j) * blockDim.x + threadIdx.x;
    };
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
        uint4 old[Q];
        if (ADD && (f & kRow) == kRow)
#pragma unroll
            for (int q = 0; q < Q; ++q) old[q] = table[row * Q + q];
        copies_wait<S - 2>();
#pragma unroll
        for (int j = 0; j < HC; ++j) {
            float x[8];
            unpack8(*slot(at, j), x);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] += x[e];
        }
        const int next = at == 0 ? S - 1 : at - 1;
        if (ADD) copy(i + S - 1, next);  // `old` is on its way; else the row goes out first
        if (f & kLast) {
            if (f & kWhole) {
                put<DT, ADD>(table, row, a, scale, old);
            } else {
                float4 *p = part + ((w * 2 + (f & kFirst ? 1 : 0)) * nv + v) * 2;
                p[0] = make_float4(a[0], a[1], a[2], a[3]);
                p[1] = make_float4(a[4], a[5], a[6], a[7]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = 0.0f;
        }
        if (!ADD) copy(i + S - 1, next);
        at = at + 1 == S ? 0 : at + 1;
    }
}

// The partial sums of an id with more than C tokens, in order: 8 warps take every
// eighth of them for 32 vectors, and their sums meet in shared memory.
template <int DT, bool ADD>
__global__ void __launch_bounds__(256)
    k_embed_join(int64_t nv, float scale, const uint32_t *__restrict__ longs_count,
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
            uint4 old[kRow16<DT>];
            if (ADD && warp == 0 && v < nv)
#pragma unroll
                for (int q = 0; q < kRow16<DT>; ++q) old[q] = table[(id * nv + v) * kRow16<DT> + q];
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
                put<DT, ADD>(table, id * nv + v, a, scale, old);
            }
            __syncthreads();
        }
    }
}

template <int DT, int HC, bool ADD>
cudaError_t launch(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    static SmemState smem;
    const Workspace w = layout(p.ws, p.n, p.d, p.vocab);
    const int c = piece_tokens(p.n, p.d);
    const int64_t nv = p.d / 8, windows = (p.n + c - 1) / c;
    const TokenOrder &o = w.order;
    cudaError_t e = launch_order(p.n, p.vocab, p.id_bytes, p.ids, o, s);
    if (e != cudaSuccess) return e;
    // slices of at most 256 vectors, as even as whole warps make them
    const int64_t slices = (nv + 255) / 256;
    const int threads = (int)(((nv + slices - 1) / slices + 31) & ~(int64_t)31);
    constexpr int per_thread = kSumStages<HC> * HC * 16;
    auto *kernel = &k_embed_sum<DT, HC, ADD>;
    e = allow_smem(smem, reinterpret_cast<const void *>(kernel), per_thread * 256, di);
    if (e != cudaSuccess) return e;
    uint4 *table = static_cast<uint4 *>(p.dtable);
    const uint2 *sorted = o.sorted[0];
    // to clear rows: a warp for each part of them, up to 64 blocks an SM and slice (16,384 x 4 x
    // 5120 into 131,072 fp32 rows: 498 us, with 16 blocks 502, with 4 about 520)
    const int64_t warps = slices * (threads / 32),
                  units = (p.vocab + 31) / 32 * clear_parts(p.d * row_type_bytes(p.dtype) / 16);
    const int64_t clear = ADD ? 0 : std::min((units + warps - 1) / warps, (int64_t)di.sms * 64);
    e = launch_overlapped(kernel, dim3((unsigned)(windows + clear), (unsigned)slices),
                          dim3(threads), (size_t)per_thread * threads, s, p.n, nv, windows, c,
                          p.vocab, p.scale, sorted, o.count, w.longs, (const uint32_t *)o.present,
                          (const uint32_t *)o.start, (const uint32_t *)o.end,
                          reinterpret_cast<const uint4 *>(p.dx), table,
                          reinterpret_cast<float4 *>(w.part));
    if (e != cudaSuccess || p.n <= c) return e;  // no id has more tokens than a piece
    // ids with more than c tokens: no more than windows, and few of them as a rule
    const int64_t parts = std::min<int64_t>((nv + 31) / 32, 1024);
    const int64_t joins = std::min(windows, std::max<int64_t>(2432 / parts, 16));
    return launch_overlapped(&k_embed_join<DT, ADD>, dim3((unsigned)joins, (unsigned)parts),
                             dim3(256), 0, s, nv, p.scale, (const uint32_t *)o.count,
                             (const uint4 *)w.longs, (const float4 *)w.part, table);
}

template <int DT, bool ADD>
cudaError_t launch(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.hc == 1   ? launch<DT, 1, ADD>(p, di, s)
           : p.hc == 4 ? launch<DT, 4, ADD>(p, di, s)
                       : launch<DT, 8, ADD>(p, di, s);
}

template <int DT>
cudaError_t launch(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    return p.accumulate ? launch<DT, true>(p, di, s) : launch<DT, false>(p, di, s);
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
