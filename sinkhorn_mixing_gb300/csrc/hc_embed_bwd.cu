// hc_embed_bwd.cu -- the gradient of an embedding table:
//   dtable[v, :] (+)= scale * sum over the tokens t with id_t = v, over the copies j, of dx[t, j, :].
//
// Tokens are sorted by id, those of one id by position (a radix sort, stable in
// each pass), so that a sum's order depends on nothing but the ids.  The sorted
// tokens are cut into windows of C places, and each id's tokens into pieces of C from
// its first one on; the block of a window sums the pieces that start in it.  An id
// with C tokens or fewer is one piece, and its sum is written to the table at once.
// Longer ones leave a row of partial sums per piece, which k_embed_join adds up in
// order.  So every gradient is read once and a frequent id's sum is spread over the
// GPU.
#include "hc_rows.cuh"

namespace hc {
namespace {

constexpr int kTile = 2048;      // tokens a block sorts at a time: 256 threads, 8 each
constexpr int kSortBlocks = 304;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
constexpr int kMaxPiece = 32;

int bits_of(int64_t v) {  // of the numbers 0 .. v
    int b = 1;
    while ((v >> b) != 0) ++b;
    return b;
}

// Tokens a piece: 32, fewer where there are too few of them to fill the GPU (in
// pieces times slices of 1,024 channels).
int piece_tokens(int64_t n, int64_t d) {
    const int64_t slices = (d + 1023) / 1024;
    int c = kMaxPiece;
    while (c > 1 && n * slices < (int64_t)c * 1216) c /= 2;
    return c;
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

struct Workspace {
    uint2 *sorted[2];  // (id, token): the last pass leaves them in [0]
    uint32_t *hist;    // [blocks, bins]
    uint32_t *longs;   // count, then first places of the ids with more than C tokens
    uint32_t *start;   // [vocab + 1], place + 1 of an id's first token, 0 where there is none
    uint32_t *end;     // [vocab + 1]
    float *part;       // [windows, 2, d]
    size_t bytes;
};

Workspace layout(uint8_t *base, int64_t n, int64_t d, int64_t vocab) {
    const int64_t c = piece_tokens(n, d), windows = (n + c - 1) / c;
    Workspace w;
    size_t at = 0;
    auto take = [&](size_t b) {
        uint8_t *p = base + at;
        at += align256(b);
        return p;
    };
    w.sorted[0] = reinterpret_cast<uint2 *>(take((size_t)n * 8));
    w.sorted[1] = reinterpret_cast<uint2 *>(take((size_t)n * 8));
    w.hist = reinterpret_cast<uint32_t *>(take((size_t)kSortBlocks * kMaxBins * 4));
    w.longs = reinterpret_cast<uint32_t *>(take((size_t)(windows + 1) * 4));
    w.start = reinterpret_cast<uint32_t *>(take((size_t)(vocab + 1) * 4));
    w.end = reinterpret_cast<uint32_t *>(take((size_t)(vocab + 1) * 4));
    w.part = reinterpret_cast<float *>(take((size_t)windows * 2 * d * 4));
    w.bytes = at;
    return w;
}

// Where the sort's first pass reads: the ids themselves; ids outside the table sort
// behind it, as `vocab`.
template <typename ID>
struct FromIds {
    const ID *ids;
    int64_t vocab;
    __device__ __forceinline__ uint2 get(int64_t i) const {
        const int64_t id = (int64_t)__ldg(ids + i);
        return make_uint2((uint32_t)(id >= 0 && id < vocab ? id : vocab), (uint32_t)i);
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

// How many of a block's tokens have each digit.  The first pass also clears the
// words that the kernels behind the sort fill.
template <typename SRC>
__global__ void __launch_bounds__(256)
    k_sort_count(int64_t n, SRC src, int shift, int bins, uint32_t *__restrict__ hist,
                 uint32_t *__restrict__ longs, uint32_t *__restrict__ start, int64_t ids) {
    __shared__ uint32_t cnt[kMaxBins];
    griddep_wait_then_release();
    for (int i = threadIdx.x; i < bins; i += 256) cnt[i] = 0;
    if (start != nullptr) {
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < ids;
             i += (int64_t)gridDim.x * 256)
            start[i] = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) longs[0] = 0;
    }
    __syncthreads();
    const int64_t i1 = first_token(n, gridDim.x, blockIdx.x + 1);
    for (int64_t i = first_token(n, gridDim.x, blockIdx.x) + threadIdx.x; i < i1; i += 256)
        atomicAdd(&cnt[(src.get(i).x >> shift) & (bins - 1)], 1u);
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += 256) hist[(int64_t)blockIdx.x * bins + i] = cnt[i];
}

// Exclusive sums of v over the 256 threads.
__device__ __forceinline__ uint32_t exclusive_256(uint32_t v, uint32_t *red) {
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
    for (int w = 0; w < 8; ++w) before += w < warp ? red[w] : 0;
    return before + s - v;
}

// A block's tokens to their places in the digit's order.  A place: tokens with a
// smaller digit, then those of blocks, tiles, warps and lanes before this one.
template <typename SRC>
__global__ void __launch_bounds__(256)
    k_sort_move(int64_t n, SRC src, int shift, int bins, const uint32_t *__restrict__ hist,
                uint2 *__restrict__ out) {
    __shared__ uint32_t base[kMaxBins], cnt[8][kMaxBins], red[8];
    griddep_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = gridDim.x;
    // two neighbouring digits a thread
    uint32_t total[2] = {0, 0}, before[2] = {0, 0};
    const int d0 = 2 * threadIdx.x;
    for (int b = 0; b < blocks; ++b) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t c = d0 + k < bins ? hist[(int64_t)b * bins + d0 + k] : 0;
            total[k] += c;
            before[k] += b < (int)blockIdx.x ? c : 0;
        }
    }
    const uint32_t lower = exclusive_256(total[0] + total[1], red);
    base[d0] = lower + before[0];
    base[d0 + 1] = lower + total[0] + before[1];
    const int64_t i1 = first_token(n, blocks, blockIdx.x + 1);
    for (int64_t i0 = first_token(n, blocks, blockIdx.x); i0 < i1; i0 += kTile) {
        for (int i = threadIdx.x; i < 8 * kMaxBins; i += 256) (&cnt[0][0])[i] = 0;
        __syncthreads();
        uint2 e[8];
        uint32_t rank[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = i0 + warp * 256 + k * 32 + lane;
            const bool in = i < i1;
            e[k] = in ? src.get(i) : make_uint2(0, 0);
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
        for (int g = threadIdx.x; g < bins; g += 256) {
            uint32_t at = base[g];
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                const uint32_t c = cnt[w][g];
                cnt[w][g] = at;
                at += c;
            }
            base[g] = at;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + warp * 256 + k * 32 + lane < i1)
                out[cnt[warp][(e[k].x >> shift) & (bins - 1)] + rank[k]] = e[k];
        }
        __syncthreads();
    }
}

// First and last places of every id, and the ids with more than c tokens (in any
// order: each is summed by itself).
__global__ void __launch_bounds__(256)
    k_embed_places(int64_t n, int c, uint32_t vocab, const uint2 *__restrict__ sorted,
                   uint32_t *__restrict__ longs, uint32_t *__restrict__ start,
                   uint32_t *__restrict__ end) {
    griddep_wait_then_release();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const uint32_t id = sorted[i].x;
    if (id == vocab) return;
    if (i == 0 || sorted[i - 1].x != id) {
        start[id] = (uint32_t)i + 1;
        if (i + c < n && sorted[i + c].x == id) longs[1 + atomicAdd(longs, 1u)] = (uint32_t)i;
    }
    if (i + 1 == n || sorted[i + 1].x != id) end[id] = (uint32_t)i + 1;
}

// Eight channels of a row of the table's gradient: scale * a, written or added.
template <int DT>
__device__ __forceinline__ void put(uint4 *table, int64_t at, const float a[8], float scale,
                                    bool accumulate) {
    constexpr int E = RowVec<DT>::E;
#pragma unroll
    for (int q = 0; q < 8 / E; ++q) {
        uint4 *p = table + at * (8 / E) + q;
        float f[E];
        if (accumulate) {
            RowVec<DT>::get(*p, f);
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = fmaf(scale, a[q * E + e], f[e]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = scale * a[q * E + e];
        }
        st_stream(p, RowVec<DT>::set(f));
    }
}

// Sums of the pieces that start in a window of c sorted tokens, for the vectors of
// a slice (blockIdx.y).  Blocks behind the windows clear rows that no token names.
template <int DT, int HC>
__global__ void __launch_bounds__(256)
    k_embed_sum(int64_t n, int64_t nv, int64_t windows, int c, uint32_t vocab, float scale,
                bool accumulate, const uint2 *__restrict__ sorted,
                const uint32_t *__restrict__ start, const uint32_t *__restrict__ end,
                const uint4 *__restrict__ dx, uint4 *__restrict__ table, float4 *__restrict__ part) {
    __shared__ uint32_t token[2 * kMaxPiece], ids[kMaxPiece], len[kMaxPiece], kind[kMaxPiece];
    griddep_wait_then_release();
    const int64_t v = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
    const int64_t w = blockIdx.x;
    if (w >= windows) {
        if (v >= nv) return;
        const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int64_t r = w - windows; r < vocab; r += gridDim.x - windows)
            if (start[r] == 0) put<DT>(table, r * nv + v, zero, 1.0f, false);
        return;
    }
    const int64_t p0 = w * c;
    for (int i = threadIdx.x; i < 2 * c; i += blockDim.x) {
        const bool in = p0 + i < n;
        const uint2 e = in ? sorted[p0 + i] : make_uint2(vocab, 0);
        token[i] = e.y;
        if (i < c) {
            ids[i] = e.x;
            len[i] = 0;
            if (e.x != vocab) {
                const uint32_t p = (uint32_t)(p0 + i), s = start[e.x] - 1, t = end[e.x];
                if ((p - s) % c == 0) {
                    len[i] = min((uint32_t)c, t - p);
                    // 0: all of an id; 1 and 2: a later and the first piece of a long one
                    kind[i] = t - s <= (uint32_t)c ? 0 : p != s ? 1 : 2;
                }
            }
        }
    }
    __syncthreads();
    if (v >= nv) return;
    for (int i = 0; i < c; ++i) {
        const int m = len[i];
        if (m == 0) continue;
        float a[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = 0.0f;
        constexpr int T = 8 / HC;  // tokens whose vectors are in flight together
        for (int k = 0; k < m; k += T) {
            uint4 g[T * HC];
#pragma unroll
            for (int q = 0; q < T; ++q) {
                const int64_t t = token[i + min(k + q, m - 1)];
#pragma unroll
                for (int j = 0; j < HC; ++j) g[q * HC + j] = ld_stream(dx + (t * HC + j) * nv + v);
            }
#pragma unroll
            for (int q = 0; q < T; ++q) {
                if (k + q < m) {
#pragma unroll
                    for (int j = 0; j < HC; ++j) {
                        float f[8];
                        unpack8(g[q * HC + j], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) a[e] += f[e];
                    }
                }
            }
        }
        if (kind[i] == 0) {
            put<DT>(table, (int64_t)ids[i] * nv + v, a, scale, accumulate);
        } else {
            float4 *p = part + ((w * 2 + (kind[i] - 1)) * nv + v) * 2;
            p[0] = make_float4(a[0], a[1], a[2], a[3]);
            p[1] = make_float4(a[4], a[5], a[6], a[7]);
        }
    }
}

// The partial sums of an id with more than c tokens, in order: 8 warps take every
// eighth of them for 32 vectors (blockIdx.y), and their sums meet in shared memory.
template <int DT>
__global__ void __launch_bounds__(256)
    k_embed_join(int64_t nv, int c, float scale, bool accumulate, const uint2 *__restrict__ sorted,
                 const uint32_t *__restrict__ longs, const uint32_t *__restrict__ end,
                 const float4 *__restrict__ part, uint4 *__restrict__ table) {
    __shared__ float red[8][32][9];
    griddep_wait_then_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t v = (int64_t)blockIdx.y * 32 + lane;
    const uint32_t count = longs[0];
    for (uint32_t i = blockIdx.x; i < count; i += gridDim.x) {
        const uint32_t s = longs[1 + i], id = sorted[s].x;
        const int64_t w = s / c, pieces = (end[id] - s + c - 1) / c;
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
            put<DT>(table, (int64_t)id * nv + v, a, scale, accumulate);
        }
        __syncthreads();
    }
}

// Places a pass of the sort: ids (or the pairs of the pass before) to `out`.
template <typename SRC>
cudaError_t sort_pass(int64_t n, SRC src, int shift, int bins, const Workspace &w, uint2 *out,
                      int64_t clear, cudaStream_t s) {
    const int64_t tiles = (n + kTile - 1) / kTile;
    const dim3 grid((unsigned)(tiles < kSortBlocks ? tiles : kSortBlocks));
    cudaError_t e = launch_overlapped(&k_sort_count<SRC>, grid, dim3(256), 0, s, n, src, shift,
                                      bins, w.hist, w.longs, clear ? w.start : nullptr, clear);
    if (e != cudaSuccess) return e;
    return launch_overlapped(&k_sort_move<SRC>, grid, dim3(256), 0, s, n, src, shift, bins,
                             (const uint32_t *)w.hist, out);
}

template <typename ID>
cudaError_t sort_ids(const EmbedBackward &p, const Workspace &w, cudaStream_t s) {
    const int bits = bits_of(p.vocab), passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    const int digit = (bits + passes - 1) / passes, bins = 1 << digit;
    int to = (passes - 1) & 1;
    cudaError_t e = sort_pass(p.n, FromIds<ID>{static_cast<const ID *>(p.ids), p.vocab}, 0, bins, w,
                              w.sorted[to], p.vocab + 1, s);
    for (int i = 1; i < passes && e == cudaSuccess; ++i, to ^= 1)
        e = sort_pass(p.n, FromPairs{w.sorted[to]}, i * digit, bins, w, w.sorted[to ^ 1], 0, s);
    return e;
}

template <int DT, int HC>
cudaError_t launch(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s) {
    const Workspace w = layout(p.ws, p.n, p.d, p.vocab);
    const int c = piece_tokens(p.n, p.d);
    const int64_t nv = p.d / 8, windows = (p.n + c - 1) / c;
    cudaError_t e = p.id_bytes == 4 ? sort_ids<int32_t>(p, w, s) : sort_ids<int64_t>(p, w, s);
    if (e != cudaSuccess) return e;
    const uint2 *sorted = w.sorted[0];
    e = launch_overlapped(&k_embed_places, dim3((unsigned)((p.n + 255) / 256)), dim3(256), 0, s,
                          p.n, c, (uint32_t)p.vocab, sorted, w.longs, w.start, w.end);
    if (e != cudaSuccess) return e;
    // slices of at most 256 vectors, as even as whole warps make them
    const int64_t slices = (nv + 255) / 256;
    const int threads = (int)(((nv + slices - 1) / slices + 31) & ~(int64_t)31);
    uint4 *table = static_cast<uint4 *>(p.dtable);
    const int64_t cap = (int64_t)di.sms * 16;
    const int64_t clear = p.accumulate ? 0 : p.vocab < cap ? p.vocab : cap;
    e = launch_overlapped(&k_embed_sum<DT, HC>, dim3((unsigned)(windows + clear), (unsigned)slices),
                          dim3(threads), 0, s, p.n, nv, windows, c, (uint32_t)p.vocab, p.scale,
                          p.accumulate, sorted, (const uint32_t *)w.start, (const uint32_t *)w.end,
                          reinterpret_cast<const uint4 *>(p.dx), table,
                          reinterpret_cast<float4 *>(w.part));
    if (e != cudaSuccess) return e;
    return launch_overlapped(&k_embed_join<DT>,
                             dim3((unsigned)(windows < 64 ? windows : 64),
                                  (unsigned)((nv + 31) / 32)),
                             dim3(256), 0, s, nv, c, p.scale, p.accumulate, sorted,
                             (const uint32_t *)w.longs, (const uint32_t *)w.end,
                             (const float4 *)w.part, table);
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
