// hc_kept.cu -- rows kept in 8 bits (hc_kept.cuh has the format): to them, back
// from them, the expansion that keeps its result, and the collapse from kept
// copies.
//
// All four are HBM streams: each input is read once and each output written
// once.  A lane moves vectors of 8 channels, 16 bytes of bf16 or 8 of codes,
// several in flight; the vectors of all rows are numbered through (Slots), so
// that narrow rows fill the warps as wide ones do, and four neighbouring lanes
// hold the 32 channels of a block: its largest magnitude takes two shuffles
// and nothing leaves the registers.
#include "hc_kept.cuh"

namespace hc {
namespace {

// Slot i stands for vector i % per of row i / per (in k_checkpoint: a pair of
// vectors); per covers whole blocks (4 vectors), so the lanes of a block never
// span two rows, and a row's last slots may lie past its end.  At most 2^31
// slots a launch: larger tensors take several.
struct Slots {
    uint32_t count;       // rows * per
    uint32_t per;         // slots per row
    uint32_t nv;          // vectors per row (d / 8)
    uint32_t mul, shift;  // i / per = (i * mul) >> (32 + shift), i < 2^31
    __device__ __forceinline__ void at(uint32_t i, int64_t &row, uint32_t &v) const {
        const uint32_t q = __umulhi(i, mul) >> shift;
        row = q;
        v = i - q * per;
    }
};

// With l = ceil(log2 per) and mul = ceil(2^(31+l) / per) the product's error
// is below 2^l * 2^31 / 2^(31+l) / per, so the quotient is exact for i < 2^31.
Slots make_slots(int64_t rows, int64_t d, int per_block = 4) {
    Slots s;
    s.nv = (uint32_t)(d / 8);
    s.per = (uint32_t)(kept_blocks(d) * per_block);
    s.count = (uint32_t)(rows * s.per);
    int l = 1;
    while ((int64_t(1) << l) < s.per) ++l;
    s.mul = (uint32_t)(((uint64_t(1) << (31 + l)) + s.per - 1) / s.per);
    s.shift = (uint32_t)(l - 1);
    return s;
}

// Calls f(first row, rows) for pieces of at most 2^30 slots.
template <typename Fn>
cudaError_t by_pieces(int64_t rows, int64_t d, Fn f) {
    const int64_t most = (int64_t(1) << 30) / (kept_blocks(d) * 4);
    for (int64_t r = 0; r < rows; r += most) {
        const cudaError_t e = f(r, rows - r < most ? rows - r : most);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// ---------------------------------------------------------- k_checkpoint
// A lane takes 16 channels where the other kernels take 8: two lanes a block,
// one shuffle, and 16 bytes of codes a store.  65,536 tokens of 4 x 5120 (4.07
// GB): 647 us, 6.3 TB/s; with 8 channels a lane 780 us.  A row's last lane may
// have 8.
template <int U>
__global__ void __launch_bounds__(256, 5) k_checkpoint(Slots sl, int64_t nblk,
                                                    const uint4 *__restrict__ x,
                                                    uint2 *__restrict__ codes,
                                                    uint8_t *__restrict__ scales) {
    griddep_wait_then_release();
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * 256u * U;
    const bool wide = sl.nv % 2 == 0;  // then 16 codes are 16-byte aligned
    for (uint32_t i0 = (blockIdx.x * 256u + (threadIdx.x & ~31u)) * U; i0 < sl.count; i0 += step) {
        uint4 r[U][2];
        int64_t row[U];
        uint32_t v[U];
#pragma unroll
        for (int a = 0; a < U; ++a) {
            sl.at(i0 + 32 * a + lane, row[a], v[a]);
            v[a] *= 2;
            if (i0 + 32 * a + lane >= sl.count) v[a] = sl.nv;
            const uint4 *p = x + row[a] * sl.nv + v[a];
            r[a][0] = v[a] < sl.nv ? ld_stream(p) : make_uint4(0, 0, 0, 0);
            r[a][1] = v[a] + 1 < sl.nv ? ld_stream(p + 1) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int a = 0; a < U; ++a) {
            uint32_t m = max(kept_largest(r[a][0]), kept_largest(r[a][1]));
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            const uint32_t byte = kept_scale_byte(m);
            const uint2 lo = kept_codes(r[a][0], byte), hi = kept_codes(r[a][1], byte);
            if (v[a] < sl.nv) {
                uint2 *p = codes + row[a] * sl.nv + v[a];
                if (wide) {
                    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(lo.x, lo.y, hi.x, hi.y));
                } else {
                    __stcs(p, lo);
                    if (v[a] + 1 < sl.nv) __stcs(p + 1, hi);
                }
                if ((lane & 1) == 0) scales[row[a] * nblk + (v[a] >> 2)] = (uint8_t)byte;
            }
        }
    }
}

// ------------------------------------------------------------- k_restore
// 16,384 tokens of 4 x 5120 (1.02 GB): 160 us, 6.35 TB/s.
template <int U>
__global__ void __launch_bounds__(256) k_restore(Slots sl, int64_t nblk, Kept k,
                                                 uint4 *__restrict__ x) {
    griddep_wait_then_release();
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * 256u * U;
    for (uint32_t i0 = (blockIdx.x * 256u + (threadIdx.x & ~31u)) * U; i0 < sl.count; i0 += step) {
        KeptVec<true> r[U];
        int64_t row[U];
        uint32_t v[U];
#pragma unroll
        for (int a = 0; a < U; ++a) {
            sl.at(i0 + 32 * a + lane, row[a], v[a]);
            if (i0 + 32 * a + lane >= sl.count) v[a] = sl.nv;
            if (v[a] < sl.nv) r[a].load(k, row[a], sl.nv, nblk, v[a]);
        }
#pragma unroll
        for (int a = 0; a < U; ++a) {
            if (v[a] < sl.nv) {
                float f[8];
                r[a].values(f);
                st_stream(x + row[a] * sl.nv + v[a], pack8(f));
            }
        }
    }
}

// --------------------------------------------------------- k_pre_restore
// y = sum_j pre_j x_j of kept copies, the copies in the order of hc_pre.  16,384
// tokens of 4 x 5120 (514 MB): 80 us, 6.4 TB/s; of 8 x 5120 (860 MB): 144 us, 6.0 TB/s.
template <int HC, int U>
__global__ void __launch_bounds__(256, HC == 4 ? 4 : 6) k_pre_restore(Slots sl, int64_t nblk, Kept k,
                                                     const float *__restrict__ pre,
                                                     uint4 *__restrict__ y) {
    griddep_wait_then_release();
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * 256u * U;
    for (uint32_t i0 = (blockIdx.x * 256u + (threadIdx.x & ~31u)) * U; i0 < sl.count; i0 += step) {
        KeptVec<true> r[U][HC];
        int64_t t[U];
        uint32_t v[U];
#pragma unroll
        for (int a = 0; a < U; ++a) {
            sl.at(i0 + 32 * a + lane, t[a], v[a]);
            if (i0 + 32 * a + lane >= sl.count) v[a] = sl.nv;
            if (v[a] < sl.nv) {
#pragma unroll
                for (int j = 0; j < HC; ++j) r[a][j].load(k, t[a] * HC + j, sl.nv, nblk, v[a]);
            }
        }
#pragma unroll
        for (int a = 0; a < U; ++a) {
            if (v[a] < sl.nv) {
                float acc[8], f[8];
#pragma unroll
                for (int q = 0; q < HC / 4; ++q) {
                    const float4 p = __ldg(reinterpret_cast<const float4 *>(pre + t[a] * HC) + q);
                    const float pj[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        r[a][4 * q + j].values(f);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[e] = q + j == 0 ? pj[0] * f[e] : fmaf(pj[j], f[e], acc[e]);
                    }
                }
                st_stream(y + t[a] * sl.nv + v[a], pack8(acc));
            }
        }
    }
}

// ------------------------------------------------------ k_post_checkpoint
// hc_post whose bf16 result is quantised before it leaves the registers: the
// new stream is not read back for its checkpoint.  The sums run in hc_post's
// order, so y is hc_post's bit for bit.  residual may equal y: a lane loads
// every copy of a vector before it stores any of them.  Coefficients are
// loaded per vector, row by row of comb: they hit the first-level cache, and
// only the accumulators stay in registers.  16,384 tokens of 4 x 5120 (1.86 GB):
// 300 us, 6.2 TB/s (one vector in flight and one-wide FMAs: 335 us); 4,096 of
// 8 x 5120 (886 MB): 186 us, 4.8 TB/s (128 registers leave 16 warps an SM).
template <int HC, int U>
__global__ void __launch_bounds__(256, 2) k_post_checkpoint(Slots sl, int64_t nblk,
                                                            const uint4 *__restrict__ out,
                                                            const uint4 *res,
                                                            const float *__restrict__ post,
                                                            const float *__restrict__ comb,
                                                            uint4 *y, uint2 *__restrict__ codes,
                                                            uint8_t *__restrict__ scales) {
    griddep_wait_then_release();
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * 256u * U;
    for (uint32_t i0 = (blockIdx.x * 256u + (threadIdx.x & ~31u)) * U; i0 < sl.count; i0 += step) {
        int64_t t[U];
        uint32_t v[U];
        bool in[U];
        uint4 o[U], r[U][HC];
#pragma unroll
        for (int a = 0; a < U; ++a) {
            sl.at(i0 + 32 * a + lane, t[a], v[a]);
            in[a] = i0 + 32 * a + lane < sl.count && v[a] < sl.nv;
            if (!in[a]) t[a] = 0, v[a] = 0;  // a row that exists, for the coefficients
            o[a] = in[a] ? ld_stream(out + t[a] * sl.nv + v[a]) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < HC; ++j)
                r[a][j] = in[a] ? ld_stream(res + (t[a] * HC + j) * sl.nv + v[a])
                                : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int a = 0; a < U; ++a) {
            // two copies wide: acc[p][e] is channel e of copies 2p and 2p+1, and the
            // coefficients' pairs are loaded as they lie
            uint64_t acc[HC / 2][8], c[HC / 2];
            float f[8];
            unpack8(o[a], f);
            auto load_row = [&](const float *p) {
#pragma unroll
                for (int q = 0; q < HC / 4; ++q) {
                    const ulonglong2 w = __ldg(reinterpret_cast<const ulonglong2 *>(p) + q);
                    c[2 * q] = w.x, c[2 * q + 1] = w.y;
                }
            };
            load_row(post + t[a] * HC);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t fe = pack2(f[e], f[e]);
#pragma unroll
                for (int p = 0; p < HC / 2; ++p) acc[p][e] = fmul2(c[p], fe);
            }
#pragma unroll
            for (int j = 0; j < HC; ++j) {
                unpack8(r[a][j], f);
                load_row(comb + (t[a] * HC + j) * HC);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint64_t fe = pack2(f[e], f[e]);
#pragma unroll
                    for (int p = 0; p < HC / 2; ++p) ffma2(acc[p][e], c[p], fe);
                }
            }
#pragma unroll
            for (int k = 0; k < HC; ++k) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float lo, hi;
                    unpack2(acc[k / 2][e], lo, hi);
                    f[e] = k % 2 ? hi : lo;
                }
                const uint4 p = pack8(f);
                uint32_t byte;
                const uint2 c8 = kept_quantise(p, byte);
                if (in[a]) {
                    const int64_t row = t[a] * HC + k;
                    st_stream(y + row * sl.nv + v[a], p);
                    __stcs(codes + row * sl.nv + v[a], c8);
                    if ((lane & 3) == 0) scales[row * nblk + (v[a] >> 2)] = (uint8_t)byte;
                }
            }
        }
    }
}

// As many blocks as are resident at once (each kernel's launch bounds): they
// share the slots evenly, where more blocks would leave a last partial wave
// (k_checkpoint 674 -> 643 us; k_restore was 2 us faster with 8 than with its 5).
dim3 stream_grid(const Slots &sl, int u, int sms, int blocks_per_sm) {
    const int64_t per_block = 256 * u;
    const int64_t want = (sl.count + per_block - 1) / per_block;
    const int64_t cap = (int64_t)sms * blocks_per_sm;
    return dim3((unsigned)(want < cap ? want : cap));
}

Kept rows_from(const Kept &k, int64_t row, int64_t d) {
    return Kept{static_cast<const uint8_t *>(k.data) + row * d, k.scales + row * kept_blocks(d)};
}

}  // namespace

cudaError_t launch_checkpoint(int64_t rows, int64_t d, const uint16_t *x, uint8_t *codes,
                              uint8_t *scales, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nblk = kept_blocks(d);
    return by_pieces(rows, d, [&](int64_t r0, int64_t nr) {
        const Slots sl = make_slots(nr, d, 2);
        return launch_overlapped(k_checkpoint<2>, stream_grid(sl, 2, di.sms, 5), dim3(256), 0, s,
                                 sl, nblk, reinterpret_cast<const uint4 *>(x + r0 * d),
                                 reinterpret_cast<uint2 *>(codes + r0 * d), scales + r0 * nblk);
    });
}

cudaError_t launch_restore(int64_t rows, int64_t d, const Kept &k, uint16_t *x,
                           const DeviceInfo &di, cudaStream_t s) {
    const int64_t nblk = kept_blocks(d);
    return by_pieces(rows, d, [&](int64_t r0, int64_t nr) {
        const Slots sl = make_slots(nr, d);
        return launch_overlapped(k_restore<4>, stream_grid(sl, 4, di.sms, 8), dim3(256), 0, s, sl,
                                 nblk, rows_from(k, r0, d), reinterpret_cast<uint4 *>(x + r0 * d));
    });
}

cudaError_t launch_pre_restore(int64_t n, int hc, int64_t d, const Kept &k, const float *pre,
                               uint16_t *y, const DeviceInfo &di, cudaStream_t s) {
    const int64_t nblk = kept_blocks(d);
    return by_pieces(n, d, [&](int64_t t0, int64_t nt) {
        const Slots sl = make_slots(nt, d);
        uint4 *yv = reinterpret_cast<uint4 *>(y + t0 * d);
        const Kept kt = rows_from(k, t0 * hc, d);
        return hc == 4 ? launch_overlapped(k_pre_restore<4, 2>, stream_grid(sl, 2, di.sms, 4),
                                           dim3(256), 0, s, sl, nblk, kt, pre + t0 * hc, yv)
                       : launch_overlapped(k_pre_restore<8, 1>, stream_grid(sl, 1, di.sms, 6),
                                           dim3(256), 0, s, sl, nblk, kt, pre + t0 * hc, yv);
    });
}

cudaError_t launch_post_checkpoint(int64_t n, int hc, int64_t d, const uint16_t *out,
                                   const uint16_t *res, const float *post, const float *comb,
                                   uint16_t *y, uint8_t *codes, uint8_t *scales,
                                   const DeviceInfo &di, cudaStream_t s) {
    const int64_t nblk = kept_blocks(d);
    return by_pieces(n, d, [&](int64_t t0, int64_t nt) {
        const Slots sl = make_slots(nt, d);
        const dim3 grid = stream_grid(sl, hc == 4 ? 2 : 1, di.sms, 2);
        const int64_t row = t0 * hc;
        const uint4 *ov = reinterpret_cast<const uint4 *>(out + t0 * d);
        const uint4 *rv = reinterpret_cast<const uint4 *>(res + row * d);
        uint4 *yv = reinterpret_cast<uint4 *>(y + row * d);
        uint2 *cv = reinterpret_cast<uint2 *>(codes + row * d);
        auto *kernel = hc == 4 ? &k_post_checkpoint<4, 2> : &k_post_checkpoint<8, 1>;
        return launch_overlapped(kernel, grid, dim3(256), 0, s, sl, nblk, ov, rv, post + row,
                                 comb + row * hc, yv, cv, scales + row * nblk);
    });
}

}  // namespace hc
