// hc_abi_rows.cu -- the C entry points of the norm and of the embedding: host-side
// argument validation and launch; nothing here allocates memory.
#include "hc_check.h"
#include "hc_rows.h"

using namespace hc::check;

namespace {

hc_status check_type(int dtype) {
    return dtype == HC_BF16 || dtype == HC_F16 || dtype == HC_F32 ? HC_OK : HC_ERR_UNSUPPORTED;
}

// rows of d channels of at most 4 bytes: the byte counts stay inside int64
hc_status check_rows(int64_t rows, int64_t d) {
    if (rows < 0 || d <= 0) return HC_ERR_INVALID_ARG;
    if (d % 8 != 0) return HC_ERR_MISALIGNED;
    if (d > (int64_t(1) << 24) || rows > (int64_t(1) << 58) / d) return HC_ERR_UNSUPPORTED;
    return HC_OK;
}

hc_status check_embed(int64_t n, int hc, int64_t d, int64_t vocab, int id_bytes, int dtype,
                      float scale) {
    hc_status st = check_rows(n, d);
    if (st != HC_OK) return st;
    if (vocab < 1 || !(scale > -INFINITY && scale < INFINITY)) return HC_ERR_INVALID_ARG;
    if ((hc != 1 && hc != 4 && hc != 8) || (id_bytes != 4 && id_bytes != 8) ||
        vocab > INT32_MAX - 1 || n > (int64_t(1) << 30))
        return HC_ERR_UNSUPPORTED;
    return check_type(dtype);
}

// null, or on a 16-byte boundary
bool maybe16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if (!al16(p)) return false;
    return true;
}

Range maybe(const void *p, uint64_t bytes) { return p ? rng(p, bytes) : Range{0, 0}; }

}  // namespace

extern "C" {

hc_status hc_norm(int64_t rows, int64_t d, int dtype, int center, float eps, const void *x,
                  const float *weight, const float *bias, void *y, hc_stream_t stream) {
    hc_status st = check_rows(rows, d);
    if (st != HC_OK || (st = check_type(dtype)) != HC_OK) return st;
    if (!finite_nonneg(eps)) return HC_ERR_INVALID_ARG;
    if (rows == 0) return HC_OK;
    if ((st = ptrs_ok({x, y})) != HC_OK) return st;
    if (!maybe16({weight, bias})) return HC_ERR_MISALIGNED;
    const uint64_t bytes = (uint64_t)rows * d * hc::row_type_bytes(dtype);
    const Range ry = rng(y, bytes);
    if ((y != x && overlap(ry, rng(x, bytes))) ||
        !disjoint({ry}, {maybe(weight, d * 4), maybe(bias, d * 4)}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_norm(
        hc::RowNorm{rows, d, dtype, center != 0, eps, x, weight, bias, y}, di,
        reinterpret_cast<cudaStream_t>(stream)));
}

size_t hc_norm_backward_bytes(int64_t rows, int64_t d, int dtype) {
    if (check_rows(rows, d) != HC_OK || check_type(dtype) != HC_OK || rows == 0) return 0;
    return hc::norm_backward_bytes(rows, d, dtype);
}

hc_status hc_norm_backward(int64_t rows, int64_t d, int dtype, int center, float eps,
                           const void *dy, const void *x, const float *weight, void *dx,
                           float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                           hc_stream_t stream) {
    hc_status st = check_rows(rows, d);
    if (st != HC_OK || (st = check_type(dtype)) != HC_OK) return st;
    if (!finite_nonneg(eps)) return HC_ERR_INVALID_ARG;
    if (!maybe16({weight, dweight, dbias})) return HC_ERR_MISALIGNED;
    const uint64_t par = (uint64_t)d * 4, bytes = (uint64_t)rows * d * hc::row_type_bytes(dtype);
    const Range rw = maybe(dweight, par), rb = maybe(dbias, par);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        // no rows: the parameters' gradients are zero, not left as they were
        if (!disjoint({rw, rb}, {maybe(weight, par)})) return HC_ERR_INVALID_ARG;
        cudaError_t e = dweight ? cudaMemsetAsync(dweight, 0, par, s) : cudaSuccess;
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, par, s);
        return from_cuda(e);
    }
    if ((st = ptrs_ok({dy, x, dx})) != HC_OK) return st;
    const size_t need = hc::norm_backward_bytes(rows, d, dtype);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need) return HC_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return HC_ERR_MISALIGNED;
    }
    const Range rdx = rng(dx, bytes), rdy = rng(dy, bytes),
                rws = need > 0 ? rng(workspace, workspace_bytes) : Range{0, 0};
    if ((dx != dy && overlap(rdx, rdy)) ||
        !disjoint({rdx, rw, rb, rws}, {rng(x, bytes), maybe(weight, par)}) ||
        !disjoint({rw, rb, rws}, {rdy}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_norm_backward(
        hc::RowNormBackward{rows, d, dtype, center != 0, eps, dy, x, weight, dx, dweight, dbias,
                            static_cast<uint8_t *>(workspace)},
        di, s));
}

hc_status hc_embed(int64_t n, int hc, int64_t d, int64_t vocab, int id_bytes, int dtype,
                   float scale, const void *ids, const void *table, uint16_t *x,
                   hc_stream_t stream) {
    hc_status st = check_embed(n, hc, d, vocab, id_bytes, dtype, scale);
    if (st != HC_OK) return st;
    if (n == 0) return HC_OK;
    if (ids == nullptr) return HC_ERR_INVALID_ARG;
    if ((st = ptrs_ok({table, x})) != HC_OK) return st;
    if ((reinterpret_cast<uintptr_t>(ids) & (uintptr_t)(id_bytes - 1)) != 0)
        return HC_ERR_MISALIGNED;
    if (!disjoint({rng(x, (uint64_t)n * hc * d * 2)},
                  {rng(ids, (uint64_t)n * id_bytes),
                   rng(table, (uint64_t)vocab * d * hc::row_type_bytes(dtype))}))
        return HC_ERR_INVALID_ARG;
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_embed(
        hc::Embed{n, d, vocab, hc, id_bytes, dtype, scale, ids, table, x}, di,
        reinterpret_cast<cudaStream_t>(stream)));
}

size_t hc_embed_backward_bytes(int64_t n, int64_t d, int64_t vocab) {
    if (check_embed(n, 1, d, vocab, 4, HC_F32, 1.0f) != HC_OK || n == 0) return 0;
    return hc::embed_backward_bytes(n, d, vocab);
}

hc_status hc_embed_backward(int64_t n, int hc, int64_t d, int64_t vocab, int id_bytes, int dtype,
                            float scale, int accumulate, const void *ids, const uint16_t *dx,
                            void *dtable, void *workspace, size_t workspace_bytes,
                            hc_stream_t stream) {
    hc_status st = check_embed(n, hc, d, vocab, id_bytes, dtype, scale);
    if (st != HC_OK || (st = ptrs_ok({dtable})) != HC_OK) return st;
    if (n > 0) {
        if (ids == nullptr) return HC_ERR_INVALID_ARG;
        if ((st = ptrs_ok({dx})) != HC_OK) return st;
        if ((reinterpret_cast<uintptr_t>(ids) & (uintptr_t)(id_bytes - 1)) != 0)
            return HC_ERR_MISALIGNED;
        if (workspace == nullptr || workspace_bytes < hc::embed_backward_bytes(n, d, vocab))
            return HC_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return HC_ERR_MISALIGNED;
        if (!disjoint({rng(dtable, (uint64_t)vocab * d * hc::row_type_bytes(dtype)),
                       rng(workspace, workspace_bytes)},
                      {rng(ids, (uint64_t)n * id_bytes), rng(dx, (uint64_t)n * hc * d * 2)}))
            return HC_ERR_INVALID_ARG;
    }
    hc::DeviceInfo di;
    if (hc::device_info(&di) != cudaSuccess) return cuda_failed();
    return from_cuda(hc::launch_embed_backward(
        hc::EmbedBackward{n, d, vocab, hc, id_bytes, dtype, scale, accumulate != 0, ids, dx, dtable,
                          static_cast<uint8_t *>(workspace)},
        di, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
