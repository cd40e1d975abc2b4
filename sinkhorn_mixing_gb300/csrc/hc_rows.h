// hc_rows.h -- launchers of the norm and of the embedding (not part of the public
// ABI).  Arguments are validated before.
#pragma once

#include "../../include/hcmix.h"
#include "hc_internal.h"

namespace hc {

inline int row_type_bytes(int dtype) { return dtype == HC_F32 ? 4 : 2; }

// y = (x - mean) / sqrt(var + eps) * weight + bias (hc_rownorm.cu)
struct RowNorm {
    int64_t rows, d;
    int dtype;
    bool center;
    float eps;
    const void *x;
    const float *weight, *bias;  // null: ones, zeros
    void *y;
};
cudaError_t launch_norm(const RowNorm &p, const DeviceInfo &di, cudaStream_t s);

// its gradients (hc_rownorm_bwd.cu)
struct RowNormBackward {
    int64_t rows, d;
    int dtype;
    bool center;
    float eps;
    const void *dy, *x;
    const float *weight;
    void *dx;
    float *dweight, *dbias;  // each may be null
    uint8_t *ws;
};
size_t norm_backward_bytes(int64_t rows, int64_t d, int dtype);
cudaError_t launch_norm_backward(const RowNormBackward &p, const DeviceInfo &di, cudaStream_t s);

// rows of a table into the copies of a stream (hc_embed.cu)
struct Embed {
    int64_t n, d, vocab;
    int hc, id_bytes, dtype;
    float scale;
    const void *ids, *table;
    uint16_t *x;
};
cudaError_t launch_embed(const Embed &p, const DeviceInfo &di, cudaStream_t s);

// the table's gradient (hc_embed_bwd.cu)
struct EmbedBackward {
    int64_t n, d, vocab;
    int hc, id_bytes, dtype;
    float scale;
    bool accumulate;
    const void *ids;
    const uint16_t *dx;
    void *dtable;
    uint8_t *ws;
};
size_t embed_backward_bytes(int64_t n, int64_t d, int64_t vocab);
cudaError_t launch_embed_backward(const EmbedBackward &p, const DeviceInfo &di, cudaStream_t s);

}  // namespace hc
