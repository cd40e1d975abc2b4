// hc_embed_order.h -- tokens in order of their ids (hc_embed_order.cu).
#pragma once

#include "hc_internal.h"

namespace hc {

// What the order leaves, and its scratch; all of it device memory of the caller's.
struct TokenOrder {
    uint2 *sorted[2];   // [n] (id, token) in [0]; ids outside the table last, as `vocab`
    uint32_t *hist;     // scratch, order_hist_bytes(n)
    uint32_t *present;  // a bit for each row of the table: some token names it
    uint32_t *start;    // [vocab], first place of an id that is present
    uint32_t *end;      // [vocab], the place behind its last
    uint32_t *count;    // one word, set to 0
};
size_t order_hist_bytes(int64_t n);
cudaError_t launch_order(int64_t n, int64_t vocab, int id_bytes, const void *ids,
                         const TokenOrder &o, cudaStream_t s);

}  // namespace hc
