// attn_places.cuh -- where a token's sequence or document lies, and the order of an attention kernel's tiles.
#pragma once

#include <cstdint>

namespace dynconv {

// Start and end (one past the last token) of token n's sequence in a dense batch, or its document, read from the
// table that the attention's preparation writes (seg, non-null for packed documents).
__device__ __forceinline__ int2 doc_of(int32_t n, const int2* __restrict__ seg, int32_t seqlen) {
    if (seg != nullptr) return __ldg(seg + n);
    const int32_t s = n - (int32_t)((uint32_t)n % (uint32_t)seqlen);
    return make_int2(s, s + seqlen);
}
// The u-th tile to be worked on, the ones with the most work first: from the table for packed documents, else
// by place in the sequence (late queries, early keys) where sequences are whole tiles, else by token.
__device__ __forceinline__ int32_t tile_of(int32_t u, int32_t tiles, int32_t per_seq, const int32_t* __restrict__ order,
                                           bool keys) {
    if (order != nullptr) return __ldg(order + u);
    if (per_seq > 0) {
        const int32_t seqs = tiles / per_seq, at = u / seqs;
        return (u - at * seqs) * per_seq + (keys ? at : per_seq - 1 - at);
    }
    return keys ? u : tiles - 1 - u;
}

}  // namespace dynconv
