// attn.h -- host-side structures of the rotary, attention and cache-attention operators.
#pragma once

#include "internal.h"

namespace dynconv {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A validated rotary problem.
struct RopeProb {
    int dtype;              // 0 fp32, 1 bf16
    int half;               // 0 interleaved pairs, 1 pairs (i, i + rot / 2)
    int inverse;
    int64_t N, seqlen;
    int heads, hd, rot;
    int64_t xs, ys;         // row strides of x and y, elements
    int64_t max_pos;
    const float* cs;
    const int32_t* cu;      // packed documents or nullptr
    int64_t n_docs;
    const int32_t* pos;     // explicit positions or nullptr
};
cudaError_t rope_launch(const RopeProb& p, const void* x, void* y, uint32_t* err, cudaStream_t st);

// A validated attention problem (N < 2^31).
struct AttnProb {
    int dtype, algo;
    int64_t N, seqlen;
    int heads, kvh, hd, group;
    int64_t qs, ks, vs, os, dos, dqs, dks, dvs;   // row strides, elements
    float scale;            // of the scores
    const int32_t* cu;
    int64_t n_docs;
    // of packed documents, written by attn_prep: every token's document (start, end), and the query and key tiles
    // in descending order of their work
    const int2* seg;
    const int32_t *order_q, *order_k;
};
// Workspace of the attention passes: the error word, D[heads][N] of the backward, what attn_prep writes.
struct AttnWs {
    size_t delta, seg, order, total;
};
AttnWs attn_ws(const AttnProb& p, bool packed);
constexpr int kTcTile = 128, kSimtTile = 64;      // tokens per tile of either kernel family
cudaError_t attn_prep(const AttnProb& p, int tile, int2* seg, int32_t* order, uint32_t* err, cudaStream_t st);
// Why the tensor-core kernels do not take the problem (nullptr when they do).
const char* attn_tc_refusal(const AttnProb& p);

cudaError_t attn_simt_fwd(const AttnProb& p, const void* q, const void* k, const void* v, void* o, float* lse,
                          cudaStream_t st);
cudaError_t attn_simt_bwd(const AttnProb& p, const void* d_o, const void* q, const void* k, const void* v,
                          const float* lse, const float* delta, void* dq, void* dk, void* dv, cudaStream_t st);
// bf16 problems attn_tc_refusal has no objection to.
cudaError_t attn_tc_fwd(const AttnProb& p, const void* q, const void* k, const void* v, void* o, float* lse,
                        uint32_t* err, cudaStream_t st);
cudaError_t attn_tc_bwd(const AttnProb& p, const void* d_o, const void* q, const void* k, const void* v,
                        const void* o, const float* lse, float* delta, void* dq, void* dk, void* dv, uint32_t* err,
                        cudaStream_t st);
// D[h][n] = d_o[n, h] . o[n, h], fp32.
cudaError_t attn_delta(const AttnProb& p, const void* d_o, const void* o, float* delta, cudaStream_t st);

// A validated step of new or drafted tokens over a cache.
struct DecodeProb {
    int dtype;
    int64_t batch, max_len;
    int M, heads, kvh, group, hd;                 // M tokens per sequence
    int64_t qs, ks, vs, os;
    int rot, half;                                // rotated channels (0: none), pair layout
    int64_t max_pos;
    const float* cs;
    float scale;
};
int64_t attn_decode_groups(const DecodeProb& p);  // blocks before the cache is split into runs: one counter each
int attn_decode_splits(const DecodeProb& p);
size_t attn_decode_part_bytes(const DecodeProb& p);
cudaError_t attn_decode(const DecodeProb& p, const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
                        const int32_t* lens, const uint64_t* tree, void* o, uint32_t* err, uint32_t* count, float* part,
                        cudaStream_t st);

}  // namespace dynconv
