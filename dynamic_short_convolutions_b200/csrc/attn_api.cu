// attn_api.cu -- C ABI of the rotary and attention operators: argument validation, workspace sizing,
// kernel-family dispatch.
#include <algorithm>
#include <cmath>

#include "../../include/dynconv_attn.h"
#include "attn.h"

namespace dynconv {

dynconv_status validate_ptr(const void* ptr, const char* name, bool required);

namespace {

constexpr int64_t kMaxBytes = int64_t(1) << 56;

bool fits(int64_t a, int64_t b, int64_t c) {
    int64_t t;
    return !__builtin_mul_overflow(a, b, &t) && !__builtin_mul_overflow(t, c, &t) && t <= kMaxBytes;
}

dynconv_status invalid(const char* what) {
    set_error("%s", what);
    return DYNCONV_ERR_INVALID;
}

dynconv_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return DYNCONV_OK;
    set_error("%s: %s", what, cudaGetErrorString(e));
    return DYNCONV_ERR_CUDA;
}

dynconv_status check_ws(void* ws, size_t ws_bytes, size_t need) {
    if (ws_bytes < need) {
        set_error("workspace %zu bytes, need %zu", ws_bytes, need);
        return DYNCONV_ERR_WORKSPACE;
    }
    return validate_ptr(ws, "ws", true);
}

// Row stride of a tensor: 0 means dense.
bool stride_of(int64_t given, int64_t width, int64_t N, int64_t es, int64_t* out) {
    *out = given ? given : width;
    return *out >= width && fits(std::max<int64_t>(N, 1), *out, es);
}

// Tokens of a dense batch or a packed run; a tile past the last token still has 31-bit indices.
constexpr int64_t kMaxTokens = INT32_MAX - 255;
dynconv_status tokens_of(int64_t batch, int64_t seqlen, int64_t* N) {
    if (batch < 0 || seqlen < 0) return invalid("negative batch/seqlen");
    if (__builtin_mul_overflow(batch, seqlen, N)) return invalid("batch * seqlen overflows 64 bits");
    if (*N > kMaxTokens || seqlen > kMaxTokens) {
        set_error("at most 2^31 - 256 tokens are supported");
        return DYNCONV_ERR_UNSUPPORTED;
    }
    return DYNCONV_OK;
}

dynconv_status check_cu(const int32_t* cu, int64_t n_docs, int64_t batch) {
    if (batch != 1) return invalid("varlen needs batch == 1");
    if (n_docs < 1) return invalid("n_docs must be >= 1");
    if (n_docs > INT32_MAX - 1) return invalid("n_docs must be below 2^31 - 1");
    return validate_ptr(cu, "cu_seqlens", true);
}

// Attention searches cu_seqlens with 32-bit sums of two indices (the rotation with 64-bit ones).
constexpr int64_t kMaxDocs = int64_t(1) << 30;
dynconv_status check_docs(const int32_t* cu, int64_t n_docs, int64_t batch) {
    if (n_docs > kMaxDocs) {
        set_error("at most 2^30 documents are supported");
        return DYNCONV_ERR_UNSUPPORTED;
    }
    return check_cu(cu, n_docs, batch);
}

dynconv_status make_attn(const dynconv_attn_desc* d, AttnProb* p) {
    *p = AttnProb{};
    if (!d) return invalid("desc is NULL");
    if (d->dtype != DYNCONV_F32 && d->dtype != DYNCONV_BF16) { set_error("bad dtype %d", d->dtype); return DYNCONV_ERR_INVALID; }
    if (d->algo < DYNCONV_ALGO_AUTO || d->algo > DYNCONV_ALGO_TC) { set_error("bad algo %d", d->algo); return DYNCONV_ERR_INVALID; }
    dynconv_status s = tokens_of(d->batch, d->seqlen, &p->N);
    if (s != DYNCONV_OK) return s;
    if (d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads) return invalid("kv_heads must divide heads");
    if (d->head_dim < 1) return invalid("head_dim must be >= 1");
    if (d->head_dim > 128) { set_error("head_dim %lld > 128 is not supported", (long long)d->head_dim); return DYNCONV_ERR_UNSUPPORTED; }
    if (d->heads > 65535 || !fits(std::max<int64_t>(p->N, 1), d->heads, 1) || p->N * d->heads > (int64_t(1) << 33)) {
        set_error("tokens * heads beyond 2^33 are not supported");
        return DYNCONV_ERR_UNSUPPORTED;
    }
    if (!(d->scale >= 0.f) || std::isinf(d->scale)) return invalid("scale must be positive and finite (0: 1 / sqrt(head_dim))");
    p->dtype = d->dtype;
    p->algo = d->algo;
    p->seqlen = d->seqlen;
    p->heads = (int)d->heads;
    p->kvh = (int)d->kv_heads;
    p->group = p->heads / p->kvh;
    p->hd = (int)d->head_dim;
    p->scale = d->scale > 0.f ? d->scale : (float)(1.0 / std::sqrt((double)d->head_dim));
    const int64_t es = d->dtype == DYNCONV_BF16 ? 2 : 4, wq = d->heads * d->head_dim, wk = d->kv_heads * d->head_dim;
    if (!stride_of(d->q_row_stride, wq, p->N, es, &p->qs) || !stride_of(d->k_row_stride, wk, p->N, es, &p->ks) ||
        !stride_of(d->v_row_stride, wk, p->N, es, &p->vs) || !stride_of(d->o_row_stride, wq, p->N, es, &p->os) ||
        !stride_of(d->do_row_stride, wq, p->N, es, &p->dos) || !stride_of(d->dq_row_stride, wq, p->N, es, &p->dqs) ||
        !stride_of(d->dk_row_stride, wk, p->N, es, &p->dks) || !stride_of(d->dv_row_stride, wk, p->N, es, &p->dvs))
        return invalid("a row stride is below its row's width, or an operand passes 2^56 bytes");
    if (p->algo == DYNCONV_ALGO_TC) {
        const char* why = attn_tc_refusal(*p);
        if (why) {
            set_error("desc->algo asks for the tensor-core kernels: %s", why);
            return DYNCONV_ERR_UNSUPPORTED;
        }
    }
    return DYNCONV_OK;
}

dynconv_status make_decode(const dynconv_attn_decode_desc* d, DecodeProb* p) {
    *p = DecodeProb{};
    if (!d) return invalid("desc is NULL");
    if (d->dtype != DYNCONV_F32 && d->dtype != DYNCONV_BF16) { set_error("bad dtype %d", d->dtype); return DYNCONV_ERR_INVALID; }
    if (d->batch < 0) return invalid("negative batch");
    if (d->tokens < 1) return invalid("tokens must be >= 1");
    if (d->tokens > 64) { set_error("%lld tokens > 64 are not supported", (long long)d->tokens); return DYNCONV_ERR_UNSUPPORTED; }
    if (d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads) return invalid("kv_heads must divide heads");
    if (d->heads > 65535) { set_error("heads above 65535 are not supported"); return DYNCONV_ERR_UNSUPPORTED; }
    const int64_t es = d->dtype == DYNCONV_BF16 ? 2 : 4, vec = 16 / es;
    if (d->head_dim < 1) return invalid("head_dim must be >= 1");
    if (d->head_dim > 128 || d->head_dim % vec) {
        set_error("head_dim %lld: a multiple of 16 bytes up to 128 channels is supported", (long long)d->head_dim);
        return DYNCONV_ERR_UNSUPPORTED;
    }
    if (d->max_len < d->tokens) return invalid("max_len must hold the new tokens");
    if (d->max_len > INT32_MAX) { set_error("max_len must be below 2^31"); return DYNCONV_ERR_UNSUPPORTED; }
    if (!fits(std::max<int64_t>(d->batch, 1), d->kv_heads * d->head_dim * es, d->max_len)) return invalid("a cache passes 2^56 bytes");
    if (!(d->scale >= 0.f) || std::isinf(d->scale)) return invalid("scale must be positive and finite (0: 1 / sqrt(head_dim))");
    const int64_t wq = d->heads * d->head_dim, wk = d->kv_heads * d->head_dim;
    int64_t N;
    if (__builtin_mul_overflow(d->batch, d->tokens, &N) || !stride_of(d->q_row_stride, wq, N, es, &p->qs) ||
        !stride_of(d->k_row_stride, wk, N, es, &p->ks) || !stride_of(d->v_row_stride, wk, N, es, &p->vs) ||
        !stride_of(d->o_row_stride, wq, N, es, &p->os))
        return invalid("a row stride is below its row's width, or an operand passes 2^56 bytes");
    if (p->qs % vec || p->ks % vec || p->vs % vec || p->os % vec) return invalid("row strides must be multiples of 16 bytes");
    if (d->rope_dim < 0 || d->rope_dim % 2 || d->rope_dim > d->head_dim) return invalid("rope_dim must be even, 0 to head_dim");
    if (d->rope_dim > 0) {
        if (d->rope_layout != DYNCONV_ROPE_INTERLEAVED && d->rope_layout != DYNCONV_ROPE_HALF) { set_error("bad layout %d", d->rope_layout); return DYNCONV_ERR_INVALID; }
        if (d->rope_max_pos < 1 || !fits(d->rope_max_pos, d->rope_dim, 4)) return invalid("rope_max_pos must be >= 1 and the table below 2^56 bytes");
    }
    p->dtype = d->dtype;
    p->batch = d->batch;
    p->max_len = d->max_len;
    p->M = (int)d->tokens;
    p->heads = (int)d->heads;
    p->kvh = (int)d->kv_heads;
    p->group = p->heads / p->kvh;
    p->hd = (int)d->head_dim;
    p->rot = (int)d->rope_dim;
    p->half = d->rope_layout == DYNCONV_ROPE_HALF;
    p->max_pos = d->rope_max_pos;
    p->cs = d->rope_cos_sin;
    p->scale = d->scale > 0.f ? d->scale : (float)(1.0 / std::sqrt((double)d->head_dim));
    if (!fits(std::max<int64_t>(d->batch, 1), d->heads * d->tokens, 64) || attn_decode_groups(*p) > (int64_t(1) << 24)) {
        set_error("batch * kv_heads beyond the grid are not supported");
        return DYNCONV_ERR_UNSUPPORTED;
    }
    return DYNCONV_OK;
}

// Workspace of a step: the error word, a counter per group of runs, the runs' parts.
struct DecodeWs {
    size_t count, part, total;
};
DecodeWs decode_ws(const DecodeProb& p) {
    DecodeWs w{};
    w.count = 256;
    w.part = w.count + ((size_t)attn_decode_groups(p) * sizeof(uint32_t) + 255) / 256 * 256;
    w.total = w.part + attn_decode_part_bytes(p);
    return w;
}

bool attn_tc(const AttnProb& p) { return p.algo != DYNCONV_ALGO_SIMT && attn_tc_refusal(p) == nullptr; }

uint32_t* err_of(void* ws) { return static_cast<uint32_t*>(ws); }

// Packed documents: the check of cu_seqlens and the kernels' view of them, into the workspace.
dynconv_status prepare_docs(AttnProb* p, void* ws, cudaStream_t st) {
    const AttnWs w = attn_ws(*p, true);
    char* base = static_cast<char*>(ws);
    int2* seg = reinterpret_cast<int2*>(base + w.seg);
    int32_t* order = reinterpret_cast<int32_t*>(base + w.order);
    const int tile = attn_tc(*p) ? kTcTile : kSimtTile;
    p->seg = seg;
    p->order_q = order;
    p->order_k = order + (p->N + tile - 1) / tile;
    return cuda_status(attn_prep(*p, tile, seg, order, err_of(ws), st), "packed documents");
}

}  // namespace

AttnWs attn_ws(const AttnProb& p, bool packed) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t N = (size_t)p.N;
    AttnWs w{};
    w.delta = 256;
    w.seg = w.delta + up(N * p.heads * sizeof(float));
    w.order = w.seg + (packed ? up(N * sizeof(int2)) : 0);
    w.total = w.order + (packed ? up(2 * ((N + kSimtTile - 1) / kSimtTile) * sizeof(int32_t)) : 0);
    return w;
}

}  // namespace dynconv

using namespace dynconv;

extern "C" {

dynconv_status dynconv_rope(const dynconv_rope_desc* d, const int32_t* cu_seqlens, int64_t n_docs,
                            const int32_t* positions, const void* x, void* y, void* ws, size_t ws_bytes,
                            void* stream) {
    set_error("%s", "");
    if (!d) return invalid("desc is NULL");
    if (d->dtype != DYNCONV_F32 && d->dtype != DYNCONV_BF16) { set_error("bad dtype %d", d->dtype); return DYNCONV_ERR_INVALID; }
    if (d->layout != DYNCONV_ROPE_INTERLEAVED && d->layout != DYNCONV_ROPE_HALF) { set_error("bad layout %d", d->layout); return DYNCONV_ERR_INVALID; }
    RopeProb p{};
    dynconv_status s = tokens_of(d->batch, d->seqlen, &p.N);
    if (s != DYNCONV_OK) return s;
    if (d->heads < 1 || d->head_dim < 1) return invalid("heads and head_dim must be >= 1");
    if (d->heads > INT32_MAX || d->head_dim > INT32_MAX || d->heads * d->head_dim > INT32_MAX) return invalid("heads * head_dim must be below 2^31");
    if (d->rot_dim < 2 || d->rot_dim % 2 || d->rot_dim > d->head_dim) return invalid("rot_dim must be even, 2 to head_dim");
    if (d->max_pos < 1 || !fits(d->max_pos, d->rot_dim, 4)) return invalid("max_pos must be >= 1 and the table below 2^56 bytes");
    if (d->inverse != 0 && d->inverse != 1) return invalid("inverse must be 0 or 1");
    const int64_t es = d->dtype == DYNCONV_BF16 ? 2 : 4, width = d->heads * d->head_dim;
    if (!stride_of(d->x_row_stride, width, p.N, es, &p.xs) || !stride_of(d->y_row_stride, width, p.N, es, &p.ys))
        return invalid("a row stride is below its row's width, or an operand passes 2^56 bytes");
    if (x != nullptr && x == y && p.xs != p.ys) return invalid("in place needs equal row strides");
    if (cu_seqlens && positions) return invalid("positions and cu_seqlens are given: one of the two at most");
    if (cu_seqlens && (s = check_cu(cu_seqlens, n_docs, d->batch)) != DYNCONV_OK) return s;
    if (p.N == 0) return DYNCONV_OK;
    if (!positions && !cu_seqlens && d->seqlen > d->max_pos) {
        set_error("seqlen %lld exceeds max_pos %lld", (long long)d->seqlen, (long long)d->max_pos);
        return DYNCONV_ERR_INVALID;
    }
    if ((s = validate_ptr(positions, "positions", false)) || (s = validate_ptr(d->cos_sin, "cos_sin", true)) ||
        (s = validate_ptr(x, "x", true)) || (s = validate_ptr(y, "y", true)) || (s = check_ws(ws, ws_bytes, 256)))
        return s;
    p.dtype = d->dtype;
    p.half = d->layout == DYNCONV_ROPE_HALF;
    p.inverse = d->inverse;
    p.seqlen = d->seqlen;
    p.heads = (int)d->heads;
    p.hd = (int)d->head_dim;
    p.rot = (int)d->rot_dim;
    p.max_pos = d->max_pos;
    p.cs = d->cos_sin;
    p.cu = cu_seqlens;
    p.n_docs = n_docs;
    p.pos = positions;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cu_seqlens && (s = cuda_status(launch_check_seqlens(cu_seqlens, n_docs, p.N, err_of(ws), st, p.max_pos),
                                       "cu_seqlens check")))
        return s;
    return cuda_status(rope_launch(p, x, y, err_of(ws), st), "rope launch");
}

size_t dynconv_attn_workspace_bytes(const dynconv_attn_desc* desc) {
    set_error("%s", "");
    AttnProb p;
    if (make_attn(desc, &p) != DYNCONV_OK) return 0;
    return attn_ws(p, desc->batch == 1).total;        // one sequence: packed documents may be given
}

dynconv_status dynconv_attn_query_family(const dynconv_attn_desc* desc, int32_t* fwd_family, int32_t* bwd_family) {
    set_error("%s", "");
    AttnProb p;
    dynconv_status s = make_attn(desc, &p);
    if (s != DYNCONV_OK) return s;
    const char* why = attn_tc_refusal(p);
    const int32_t f = attn_tc(p) ? DYNCONV_FAMILY_TENSOR_CORE : DYNCONV_FAMILY_CUDA_CORE;
    if (fwd_family) *fwd_family = f;
    if (bwd_family) *bwd_family = f;
    if (p.algo == DYNCONV_ALGO_SIMT) set_error("desc->algo asks for the CUDA-core kernels");
    else if (why) set_error("forward and backward on the CUDA-core kernels: %s", why);
    return DYNCONV_OK;
}

dynconv_status dynconv_attn_fwd(const dynconv_attn_desc* desc, const int32_t* cu_seqlens, int64_t n_docs,
                                const void* q, const void* k, const void* v, void* o, float* lse, void* ws,
                                size_t ws_bytes, void* stream) {
    set_error("%s", "");
    AttnProb p;
    dynconv_status s = make_attn(desc, &p);
    if (s != DYNCONV_OK) return s;
    if (cu_seqlens && (s = check_docs(cu_seqlens, n_docs, desc->batch)) != DYNCONV_OK) return s;
    p.cu = cu_seqlens;
    p.n_docs = n_docs;
    if (p.N == 0) return DYNCONV_OK;
    if ((s = validate_ptr(q, "q", true)) || (s = validate_ptr(k, "k", true)) || (s = validate_ptr(v, "v", true)) ||
        (s = validate_ptr(o, "o", true)) || (s = validate_ptr(lse, "lse", false)) ||
        (s = check_ws(ws, ws_bytes, attn_ws(p, desc->batch == 1).total)))
        return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cu_seqlens && (s = prepare_docs(&p, ws, st)) != DYNCONV_OK) return s;
    return cuda_status(attn_tc(p) ? attn_tc_fwd(p, q, k, v, o, lse, err_of(ws), st)
                                  : attn_simt_fwd(p, q, k, v, o, lse, st),
                       "attention forward launch");
}

dynconv_status dynconv_attn_bwd(const dynconv_attn_desc* desc, const int32_t* cu_seqlens, int64_t n_docs,
                                const void* d_o, const void* q, const void* k, const void* v, const void* o,
                                const float* lse, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                void* stream) {
    set_error("%s", "");
    AttnProb p;
    dynconv_status s = make_attn(desc, &p);
    if (s != DYNCONV_OK) return s;
    if (cu_seqlens && (s = check_docs(cu_seqlens, n_docs, desc->batch)) != DYNCONV_OK) return s;
    p.cu = cu_seqlens;
    p.n_docs = n_docs;
    if (p.N == 0) return DYNCONV_OK;
    if ((s = validate_ptr(d_o, "d_o", true)) || (s = validate_ptr(q, "q", true)) || (s = validate_ptr(k, "k", true)) ||
        (s = validate_ptr(v, "v", true)) || (s = validate_ptr(o, "o", true)) || (s = validate_ptr(lse, "lse", true)) ||
        (s = validate_ptr(dq, "dq", true)) || (s = validate_ptr(dk, "dk", true)) || (s = validate_ptr(dv, "dv", true)) ||
        (s = check_ws(ws, ws_bytes, attn_ws(p, desc->batch == 1).total)))
        return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cu_seqlens && (s = prepare_docs(&p, ws, st)) != DYNCONV_OK) return s;
    float* delta = reinterpret_cast<float*>(static_cast<char*>(ws) + attn_ws(p, desc->batch == 1).delta);
    if (attn_tc(p))
        return cuda_status(attn_tc_bwd(p, d_o, q, k, v, o, lse, delta, dq, dk, dv, err_of(ws), st),
                           "attention backward launch");
    if ((s = cuda_status(attn_delta(p, d_o, o, delta, st), "attention row products"))) return s;
    return cuda_status(attn_simt_bwd(p, d_o, q, k, v, lse, delta, dq, dk, dv, st), "attention backward launch");
}

size_t dynconv_attn_decode_workspace_bytes(const dynconv_attn_decode_desc* desc) {
    set_error("%s", "");
    DecodeProb p;
    if (make_decode(desc, &p) != DYNCONV_OK) return 0;
    return decode_ws(p).total;
}

dynconv_status dynconv_attn_decode(const dynconv_attn_decode_desc* desc, const void* q, const void* k, const void* v,
                                   void* k_cache, void* v_cache, const int32_t* lens, const uint64_t* ancestors,
                                   void* o, void* ws, size_t ws_bytes, void* stream) {
    set_error("%s", "");
    DecodeProb p;
    dynconv_status s = make_decode(desc, &p);
    if (s != DYNCONV_OK) return s;
    if (p.batch == 0) return DYNCONV_OK;
    const DecodeWs w = decode_ws(p);
    if ((s = validate_ptr(q, "q", true)) || (s = validate_ptr(k, "k", true)) || (s = validate_ptr(v, "v", true)) ||
        (s = validate_ptr(k_cache, "k_cache", true)) || (s = validate_ptr(v_cache, "v_cache", true)) ||
        (s = validate_ptr(lens, "lens", true)) || (s = validate_ptr(ancestors, "ancestors", false)) ||
        (s = validate_ptr(p.cs, "rope_cos_sin", p.rot > 0)) || (s = validate_ptr(o, "o", true)) ||
        (s = check_ws(ws, ws_bytes, w.total)))
        return s;
    char* base = static_cast<char*>(ws);
    return cuda_status(attn_decode(p, q, k, v, k_cache, v_cache, lens, ancestors, o, err_of(ws),
                                   reinterpret_cast<uint32_t*>(base + w.count), reinterpret_cast<float*>(base + w.part),
                                   static_cast<cudaStream_t>(stream)),
                       "attention decode launch");
}

}  // extern "C"
