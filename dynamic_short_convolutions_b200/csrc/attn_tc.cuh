// attn_tc.cuh -- what the tensor-core attention kernels share: tensor maps over heads, TMEM moves and
// the tcgen05 form whose A operand lies in TMEM, masks of a tile, and the row-by-row recomputation for
// tiles whose masked places hold infinities or NaN.
#pragma once

#include "attn.h"
#include "attn_places.cuh"
#include "common.cuh"
#include "tc_common.cuh"
#include "tmap.h"

namespace dynconv {
namespace attn_tc {

using namespace tc;

constexpr int kRows = kTcTile;                   // 128 tokens per tile: the lanes of TMEM
constexpr uint32_t kAtom = kRows * 128;          // bytes of a 128-token x 64-channel tile

// ---------------------------------------------------------------- tensor maps
// [N tokens][heads][hd] bf16, a box of `rows` tokens x one head x 64 channels; channels from hd on and tokens
// from N on read zero, so every head width up to 128 runs on tiles of 64 or 128 channels.
inline bool make_head_map(CUtensorMap* map, const void* base, int64_t N, int heads, int hd, int64_t row_stride,
                          uint32_t rows = kRows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)N};
    cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)row_stride * 2};
    cuuint32_t box[3] = {64, 1, rows};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// One tile of HD channels (HD / 64 atoms) of a head, 128 tokens from `row` on.
template <int HD>
__device__ __forceinline__ void load_head_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int head,
                                               int32_t row) {
#pragma unroll
    for (int a = 0; a < HD / 64; ++a) tma_load_3d(dst + a * kAtom, map, bar, 64 * a, head, row);
}

// The reverse (one thread); tokens from N on and channels from hd on are not written.
template <int HD>
__device__ __forceinline__ void store_head_tile(const CUtensorMap* map, const uint8_t* src, int head, int32_t row) {
#pragma unroll
    for (int a = 0; a < HD / 64; ++a) tma_store_3d(map, src + a * kAtom, 64 * a, head, row);
}

// ---------------------------------------------------------------- tcgen05 forms
// D[tmem] (+)= A[tmem] * B[smem]: A holds a row per lane, two bf16 of the K index per column.
__device__ __forceinline__ void umma_ts_bf16(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(tmem_d), "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&f)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
          "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&f)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::"r"(__float_as_uint(f[0])), "r"(__float_as_uint(f[1])), "r"(__float_as_uint(f[2])), "r"(__float_as_uint(f[3])),
          "r"(__float_as_uint(f[4])), "r"(__float_as_uint(f[5])), "r"(__float_as_uint(f[6])), "r"(__float_as_uint(f[7])),
          "r"(__float_as_uint(f[8])), "r"(__float_as_uint(f[9])), "r"(__float_as_uint(f[10])),
          "r"(__float_as_uint(f[11])), "r"(__float_as_uint(f[12])), "r"(__float_as_uint(f[13])),
          "r"(__float_as_uint(f[14])), "r"(__float_as_uint(f[15])), "r"(__float_as_uint(f[16])),
          "r"(__float_as_uint(f[17])), "r"(__float_as_uint(f[18])), "r"(__float_as_uint(f[19])),
          "r"(__float_as_uint(f[20])), "r"(__float_as_uint(f[21])), "r"(__float_as_uint(f[22])),
          "r"(__float_as_uint(f[23])), "r"(__float_as_uint(f[24])), "r"(__float_as_uint(f[25])),
          "r"(__float_as_uint(f[26])), "r"(__float_as_uint(f[27])), "r"(__float_as_uint(f[28])),
          "r"(__float_as_uint(f[29])), "r"(__float_as_uint(f[30])), "r"(__float_as_uint(f[31])), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mul2(float& x, float& y, float f) {
    uint64_t a, b;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(b) : "f"(f));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}
// (x, y) = (x f + g, y f + g)
__device__ __forceinline__ void fma2(float& x, float& y, float f, float g) {
    uint64_t a, b, c;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(b) : "f"(f));
    asm("mov.b64 %0, {%1, %1};" : "=l"(c) : "f"(g));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a) : "l"(b), "l"(c));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}
// (x, y) = (x f + g0, y f + g1)
__device__ __forceinline__ void fma2v(float& x, float& y, float f, float g0, float g1) {
    uint64_t a, b, c;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %1};" : "=l"(b) : "f"(f));
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(g0), "f"(g1));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a) : "l"(b), "l"(c));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}
__device__ __forceinline__ void mul2v(float& x, float& y, float f0, float f1) {
    uint64_t a, b;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(f0), "f"(f1));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}
__device__ __forceinline__ void add2(float& x, float& y, float a0, float a1) {
    uint64_t a, b;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(a0), "f"(a1));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
}

// Columns 32 b .. 32 b + 31 of a row of an accumulator, times `mul`, as bf16 into a tile that TMA stores.
__device__ __forceinline__ void tile_put32(uint8_t* tile, uint32_t row, int b, const float (&f)[32], float mul) {
#pragma unroll
    for (int e = 0; e < 32; e += 8)
        *reinterpret_cast<uint4*>(tile + (b / 2) * kAtom + sw128_off(row, (b % 2) * 4 + e / 8)) =
            make_uint4(pack_bf16(f[e] * mul, f[e + 1] * mul), pack_bf16(f[e + 2] * mul, f[e + 3] * mul),
                       pack_bf16(f[e + 4] * mul, f[e + 5] * mul), pack_bf16(f[e + 6] * mul, f[e + 7] * mul));
}

// ---------------------------------------------------------------- masks
// Columns from .. to of a tile are seen by a row.  What a warp's rows see of columns base .. base + 31: in the
// diagonal tile most such runs are seen by all of its rows or by none, and only the rest is masked one by one.
enum { kSeeNone = 0, kSeeSome = 1, kSeeAll = 2 };
__device__ __forceinline__ int seen_run(int base, int from, int to) {
    if (__all_sync(0xFFFFFFFFu, from <= base && to >= base + 31)) return kSeeAll;
    return __any_sync(0xFFFFFFFFu, from <= base + 31 && to >= base && from <= to) ? kSeeSome : kSeeNone;
}
// A bit per column of the run that the row sees.
__device__ __forceinline__ uint32_t seen_bits(int base, int from, int to) {
    const int lo = from - base, hi = to - base;
    const uint32_t upto = hi >= 31 ? ~0u : hi < 0 ? 0u : (2u << hi) - 1;
    return lo <= 0 ? upto : lo > 31 ? 0u : upto & (~0u << lo);
}
__device__ __forceinline__ void fill32(float (&s)[32], float x) {
#pragma unroll
    for (int e = 0; e < 32; ++e) s[e] = x;
}
// Columns a row does not see become `x`.
__device__ __forceinline__ void hide32(float (&s)[32], uint32_t bits, float x) {
#pragma unroll
    for (int e = 0; e < 32; ++e) s[e] = bits >> e & 1 ? s[e] : x;
}

// ---------------------------------------------------------------- softmax of a row
constexpr float kGrow = 8.f;                     // log2 growth of the maximum that makes a row rescale
__device__ __forceinline__ float max32(const float (&s)[32]) {
    float a = fmaxf(s[0], s[1]), b = fmaxf(s[2], s[3]);
#pragma unroll
    for (int e = 4; e < 32; e += 4) {
        a = fmaxf(fmaxf(a, s[e]), s[e + 1]);
        b = fmaxf(fmaxf(b, s[e + 2]), s[e + 3]);
    }
    return fmaxf(a, b);
}
// 32 probabilities 2^(s f + g): summed (even and odd columns apart), rounded to bf16 and stored to 16 columns of TMEM
__device__ __forceinline__ void probs32(float (&s)[32], float f, float g, float& l0, float& l1, uint32_t to) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        fma2(s[e], s[e + 1], f, g);
        s[e] = ex2(s[e]);
        s[e + 1] = ex2(s[e + 1]);
        add2(l0, l1, s[e], s[e + 1]);
        w[e / 2] = pack_bf16(s[e], s[e + 1]);
    }
    tmem_st16(to, w);
}

__device__ __forceinline__ void zeros16(uint32_t to) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = 0;
    tmem_st16(to, w);
}


// ---------------------------------------------------------------- infinities and NaN
// Whether a word of two bf16 holds an infinity or a NaN (an exponent of ones): bit 7 of either half of
// the sum is set only then, and the low half's sum does not carry.
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// True when a tile of `bytes` in shared memory holds an infinity or a NaN (one warp reads it).
__device__ __forceinline__ bool tile_nonfinite(const uint8_t* tile, uint32_t bytes, int lane) {
    uint32_t bad = 0;
#pragma unroll 4
    for (uint32_t o = lane * 16; o < bytes; o += 512) {
        const uint4 w = *reinterpret_cast<const uint4*>(tile + o);
        bad |= nonfinite_bits(w.x) | nonfinite_bits(w.y) | nonfinite_bits(w.z) | nonfinite_bits(w.w);
    }
    return __any_sync(0xFFFFFFFFu, bad != 0);
}

// Four channels (4 lane .. 4 lane + 3) of a row; zero beyond hd.
__device__ __forceinline__ float4 row4(const __nv_bfloat16* p, int lane, int hd) {
    if (4 * lane >= hd) return make_float4(0.f, 0.f, 0.f, 0.f);
    const uint2 w = *reinterpret_cast<const uint2*>(p + 4 * lane);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, int lane, int hd, float4 f) {
    if (4 * lane >= hd) return;
    *reinterpret_cast<uint2*>(p + 4 * lane) = make_uint2(pack_bf16(f.x, f.y), pack_bf16(f.z, f.w));
}
__device__ __forceinline__ float warp_dot(float4 a, float4 b) {
    float s = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}
__device__ __forceinline__ void axpy4(float4& a, float f, float4 x) {
    a.x = fmaf(f, x.x, a.x);
    a.y = fmaf(f, x.y, a.y);
    a.z = fmaf(f, x.z, a.z);
    a.w = fmaf(f, x.w, a.w);
}

struct AttnTcArgs {
    int32_t N, seqlen;
    int heads, kvh, group, hd;
    const int2* seg;
    const int32_t *order_q, *order_k;
    float scale;
    uint32_t* err;
    // plain addresses, for the rows recomputed one by one and the outputs
    const __nv_bfloat16 *q, *k, *v, *d_o;
    __nv_bfloat16 *o, *dq, *dk, *dv;
    float* lse;
    float* delta;                                // D [heads][N], written by the dq kernel, read by the other
    int64_t qs, ks, vs, os, dos, dqs, dks, dvs;
};

inline AttnTcArgs tc_args(const AttnProb& p) {
    AttnTcArgs a{};
    a.N = (int32_t)p.N;
    a.seqlen = (int32_t)p.seqlen;
    a.heads = p.heads;
    a.kvh = p.kvh;
    a.group = p.group;
    a.hd = p.hd;
    a.seg = p.seg;
    a.order_q = p.order_q;
    a.order_k = p.order_k;
    a.scale = p.scale;
    a.qs = p.qs; a.ks = p.ks; a.vs = p.vs; a.os = p.os;
    a.dos = p.dos; a.dqs = p.dqs; a.dks = p.dks; a.dvs = p.dvs;
    return a;
}

}  // namespace attn_tc
}  // namespace dynconv
