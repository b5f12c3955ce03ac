// attn_tc_bwd.cu -- causal attention backward on the tensor cores (bf16 storage).
//
//   P = exp(scale S - lse),  dP = dO V^T,  dS = P (dP - D)
//   dV = P^T dO,  dK = scale dS^T Q   (over every query of the document, every head of the group)
//   dQ = scale dS K                   (over every key the query sees)
//
// Two kernels, each with its sums in TMEM for its whole run and written once: attn_dkv_kernel takes 128
// keys of one key/value head and walks the query tiles of every head of the group; attn_dq_kernel takes 128
// queries of one head and walks the key tiles.  S and dP are computed in both (7 products of a tile pair
// where one fused kernel needs 5), because the fused kernel would add a 128 x HD fp32 tile of dQ into global
// memory for every tile pair -- 64 KB per 2.6 us of tensor work and SM at HD = 128, above what L2 reduces --
// and in an order that changes from run to run.  Here nothing is added atomically and results repeat bitwise.
//
// No operand passes through shared memory by hand: the transposed scores S^T = K Q^T put keys on the TMEM
// lanes, P^T and dS^T are written back to TMEM as bf16 and are the A operands of dV and dK; in attn_dq_kernel
// dS is the A operand of dQ.  P and dS are rounded to bf16 because the tensor cores take them so; dS is
// computed from the fp32 P.
//
// Warps: 0-7 the element work (a lane is a row; warps 0-3 take columns 0-63, 4-7 columns 64-127, each
// writing its bf16 results over scores that it alone has read), 8 MMA issue, 9 TMA, 10 infinities and NaN in
// masked tiles (see attn_tc_fwd.cu), 11 (dkv) the rows' lse and D.  MMAs run in issue order, and the order
// is chosen so that the tensor cores have the other half of the work while the element warps do theirs:
//   dkv: dV(i) S(i+1) | dK(i) dP(i+1)    while the element warps compute dS(i) | P(i+1)
//   dq:  S(i+1) dP(i+1) dQ(i)            while they compute P(i), dS(i), from registers
#include <algorithm>

#include "attn_tc.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {
namespace attn_tc {
namespace {

constexpr int kBwdThreads = 384;

template <int HD>
struct BwdSmem {
    static constexpr uint32_t tile = kAtom * (HD / 64);
    static constexpr int stages = HD == 128 ? 2 : 4;
    static constexpr uint32_t stats = stages * 2 * kRows * sizeof(float);       // lse and D of a stage's queries
    static constexpr uint32_t bytes = 1024 + tile * (2 + 2 * stages) + stats;
};

// p (columns base .. base + 31 of a row) = 2^(s f - lse2), 0 outside columns from .. to where masked
__device__ __forceinline__ void hide32z(float (&s)[32], int base, int from, int to) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (base + e < from || base + e > to) s[e] = 0.f;
}
__device__ __forceinline__ void store32(uint32_t to, const float (&f)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
    tmem_st16(to, w);
}
// 32 columns of an accumulator, times `mul`, to channels base .. base + 31 of a row (hd of them are real)
__device__ __forceinline__ void put32(__nv_bfloat16* row, int base, int hd, const float (&f)[32], float mul) {
#pragma unroll
    for (int e = 0; e < 32; e += 8)
        if (base + e < hd)
            *reinterpret_cast<uint4*>(row + base + e) =
                make_uint4(pack_bf16(f[e] * mul, f[e + 1] * mul), pack_bf16(f[e + 2] * mul, f[e + 3] * mul),
                           pack_bf16(f[e + 4] * mul, f[e + 5] * mul), pack_bf16(f[e + 6] * mul, f[e + 7] * mul));
}

// dk and dv of `count` keys from key0 on (all below N), key by key over the queries that see it.
__device__ __noinline__ void dkv_rows_again(const AttnTcArgs& a, int kv, int32_t key0, int count, int lane) {
    const float cs = a.scale * kLog2e;
    for (int r = 0; r < count; ++r) {
        const int32_t j = key0 + r;
        int32_t s0, end;
        seg_bounds32(j, a.cu, a.n_docs, a.seqlen, a.N, s0, end);
        const float4 k = row4(a.k + (int64_t)j * a.ks + (int64_t)kv * a.hd, lane, a.hd);
        const float4 v = row4(a.v + (int64_t)j * a.vs + (int64_t)kv * a.hd, lane, a.hd);
        float4 dk = make_float4(0.f, 0.f, 0.f, 0.f), dv = dk;
        for (int g = 0; g < a.group; ++g) {
            const int64_t h = kv * a.group + g;
            for (int32_t n = j; n < end; ++n) {
                const float4 q = row4(a.q + (int64_t)n * a.qs + h * a.hd, lane, a.hd);
                const float4 d = row4(a.d_o + (int64_t)n * a.dos + h * a.hd, lane, a.hd);
                const float p = exp2f(fmaf(warp_dot(q, k), cs, -a.lse[h * a.N + n] * kLog2e));
                const float ds = p * (warp_dot(d, v) - a.delta[h * a.N + n]);
                axpy4(dv, p, d);
                axpy4(dk, ds, q);
            }
        }
        put4(a.dv + (int64_t)j * a.dvs + (int64_t)kv * a.hd, lane, a.hd, dv);
        put4(a.dk + (int64_t)j * a.dks + (int64_t)kv * a.hd, lane, a.hd,
             make_float4(dk.x * a.scale, dk.y * a.scale, dk.z * a.scale, dk.w * a.scale));
    }
}

// dq of `count` queries from row0 on (all below N), row by row over the keys it sees.
__device__ __noinline__ void dq_rows_again(const AttnTcArgs& a, int head, int32_t row0, int count, int lane) {
    const int kv = head / a.group;
    const float cs = a.scale * kLog2e;
    for (int r = 0; r < count; ++r) {
        const int32_t n = row0 + r;
        const float4 q = row4(a.q + (int64_t)n * a.qs + (int64_t)head * a.hd, lane, a.hd);
        const float4 d = row4(a.d_o + (int64_t)n * a.dos + (int64_t)head * a.hd, lane, a.hd);
        const float ls = a.lse[(int64_t)head * a.N + n] * kLog2e, dl = a.delta[(int64_t)head * a.N + n];
        float4 dq = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t j = seg_start32(n, a.cu, a.n_docs, a.seqlen); j <= n; ++j) {
            const float4 k = row4(a.k + (int64_t)j * a.ks + (int64_t)kv * a.hd, lane, a.hd);
            const float4 v = row4(a.v + (int64_t)j * a.vs + (int64_t)kv * a.hd, lane, a.hd);
            const float p = exp2f(fmaf(warp_dot(q, k), cs, -ls));
            axpy4(dq, p * (warp_dot(d, v) - dl), k);
        }
        put4(a.dq + (int64_t)n * a.dqs + (int64_t)head * a.hd, lane, a.hd,
             make_float4(dq.x * a.scale, dq.y * a.scale, dq.z * a.scale, dq.w * a.scale));
    }
}

// ---------------------------------------------------------------- dk, dv
template <int HD>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dkv_kernel(const __grid_constant__ CUtensorMap tq,
                                                                  const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv,
                                                                  const __grid_constant__ CUtensorMap td,
                                                                  const AttnTcArgs a) {
    using S = BwdSmem<HD>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = align1024(raw);
    uint8_t* sK = sm;
    uint8_t* sV = sm + S::tile;
    uint8_t* sQ = sm + 2 * S::tile;                          // stage s: Q at sQ + 2 s tile, dO behind it
    float* sStat = reinterpret_cast<float*>(sm + (2 + 2 * S::stages) * S::tile);
    __shared__ uint64_t kv_full, full[S::stages], empty[S::stages], s_full, dp_full, p_ready, ds_ready, done, scanned;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, again;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kv = blockIdx.x % a.kvh;
    const int32_t key0 = (int32_t)(blockIdx.x / a.kvh) * kRows;          // early keys have the most queries
    int32_t s0, full_to, e_last;
    seg_bounds32(key0, a.cu, a.n_docs, a.seqlen, a.N, s0, full_to);      // queries below it see every key of the tile
    seg_bounds32(min(key0 + kRows, a.N) - 1, a.cu, a.n_docs, a.seqlen, a.N, s0, e_last);
    const int32_t t0 = key0 / kRows, per_head = (e_last - 1) / kRows - t0 + 1;
    const int64_t items = (int64_t)per_head * a.group;
    if (threadIdx.x == 0) {
        mbar_init(&kv_full, 1);
        for (int s = 0; s < S::stages; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 2);
        }
        mbar_init(&s_full, 1);
        mbar_init(&dp_full, 1);
        mbar_init(&p_ready, 8);
        mbar_init(&ds_ready, 8);
        mbar_init(&done, 1);
        mbar_init(&scanned, 1);
        abort_flag = 0;
        again = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base;
    constexpr uint32_t kDP = 128, kDV = 256, kDK = 256 + HD;

    if (warp == 9) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&kv_full, 2 * S::tile);
            load_head_tile<HD>(sK, &tk, &kv_full, kv, key0);
            load_head_tile<HD>(sV, &tv, &kv_full, kv, key0);
            int64_t issued = 0;
            int32_t g = 0, t = 0;
            for (; issued < items; ++issued) {
                const int s = (int)(issued % S::stages);
                const int64_t use = issued / S::stages;
                if (use > 0 && !mbar_wait(&empty[s], (uint32_t)(use - 1) & 1, &abort_flag, a.err)) break;
                mbar_arrive_expect_tx(&full[s], 2 * S::tile);
                load_head_tile<HD>(sQ + 2 * s * S::tile, &tq, &full[s], kv * a.group + g, (t0 + t) * kRows);
                load_head_tile<HD>(sQ + (2 * s + 1) * S::tile, &td, &full[s], kv * a.group + g, (t0 + t) * kRows);
                if (++t == per_head) { t = 0; ++g; }
            }
            if (abort_flag) {
                mbar_wait_drain(&kv_full, 0);
                for (int s = 0; s < S::stages && s < issued; ++s)
                    mbar_wait_drain(&full[s], (uint32_t)((issued - 1 - s) / S::stages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdG = idesc_bf16(128, HD, false, true);
        const uint32_t k_at = smem_u32(sK), v_at = smem_u32(sV), q_at = smem_u32(sQ);
        const bool lead = elect_one();
        // D (128 columns at `to`) = A B^T of two K-major tiles
        auto nt = [&](uint32_t to, uint32_t A, uint32_t B, uint64_t* bar) {
            if (lead) {
#pragma unroll
                for (int c = 0; c < HD / 16; ++c)
                    umma_bf16(tb + to, kmajor_desc(A + (c / 4) * kAtom, c % 4), kmajor_desc(B + (c / 4) * kAtom, c % 4),
                              kIdS, c != 0);
                umma_commit(bar);
            }
        };
        // D (HD columns at `to`) += the bf16 rows at `from` (columns 0-63 and 64-127 of the tile 64 columns apart) X
        auto grad = [&](uint32_t to, uint32_t from, uint32_t X, bool add) {
            if (lead) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    umma_ts_bf16(tb + to, tb + from + (c < 4 ? 8 * c : 64 + 8 * (c - 4)), mnmajor_desc(X, kAtom, 16 * c),
                                 kIdG, add || c > 0);
            }
        };
        bool ok = mbar_wait(&kv_full, 0, &abort_flag, a.err) && mbar_wait(&full[0], 0, &abort_flag, a.err);
        tc_fence_after();
        if (ok) {
            nt(0, k_at, q_at, &s_full);
            nt(kDP, v_at, q_at + S::tile, &dp_full);
        }
        uint32_t phase = 0;
        for (int64_t i = 0; ok && i < items; ++i, phase ^= 1) {
            const uint32_t at = q_at + 2 * (uint32_t)(i % S::stages) * S::tile;
            const int ns = (int)((i + 1) % S::stages);
            const uint32_t next = q_at + 2 * ns * S::tile;
            ok = mbar_wait(&p_ready, phase, &abort_flag, a.err);
            tc_fence_after();
            if (ok) grad(kDV, 0, at + S::tile, i > 0);
            if (ok && i + 1 < items) {
                ok = mbar_wait(&full[ns], (uint32_t)((i + 1) / S::stages) & 1, &abort_flag, a.err);
                tc_fence_after();
                if (ok) nt(0, k_at, next, &s_full);
            }
            ok = ok && mbar_wait(&ds_ready, phase, &abort_flag, a.err);
            tc_fence_after();
            if (ok) {
                grad(kDK, kDP, at, i > 0);
                if (lead) umma_commit(&empty[i % S::stages]);
                if (i + 1 < items) nt(kDP, v_at, next + S::tile, &dp_full);
            }
            __syncwarp();
        }
        if (lead) umma_commit(&done);                        // every MMA done
        mbar_wait_drain(&done, 0);
    } else if (warp == 10) {
        bool ok = true;
        int32_t t = 0;
        for (int64_t i = 0; ok && i < items; ++i) {
            const int s = (int)(i % S::stages);
            ok = mbar_wait(&full[s], (uint32_t)(i / S::stages) & 1, &abort_flag, a.err);
            if (!ok) break;
            if (t == 0 || (t0 + t + 1) * kRows > full_to) {
                if (tile_nonfinite(sQ + 2 * s * S::tile, 2 * S::tile, lane) && lane == 0) again = 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (++t == per_head) t = 0;
        }
        if (lane == 0) mbar_arrive(&scanned);
    } else if (warp == 11) {
        // lse (log2 units, negated) and D of each stage's queries: read ahead, four per lane
        int32_t g = 0, t = 0;
        float ls[4], dl[4];
        auto fetch = [&]() {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t n = (t0 + t) * kRows + 4 * lane + e;
                const int64_t at = (int64_t)(kv * a.group + g) * a.N + n;
                ls[e] = n < a.N ? -a.lse[at] * kLog2e : 0.f;
                dl[e] = n < a.N ? a.delta[at] : 0.f;
            }
            if (++t == per_head) { t = 0; ++g; }
        };
        fetch();
        for (int64_t i = 0; i < items; ++i) {
            const int s = (int)(i % S::stages);
            const int64_t use = i / S::stages;
            if (use > 0 && !mbar_wait(&empty[s], (uint32_t)(use - 1) & 1, &abort_flag, a.err)) break;
            float4* st = reinterpret_cast<float4*>(sStat + s * 2 * kRows);
            st[lane] = make_float4(ls[0], ls[1], ls[2], ls[3]);
            st[32 + lane] = make_float4(dl[0], dl[1], dl[2], dl[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
            if (i + 1 < items) fetch();
        }
    } else {
        const int w = warp >> 2;                             // columns 64 w .. 64 w + 63
        const int32_t j = key0 + (warp & 3) * 32 + lane;
        const uint32_t at = tb + ((uint32_t)((warp & 3) * 32) << 16) + 64 * w;
        const float cs = a.scale * kLog2e;
        int32_t end = 0;
        if (j < a.N) seg_bounds32(j, a.cu, a.n_docs, a.seqlen, a.N, s0, end);
        bool ok = true;
        uint32_t phase = 0;
        int32_t t = 0;
        for (int64_t i = 0; i < items; ++i, phase ^= 1) {
            const int32_t q0 = (t0 + t) * kRows;
            const bool masked = t == 0 || q0 + kRows > full_to;
            const int from = j - q0 - 64 * w, to = end - 1 - q0 - 64 * w;
            const float* st = sStat + (i % S::stages) * 2 * kRows + 64 * w;
            ok = mbar_wait(&full[i % S::stages], (uint32_t)(i / S::stages) & 1, &abort_flag, a.err) &&
                 mbar_wait(&s_full, phase, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            float p[2][32], f[32];
            tmem_ld32(at, p[0]);
            tmem_ld32(at + 32, p[1]);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 l = *reinterpret_cast<const float4*>(st + 32 * b + e);
                    fma2v(p[b][e], p[b][e + 1], cs, l.x, l.y);
                    fma2v(p[b][e + 2], p[b][e + 3], cs, l.z, l.w);
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) p[b][e] = ex2(p[b][e]);
                if (masked) hide32z(p[b], 32 * b, from, to);
                store32(at + 16 * b, p[b]);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready);
            ok = mbar_wait(&dp_full, phase, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            float f2[32];
            tmem_ld32(at + kDP, f);
            tmem_ld32(at + kDP + 32, f2);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float(&x)[32] = b ? f2 : f;
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 d = *reinterpret_cast<const float4*>(st + kRows + 32 * b + e);
                    add2(x[e], x[e + 1], -d.x, -d.y);
                    add2(x[e + 2], x[e + 3], -d.z, -d.w);
                    mul2v(x[e], x[e + 1], p[b][e], p[b][e + 1]);
                    mul2v(x[e + 2], x[e + 3], p[b][e + 2], p[b][e + 3]);
                }
                if (masked) hide32z(x, 32 * b, from, to);
                store32(at + kDP + 16 * b, x);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ds_ready);
            if (++t == per_head) t = 0;
        }
        ok = ok && mbar_wait(&done, 0, &abort_flag, a.err) && mbar_wait(&scanned, 0, &abort_flag, a.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && !again) {
            // warps 0-3 write dv, warps 4-7 dk
            __nv_bfloat16* row = w ? a.dk + (int64_t)j * a.dks : a.dv + (int64_t)j * a.dvs;
            row += (int64_t)kv * a.hd;
            const uint32_t src = tb + ((uint32_t)((warp & 3) * 32) << 16) + (w ? kDK : kDV);
            const float mul = w ? a.scale : 1.f;
#pragma unroll
            for (int b = 0; b < HD / 32; ++b) {
                float f[32];
                tmem_ld32(src + 32 * b, f);
                tmem_wait_ld();
                if (j < a.N) put32(row, 32 * b, a.hd, f, mul);
            }
        } else if (ok) {
            const int32_t r = key0 + warp * 16;
            dkv_rows_again(a, kv, r, min(16, a.N - r), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

// ---------------------------------------------------------------- dq
template <int HD>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dq_kernel(const __grid_constant__ CUtensorMap tq,
                                                                 const __grid_constant__ CUtensorMap tk,
                                                                 const __grid_constant__ CUtensorMap tv,
                                                                 const __grid_constant__ CUtensorMap td,
                                                                 const AttnTcArgs a) {
    using S = BwdSmem<HD>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = align1024(raw);
    uint8_t* sQ = sm;
    uint8_t* sO = sm + S::tile;
    uint8_t* sK = sm + 2 * S::tile;                          // stage s: K at sK + 2 s tile, V behind it
    __shared__ uint64_t q_full, full[S::stages], empty[S::stages], s_full, dp_full, s_free, dp_free, ds_ready, done, scanned;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, again;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.heads, kv = head / a.group;
    const int32_t tiles = (a.N + kRows - 1) / kRows;
    const int32_t row0 = (tiles - 1 - (int32_t)(blockIdx.x / a.heads)) * kRows;           // long rows first
    const int32_t lo = seg_start32(row0, a.cu, a.n_docs, a.seqlen) / kRows, hi = row0 / kRows;
    const int32_t full_from = seg_start32(min(row0 + kRows, a.N) - 1, a.cu, a.n_docs, a.seqlen);
    const int32_t items = hi - lo + 1;
    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        for (int s = 0; s < S::stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        mbar_init(&s_full, 1);
        mbar_init(&dp_full, 1);
        mbar_init(&s_free, 8);
        mbar_init(&dp_free, 8);
        mbar_init(&ds_ready, 8);
        mbar_init(&done, 1);
        mbar_init(&scanned, 1);
        abort_flag = 0;
        again = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = tmem_base;
    constexpr uint32_t kDP = 128, kDQ = 256, kDS = 384;      // dS: two buffers of 64 columns

    if (warp == 9) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&q_full, 2 * S::tile);
            load_head_tile<HD>(sQ, &tq, &q_full, head, row0);
            load_head_tile<HD>(sO, &td, &q_full, head, row0);
            int32_t issued = 0;
            for (; issued < items; ++issued) {
                const int s = issued % S::stages, use = issued / S::stages;
                if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1, &abort_flag, a.err)) break;
                mbar_arrive_expect_tx(&full[s], 2 * S::tile);
                load_head_tile<HD>(sK + 2 * s * S::tile, &tk, &full[s], kv, (lo + issued) * kRows);
                load_head_tile<HD>(sK + (2 * s + 1) * S::tile, &tv, &full[s], kv, (lo + issued) * kRows);
            }
            if (abort_flag) {
                mbar_wait_drain(&q_full, 0);
                for (int s = 0; s < S::stages && s < issued; ++s)
                    mbar_wait_drain(&full[s], ((issued - 1 - s) / S::stages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdG = idesc_bf16(128, HD, false, true);
        const uint32_t q_at = smem_u32(sQ), o_at = smem_u32(sO), k_at = smem_u32(sK);
        const bool lead = elect_one();
        auto nt = [&](uint32_t to, uint32_t A, uint32_t B, uint64_t* bar) {
            if (lead) {
#pragma unroll
                for (int c = 0; c < HD / 16; ++c)
                    umma_bf16(tb + to, kmajor_desc(A + (c / 4) * kAtom, c % 4), kmajor_desc(B + (c / 4) * kAtom, c % 4),
                              kIdS, c != 0);
                umma_commit(bar);
            }
        };
        bool ok = mbar_wait(&q_full, 0, &abort_flag, a.err) && mbar_wait(&full[0], 0, &abort_flag, a.err);
        tc_fence_after();
        if (ok) {
            nt(0, q_at, k_at, &s_full);
            nt(kDP, o_at, k_at + S::tile, &dp_full);
        }
        uint32_t phase = 0;
        for (int32_t i = 0; ok && i < items; ++i, phase ^= 1) {
            const uint32_t at = k_at + 2 * (i % S::stages) * S::tile;
            const int ns = (i + 1) % S::stages;
            const uint32_t next = k_at + 2 * ns * S::tile;
            if (i + 1 < items) {
                ok = mbar_wait(&full[ns], ((i + 1) / S::stages) & 1, &abort_flag, a.err) &&
                     mbar_wait(&s_free, phase, &abort_flag, a.err);
                tc_fence_after();
                if (ok) nt(0, q_at, next, &s_full);
                ok = ok && mbar_wait(&dp_free, phase, &abort_flag, a.err);
                tc_fence_after();
                if (ok) nt(kDP, o_at, next + S::tile, &dp_full);
            }
            ok = ok && mbar_wait(&ds_ready, phase, &abort_flag, a.err);
            tc_fence_after();
            if (ok && lead) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    umma_ts_bf16(tb + kDQ, tb + kDS + 64 * (i & 1) + 8 * c, mnmajor_desc(at, kAtom, 16 * c), kIdG,
                                 i > 0 || c > 0);
                umma_commit(&empty[i % S::stages]);
            }
            __syncwarp();
        }
        if (lead) umma_commit(&done);
        mbar_wait_drain(&done, 0);
    } else if (warp == 10) {
        bool ok = true;
        for (int32_t i = 0; ok && i < items; ++i) {
            const int s = i % S::stages;
            ok = mbar_wait(&full[s], (i / S::stages) & 1, &abort_flag, a.err);
            if (!ok) break;
            if (i == items - 1 || (lo + i) * kRows < full_from) {
                if (tile_nonfinite(sK + 2 * s * S::tile, S::tile, lane) && lane == 0) again = 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        if (lane == 0) mbar_arrive(&scanned);
    } else if (warp < 8) {
        const int w = warp >> 2;
        const int32_t n = row0 + (warp & 3) * 32 + lane;
        const uint32_t at = tb + ((uint32_t)((warp & 3) * 32) << 16) + 64 * w;
        const uint32_t ds_at = tb + ((uint32_t)((warp & 3) * 32) << 16) + kDS + 32 * w;
        const float cs = a.scale * kLog2e;
        const int32_t start = n < a.N ? seg_start32(n, a.cu, a.n_docs, a.seqlen) : INT32_MAX;
        const float ls = n < a.N ? -a.lse[(int64_t)head * a.N + n] * kLog2e : 0.f;
        const float dl = n < a.N ? -a.delta[(int64_t)head * a.N + n] : 0.f;
        bool ok = true;
        uint32_t phase = 0;
        for (int32_t i = 0; i < items; ++i, phase ^= 1) {
            const int32_t c0 = (lo + i) * kRows;
            const bool masked = i == items - 1 || c0 < full_from;
            const int from = start - c0 - 64 * w, to = n - c0 - 64 * w;
            ok = mbar_wait(&s_full, phase, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            float p[2][32], f[2][32];
            tmem_ld32(at, p[0]);
            tmem_ld32(at + 32, p[1]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    fma2(p[b][e], p[b][e + 1], cs, ls);
                    p[b][e] = ex2(p[b][e]);
                    p[b][e + 1] = ex2(p[b][e + 1]);
                }
            ok = mbar_wait(&dp_full, phase, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            tmem_ld32(at + kDP, f[0]);
            tmem_ld32(at + kDP + 32, f[1]);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dp_free);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    add2(f[b][e], f[b][e + 1], dl, dl);
                    mul2v(f[b][e], f[b][e + 1], p[b][e], p[b][e + 1]);
                }
                if (masked) hide32z(f[b], 32 * b, from, to);
                store32(ds_at + 64 * (i & 1) + 16 * b, f[b]);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ds_ready);
        }
        ok = ok && mbar_wait(&done, 0, &abort_flag, a.err) && mbar_wait(&scanned, 0, &abort_flag, a.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        tc_fence_after();
        if (ok && !again) {
            __nv_bfloat16* row = a.dq + (int64_t)n * a.dqs + (int64_t)head * a.hd;
#pragma unroll
            for (int b = 0; b < HD / 64; ++b) {              // each half of the warps writes half of the channels
                const int c = 32 * (b + w * (HD / 64));
                float f[32];
                tmem_ld32(tb + ((uint32_t)((warp & 3) * 32) << 16) + kDQ + c, f);
                tmem_wait_ld();
                if (n < a.N) put32(row, c, a.hd, f, a.scale);
            }
        } else if (ok) {
            const int32_t r = row0 + warp * 16;
            dq_rows_again(a, head, r, min(16, a.N - r), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
}

template <int HD>
cudaError_t bwd_hd(const AttnProb& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& td, const AttnTcArgs& a, cudaStream_t st) {
    constexpr uint32_t smem = BwdSmem<HD>::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_dkv_kernel<HD>, smem);
    if (e == cudaSuccess) e = DC_SMEM_LIMIT(attn_dq_kernel<HD>, smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + kRows - 1) / kRows;
    DC_LAUNCH(kAttnTcDkv, st, attn_dkv_kernel<HD><<<(unsigned)(tiles * p.kvh), kBwdThreads, smem, st>>>(tq, tk, tv, td, a));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    DC_LAUNCH(kAttnTcDq, st, attn_dq_kernel<HD><<<(unsigned)(tiles * p.heads), kBwdThreads, smem, st>>>(tq, tk, tv, td, a));
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn_tc

cudaError_t attn_tc_bwd(const AttnProb& p, const void* d_o, const void* q, const void* k, const void* v,
                        const float* lse, const float* delta, void* dq, void* dk, void* dv, uint32_t* err,
                        cudaStream_t st) {
    using namespace attn_tc;
    CUtensorMap tq, tk, tv, td;
    if (!make_head_map(&tq, q, p.N, p.heads, p.hd, p.qs) || !make_head_map(&tk, k, p.N, p.kvh, p.hd, p.ks) ||
        !make_head_map(&tv, v, p.N, p.kvh, p.hd, p.vs) || !make_head_map(&td, d_o, p.N, p.heads, p.hd, p.dos))
        return cudaErrorInvalidValue;
    AttnTcArgs a = tc_args(p);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.d_o = static_cast<const __nv_bfloat16*>(d_o);
    a.dq = static_cast<__nv_bfloat16*>(dq);
    a.dk = static_cast<__nv_bfloat16*>(dk);
    a.dv = static_cast<__nv_bfloat16*>(dv);
    a.lse = const_cast<float*>(lse);
    a.delta = delta;
    a.err = err;
    return p.hd <= 64 ? bwd_hd<64>(p, tq, tk, tv, td, a, st) : bwd_hd<128>(p, tq, tk, tv, td, a, st);
}

}  // namespace dynconv
