// attn_tc_fwd.cu -- causal attention forward on the tensor cores (bf16 storage).
//
// A CTA takes 256 consecutive tokens of one query head as two tiles of 128 rows and walks the
// 128-token tiles of keys and values from the first row's document start to the diagonal:
//   S = Q K^T (tcgen05, fp32 in TMEM) -> softmax warps: one row per thread, running maximum and sum in
//   fp32 -> P rounded to bf16, written over S in TMEM -> O += P V (tcgen05, A operand from TMEM).
// P is rounded to bf16 because the tensor cores take it so; its sum is taken before the rounding.
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1, 8 issues the MMAs, 9 the TMA loads, 10 looks at the
// values of masked tiles.  The two tiles alternate: while one's softmax runs, the tensor cores work for
// the other.  TMEM: S0, S1 128 columns each, O0, O1 HD columns each.  tcgen05.mma of one thread run in
// issue order, so S(i+1) may be issued over P(i) right behind the product that reads it, and S(i+1)
// complete means O holds every product up to i: the softmax thread may then rescale its row of O without
// another barrier.  It does so only where the running maximum has grown by more than 2^8 (a stale maximum
// cancels in the division by the sum and costs no precision below that), which after the first tiles is
// rare.
//
// Tiles follow the packed token index, so documents need no list of work.  Masked scores are replaced by
// -inf before the maximum.  P = 0 there, but 0 x NaN is NaN, so warp 10 looks for infinities and NaN among
// the values of tiles that are masked for some row; where it finds one, the rows of that tile are computed
// again one by one over the tokens they see.
#include <algorithm>

#include "attn_tc.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {
namespace attn_tc {
namespace {

constexpr int kFwdThreads = 352;
constexpr float kGrow = 8.f;                     // log2 growth of the maximum that makes a row rescale

template <int HD>
struct FwdSmem {
    static constexpr uint32_t tile = kAtom * (HD / 64);
    static constexpr int slots = HD == 128 ? 4 : 6;
    static constexpr uint32_t bytes = 1024 + tile * (2 + slots);
};

// o and lse of rows row0 .. row0 + count - 1 (one warp's, all below N), over the tokens each sees, row by row.
__device__ __noinline__ void fwd_rows_again(const AttnTcArgs& a, int head, int32_t row0, int count, int lane) {
    const int kv = head / a.group;
    const __nv_bfloat16* kp = a.k + (int64_t)kv * a.hd;
    const __nv_bfloat16* vp = a.v + (int64_t)kv * a.hd;
    const float cs = a.scale * kLog2e;
    for (int r = 0; r < count; ++r) {
        const int32_t n = row0 + r;
        const int32_t s0 = seg_start32(n, a.cu, a.n_docs, a.seqlen);
        const float4 q = row4(a.q + (int64_t)n * a.qs + (int64_t)head * a.hd, lane, a.hd);
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t j = s0; j <= n; ++j) {
            const float s = warp_dot(q, row4(kp + (int64_t)j * a.ks, lane, a.hd)) * cs;
            const float mx = fmaxf(m, s), use = mx == -INFINITY ? 0.f : mx;
            const float c = exp2f(m - use), p = exp2f(s - use);
            acc.x *= c; acc.y *= c; acc.z *= c; acc.w *= c;
            axpy4(acc, p, row4(vp + (int64_t)j * a.vs, lane, a.hd));
            l = l * c + p;
            m = mx;
        }
        const float inv = l > 0.f ? 1.f / l : l;
        put4(a.o + (int64_t)n * a.os + (int64_t)head * a.hd, lane, a.hd,
             make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (a.lse != nullptr && lane == 0) a.lse[(int64_t)head * a.N + n] = (m + log2f(l)) * kLn2;
    }
}

// -inf outside columns from .. to of a row; s holds columns base .. base + 31
__device__ __forceinline__ void hide32(float (&s)[32], int base, int from, int to) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (base + e < from || base + e > to) s[e] = -INFINITY;
}
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

template <int HD>
__global__ void __launch_bounds__(kFwdThreads, 1) attn_fwd_kernel(const __grid_constant__ CUtensorMap tq,
                                                                  const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv,
                                                                  const AttnTcArgs a) {
    using S = FwdSmem<HD>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = align1024(raw);
    uint8_t* sQ = sm;
    uint8_t* sKV = sm + 2 * S::tile;
    __shared__ uint64_t q_full, kv_full[S::slots], kv_empty[S::slots], s_full[2], p_ready[2], o_full[2], scanned, drained;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, again[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.heads, kv = head / a.group;
    const int32_t blocks = (a.N + 2 * kRows - 1) / (2 * kRows);
    const int32_t row0 = (blocks - 1 - (int32_t)(blockIdx.x / a.heads)) * 2 * kRows;      // long rows first
    // tiles of keys that each row tile walks, lo[t] .. hi[t] (none: lo > hi), and the first key that every row sees
    int32_t lo[2], hi[2], full_from[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int32_t r = row0 + t * kRows;
        lo[t] = 0; hi[t] = -1; full_from[t] = 0;
        if (r < a.N) {
            lo[t] = seg_start32(r, a.cu, a.n_docs, a.seqlen) / kRows;
            hi[t] = r / kRows;
            full_from[t] = seg_start32(min(r + kRows, a.N) - 1, a.cu, a.n_docs, a.seqlen);
        }
    }
    const int32_t first = lo[0], last = max(hi[0], hi[1]);
    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        for (int s = 0; s < S::slots; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_ready[t], 4);
            mbar_init(&o_full[t], 1);
            again[t] = 0;
        }
        mbar_init(&scanned, 1);
        mbar_init(&drained, 1);
        abort_flag = 0;
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

    if (warp == 9) {
        // ---- TMA: Q once, then K(i), V(i) in turn through the ring
        if (lane == 0) {
            tma_prefetch(&tk);
            tma_prefetch(&tv);
            mbar_arrive_expect_tx(&q_full, 2 * S::tile);
            load_head_tile<HD>(sQ, &tq, &q_full, head, row0);
            load_head_tile<HD>(sQ + S::tile, &tq, &q_full, head, row0 + kRows);
            int issued = 0;
            for (int32_t i = first; i <= last; ++i) {
                bool ok = true;
#pragma unroll
                for (int w = 0; w < 2 && ok; ++w, ++issued) {
                    const int s = issued % S::slots, use = issued / S::slots;
                    if (use > 0 && !mbar_wait(&kv_empty[s], (use - 1) & 1, &abort_flag, a.err)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&kv_full[s], S::tile);
                    load_head_tile<HD>(sKV + s * S::tile, w ? &tv : &tk, &kv_full[s], kv, i * kRows);
                }
                if (!ok) break;
            }
            if (abort_flag) {       // no copy may land after the CTA has gone
                mbar_wait_drain(&q_full, 0);
                for (int s = 0; s < S::slots && s < issued; ++s)
                    mbar_wait_drain(&kv_full[s], ((issued - 1 - s) / S::slots) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        // ---- MMA
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdO = idesc_bf16(128, HD, false, true);
        const uint32_t q_at = smem_u32(sQ), kv_at = smem_u32(sKV);
        const bool lead = elect_one();
        auto scores = [&](int t, int slot) {
            if (lead) {
#pragma unroll
                for (int c = 0; c < HD / 16; ++c)
                    umma_bf16(tb + 128 * t, kmajor_desc(q_at + t * S::tile + (c / 4) * kAtom, c % 4),
                              kmajor_desc(kv_at + slot * S::tile + (c / 4) * kAtom, c % 4), kIdS, c != 0);
                umma_commit(&s_full[t]);
            }
        };
        bool ok = mbar_wait(&q_full, 0, &abort_flag, a.err) && mbar_wait(&kv_full[0], 0, &abort_flag, a.err);
        tc_fence_after();
        if (ok) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (lo[t] <= first && first <= hi[t]) scores(t, 0);
            if (lead) umma_commit(&kv_empty[0]);
        }
        int at = 1;                                          // ring place of V(i)
        uint32_t phase[2] = {0, 0};
        for (int32_t i = first; ok && i <= last; ++i, at += 2) {
            const int vs = at % S::slots, ks = (at + 1) % S::slots;
            ok = mbar_wait(&kv_full[vs], (at / S::slots) & 1, &abort_flag, a.err);
            if (ok && i < last) ok = mbar_wait(&kv_full[ks], ((at + 1) / S::slots) & 1, &abort_flag, a.err);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (ok && lo[t] <= i && i <= hi[t]) {
                    ok = mbar_wait(&p_ready[t], phase[t], &abort_flag, a.err);
                    phase[t] ^= 1;
                    tc_fence_after();
                    if (ok && lead) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            umma_ts_bf16(tb + 256 + HD * t, tb + 128 * t + 8 * c,
                                         mnmajor_desc(kv_at + vs * S::tile, kAtom, 16 * c), kIdO, i > lo[t] || c > 0);
                        if (i == hi[t]) umma_commit(&o_full[t]);
                    }
                }
                if (ok && lo[t] <= i + 1 && i + 1 <= hi[t]) scores(t, ks);
            }
            if (ok && lead) {
                umma_commit(&kv_empty[vs]);
                if (i < last) umma_commit(&kv_empty[ks]);
            }
            __syncwarp();
        }
        if (lead) umma_commit(&drained);                     // every MMA done before TMEM is freed
        mbar_wait_drain(&drained, 0);
    } else if (warp == 10) {
        // ---- values of masked tiles: infinities and NaN
        int at = 0;
        bool ok = true;
        for (int32_t i = first; ok && i <= last; ++i) {
            for (int w = 0; w < 2 && ok; ++w, ++at) {
                const int s = at % S::slots;
                ok = mbar_wait(&kv_full[s], (at / S::slots) & 1, &abort_flag, a.err);
                if (!ok) break;
                if (w == 1) {
                    bool masked[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        masked[t] = lo[t] <= i && i <= hi[t] && (i == hi[t] || i * kRows < full_from[t]);
                    if ((masked[0] || masked[1]) && tile_nonfinite(sKV + s * S::tile, S::tile, lane) && lane == 0) {
                        if (masked[0]) again[0] = 1;
                        if (masked[1]) again[1] = 1;
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&kv_empty[s]);
            }
        }
        if (lane == 0) mbar_arrive(&scanned);
    } else {
        // ---- softmax: one row per thread
        const int t = warp >> 2;
        const int32_t tile0 = row0 + t * kRows, n = tile0 + (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tb + lanes + 128 * t, tO = tb + lanes + 256 + HD * t;
        const float cs = a.scale * kLog2e;
        const int32_t start = n < a.N ? seg_start32(n, a.cu, a.n_docs, a.seqlen) : INT32_MAX;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // running maximum (log2 units), halves of the sum
        bool ok = true;
        uint32_t phase = 0;
        for (int32_t i = lo[t]; i <= hi[t]; ++i) {
            ok = mbar_wait(&s_full[t], phase, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            phase ^= 1;
            tc_fence_after();
            // Maximum over columns 64-127, then 0-63; the latter stay in registers, the former are read again
            // below (a row of 128 scores next to its probabilities does not fit the registers).
            const bool masked = i == hi[t] || i * kRows < full_from[t];
            const int from = start - i * kRows, to = n - i * kRows;
            float s0[32], s1[32], mx[4];
            tmem_ld32(tS + 64, s0);
            tmem_ld32(tS + 96, s1);
            tmem_wait_ld();
            if (masked) {
                hide32(s0, 64, from, to);
                hide32(s1, 96, from, to);
            }
            mx[0] = max32(s0);
            mx[1] = max32(s1);
            tmem_ld32(tS, s0);
            tmem_ld32(tS + 32, s1);
            tmem_wait_ld();
            if (masked) {
                hide32(s0, 0, from, to);
                hide32(s1, 32, from, to);
            }
            mx[2] = max32(s0);
            mx[3] = max32(s1);
            const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs);
            if (__any_sync(0xFFFFFFFFu, top - m > kGrow)) {
                if (i > lo[t]) {
                    // O is complete up to the previous tile: rescale this row of it
                    const float c = top == -INFINITY ? 1.f : ex2(m - top);
                    l0 *= c;
                    l1 *= c;
#pragma unroll
                    for (int b = 0; b < HD / 32; ++b) {
                        float f[32];
                        tmem_ld32(tO + 32 * b, f);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; e += 2) mul2(f[e], f[e + 1], c);
                        tmem_st32(tO + 32 * b, f);
                    }
                }
                m = top;
            }
            const float neg = m == -INFINITY ? 0.f : -m;     // a row that has seen no key yet
            probs32(s0, cs, neg, l0, l1, tS);
            tmem_ld32(tS + 64, s0);
            probs32(s1, cs, neg, l0, l1, tS + 16);
            tmem_ld32(tS + 96, s1);
            tmem_wait_ld();
            if (masked) {
                hide32(s0, 64, from, to);
                hide32(s1, 96, from, to);
            }
            probs32(s0, cs, neg, l0, l1, tS + 32);
            probs32(s1, cs, neg, l0, l1, tS + 48);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[t]);
        }
        if (lo[t] <= hi[t]) {
            ok = ok && mbar_wait(&o_full[t], 0, &abort_flag, a.err);
            ok = ok && mbar_wait(&scanned, 0, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            const float l = l0 + l1;
            const float inv = l > 0.f ? 1.f / l : l;
            if (ok && !again[t]) {
                __nv_bfloat16* row = a.o + (int64_t)n * a.os + (int64_t)head * a.hd;
#pragma unroll
                for (int b = 0; b < HD / 32; ++b) {
                    float f[32];
                    tmem_ld32(tO + 32 * b, f);
                    tmem_wait_ld();
                    if (n < a.N) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            if (32 * b + e < a.hd)
                                *reinterpret_cast<uint4*>(row + 32 * b + e) =
                                    make_uint4(pack_bf16(f[e] * inv, f[e + 1] * inv), pack_bf16(f[e + 2] * inv, f[e + 3] * inv),
                                               pack_bf16(f[e + 4] * inv, f[e + 5] * inv), pack_bf16(f[e + 6] * inv, f[e + 7] * inv));
                    }
                }
                if (a.lse != nullptr && n < a.N) a.lse[(int64_t)head * a.N + n] = (m + __log2f(l)) * kLn2;
            } else if (ok) {
                const int32_t r = tile0 + (warp & 3) * 32;
                fwd_rows_again(a, head, r, min(32, a.N - r), lane);
            }
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
cudaError_t fwd_hd(const AttnProb& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const AttnTcArgs& a, cudaStream_t st) {
    constexpr uint32_t smem = FwdSmem<HD>::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_fwd_kernel<HD>, smem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((p.N + 2 * kRows - 1) / (2 * kRows) * p.heads);
    DC_LAUNCH(kAttnTcFwd, st, attn_fwd_kernel<HD><<<grid, kFwdThreads, smem, st>>>(tq, tk, tv, a));
    return cudaGetLastError();
}

}  // namespace
}  // namespace attn_tc

const char* attn_tc_refusal(const AttnProb& p) {
    if (p.dtype != 1) return "fp32 storage";
    if (p.hd % 8) return "head_dim is no multiple of 8";
    if (p.qs % 8 || p.ks % 8 || p.vs % 8 || p.os % 8 || p.dos % 8 || p.dqs % 8 || p.dks % 8 || p.dvs % 8)
        return "a row stride is no multiple of 8 elements";
    return nullptr;
}

cudaError_t attn_tc_fwd(const AttnProb& p, const void* q, const void* k, const void* v, void* o, float* lse,
                        uint32_t* err, cudaStream_t st) {
    using namespace attn_tc;
    CUtensorMap tq, tk, tv;
    if (!make_head_map(&tq, q, p.N, p.heads, p.hd, p.qs) || !make_head_map(&tk, k, p.N, p.kvh, p.hd, p.ks) ||
        !make_head_map(&tv, v, p.N, p.kvh, p.hd, p.vs))
        return cudaErrorInvalidValue;
    AttnTcArgs a = tc_args(p);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.err = err;
    return p.hd <= 64 ? fwd_hd<64>(p, tq, tk, tv, a, st) : fwd_hd<128>(p, tq, tk, tv, a, st);
}

}  // namespace dynconv
