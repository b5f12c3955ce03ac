// attn_tc_fwd.cu -- causal attention forward on the tensor cores (bf16 storage).
//
// A CTA takes 128 consecutive tokens of one query head and walks the 128-token tiles of keys and values from
// the first row's document start to the diagonal:
//   S = Q K^T (tcgen05, fp32 in TMEM) -> softmax warps: one row per thread, running maximum and sum in
//   fp32 -> P rounded to bf16 in TMEM -> O += P V (tcgen05, A operand from TMEM).
// P is rounded to bf16 because the tensor cores take it so; its sum is taken before the rounding.
//
// Two CTAs share an SM (half of its TMEM and shared memory each): one's softmax runs while the tensor cores
// work for the other, and so do its prologue and epilogue, which a CTA of 256 rows per SM left bare.
// Warps: 0-3 softmax, 4 issues the MMAs, 5 the TMA loads; 6 warps at 168 registers are what fits twice.
// TMEM (256 columns): S 128, O HD; P lies over S at HD = 128 and beside it at HD = 64, where the next
// scores can then be computed as soon as this tile's are read.
//
// The softmax thread rescales its row of O only where the running maximum has grown by more than 2^8 (a stale
// maximum cancels in the division by the sum and costs no precision below that), which after the first tiles is
// rare.
//
// Tiles follow the packed token index, so documents need no list of work.  Masked scores are replaced by
// -inf before the maximum.  P = 0 there, but 0 x NaN is NaN, so the softmax warps look for infinities and NaN
// among the values of tiles that are masked for some row; where they find one, the rows of the CTA are computed
// again one by one over the tokens they see.
//
// Measured: 4 sequences of 4096, 16 heads of 128 over 4: 263 us at 1965 MHz, 1045 TFLOP/s (0.64 of the measured
// matrix-product rate), and 299 to 304 us in calls that follow one another, where the power cap (989 W) holds the clock
// at 1605 to 1627 MHz: the same number of cycles.  The tensor pipe is busy for 52 % of them, that of the exponentials
// for 52 %; the rest is the chain of an item's steps that two blocks do not hide.  One of 16384 about 1200 TFLOP/s;
// 8 of 2048, 12 heads of 64: 104 us at 1965 MHz with no cap, 495 TFLOP/s (exponentials, one per 256 operations here:
// 50 %, tensor pipe 24 %); one of 77: 6.0 us, the length of one tile's chain from the first load to the last store.
#include <algorithm>
#include <type_traits>

#include "attn_tc.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {
namespace attn_tc {
namespace {

constexpr int kFwdThreads = 192;
// The softmax warps' barrier.
// Barriers and TMEM stand once all have come here; the loading warp only arrives.
__device__ __forceinline__ void started_arrive() { asm volatile("bar.arrive 2, 192;" ::: "memory"); }
__device__ __forceinline__ void started_sync() {
    tc_fence_before();
    asm volatile("bar.sync 2, 192;" ::: "memory");
    tc_fence_after();
}
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int HD>
struct FwdSmem {
    static constexpr uint32_t tile = kAtom * (HD / 64);
    static constexpr int slots = HD == 128 ? 2 : 5;          // K and V tiles in turn
    static constexpr uint32_t bytes = 1024 + tile * (1 + slots);
    static_assert(2 * (bytes + 2048) <= 233472, "two blocks per SM");
};

// o and lse of rows row0 .. row0 + count - 1 (one warp's, all below N), over the tokens each sees, row by row.
__device__ __noinline__ void fwd_rows_again(const AttnTcArgs& a, int head, int32_t row0, int count, int lane) {
    const int kv = head / a.group;
    const __nv_bfloat16* kp = a.k + (int64_t)kv * a.hd;
    const __nv_bfloat16* vp = a.v + (int64_t)kv * a.hd;
    const float cs = a.scale * kLog2e;
    for (int r = 0; r < count; ++r) {
        const int32_t n = row0 + r;
        const int32_t s0 = doc_of(n, a.seg, a.seqlen).x;
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
        const float inv = 1.f / l;
        put4(a.o + (int64_t)n * a.os + (int64_t)head * a.hd, lane, a.hd,
             make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
        if (a.lse != nullptr && lane == 0) a.lse[(int64_t)head * a.N + n] = (m + log2f(l)) * kLn2;
    }
}

template <int HD>
__global__ void __launch_bounds__(kFwdThreads, 2) attn_fwd_kernel(const __grid_constant__ CUtensorMap tq,
                                                                  const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv,
                                                                  const __grid_constant__ CUtensorMap to,
                                                                  const AttnTcArgs a) {
    using S = FwdSmem<HD>;
    constexpr bool kBeside = HD == 64;                       // P beside S
    constexpr uint32_t kP = kBeside ? 128 : 0, kO = kBeside ? 192 : 128;
    extern __shared__ uint8_t raw[];
    uint8_t* sQ = align1024(raw);
    uint8_t* ring = sQ + S::tile;                            // place 2 i: K of tile i, 2 i + 1: its V
    __shared__ uint64_t q_full, full[S::slots], empty[S::slots], s_full, s_free, p_ready, pv_done, drained;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, again;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.heads, kv = head / a.group;
    const int32_t tiles = (a.N + kRows - 1) / kRows;
    const int32_t row0 = tile_of((int32_t)(blockIdx.x / a.heads), tiles, a.seqlen % kRows ? 0 : a.seqlen / kRows, a.order_q,
                                 false) * kRows;
    const int32_t lo = doc_of(row0, a.seg, a.seqlen).x / kRows;
    const int32_t items = row0 / kRows - lo + 1;             // tiles of keys

    if (warp == 5) {
        if (lane == 0) {
            mbar_init(&q_full, 1);
            for (int s = 0; s < S::slots; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            mbar_init(&s_full, 1);
            mbar_init(&s_free, 4);
            mbar_init(&p_ready, 4);
            mbar_init(&pv_done, 1);
            mbar_init(&drained, 1);
            abort_flag = 0;
            again = 0;
            fence_mbar_init();
        }
        __syncwarp();
        started_arrive();                                    // the loads need no TMEM
        if (lane == 0) {
            mbar_arrive_expect_tx(&q_full, S::tile);
            load_head_tile<HD>(sQ, &tq, &q_full, head, row0);
            int n = 0;
            for (; n < 2 * items; ++n) {
                const int s = n % S::slots, use = n / S::slots;
                if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1, &abort_flag, a.err)) break;
                mbar_arrive_expect_tx(&full[s], S::tile);
                load_head_tile<HD>(ring + s * S::tile, n & 1 ? &tv : &tk, &full[s], kv, (lo + (n >> 1)) * kRows);
            }
            if (*(volatile int*)&abort_flag) {               // no copy may land after the CTA has gone
                mbar_wait_drain(&q_full, 0);
                for (int m = n > S::slots ? n - S::slots : 0; m < n; ++m)
                    mbar_wait_drain(&full[m % S::slots], (m / S::slots) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 4) {
        tmem_alloc(&tmem_base, 256);
        tmem_relinquish();
        started_sync();
        const uint32_t tb = tmem_base;
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdO = idesc_bf16(128, HD, false, true);
        const uint32_t q_at = smem_u32(sQ), r_at = smem_u32(ring);
        const bool lead = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = mbar_wait(bar, parity, &abort_flag, a.err);
            tc_fence_after();
            return got;
        };
        auto scores = [&](int n) {                           // of the keys at place n
            const int s = n % S::slots;
            if (!wait(&full[s], (n / S::slots) & 1)) return false;
            if (lead) {
#pragma unroll
                for (int c = 0; c < HD / 16; ++c)
                    umma_bf16(tb, kmajor_desc(q_at + (c / 4) * kAtom, c % 4),
                              kmajor_desc(r_at + s * S::tile + (c / 4) * kAtom, c % 4), kIdS, c != 0);
                umma_commit(&s_full);
                umma_commit(&empty[s]);
            }
            return true;
        };
        bool ok = wait(&q_full, 0) && scores(0);
        uint32_t phase = 0;
        for (int32_t i = 0; ok && i < items; ++i, phase ^= 1) {
            const int s = (2 * i + 1) % S::slots;
            if (kBeside && i + 1 < items) ok = wait(&s_free, phase) && scores(2 * i + 2);
            ok = ok && wait(&full[s], ((2 * i + 1) / S::slots) & 1) && wait(&p_ready, phase);
            if (ok && lead) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    umma_ts_bf16(tb + kO, tb + kP + 8 * c, mnmajor_desc(r_at + s * S::tile, kAtom, 16 * c), kIdO,
                                 i > 0 || c > 0);
                umma_commit(&pv_done);
                umma_commit(&empty[s]);
            }
            // P over S: these come behind the product that reads P
            if (!kBeside && ok && i + 1 < items) ok = scores(2 * i + 2);
            __syncwarp();
        }
        if (lead) umma_commit(&drained);                     // every MMA done before TMEM is freed
        mbar_wait_drain(&drained, 0);
    } else {
        // ---- softmax: one row per thread
        const int32_t n = row0 + warp * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        started_sync();
        const uint32_t tS = tmem_base + lanes, tP = tS + kP, tO = tS + kO;
        const float cs = a.scale * kLog2e;
        const int32_t full_from = doc_of(min(row0 + kRows, a.N) - 1, a.seg, a.seqlen).x;
        const int32_t start = n < a.N ? doc_of(n, a.seg, a.seqlen).x : INT32_MAX;
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;             // running maximum (log2 units), halves of the sum
        bool ok = true;
        uint32_t phase = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = mbar_wait(bar, parity, &abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            return ok;
        };
        auto signal = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto look = [&](int32_t i) {
            const int v = 2 * i + 1;
            if (!wait(&full[v % S::slots], (v / S::slots) & 1)) return false;
            constexpr uint32_t part = S::tile / 4;
            if (tile_nonfinite(ring + (v % S::slots) * S::tile + warp * part, part, lane) && lane == 0) again = 1;
            return true;
        };
        // One tile; two copies of the code, so that the tiles every row sees whole pay nothing for masks.
        auto tile = [&](auto with_mask, int32_t i) {
            constexpr bool kMask = decltype(with_mask)::value;
            const int32_t c0 = (lo + i) * kRows;
            const int from = start - c0, to_col = n - c0;
            if (!wait(&s_full, phase)) return false;
            // Maximum over columns 64-127, then 0-63; the latter stay in registers, the former are read again
            // below (a row of 128 scores next to its probabilities does not fit the registers).
            float s0[32], s1[32], mx[4];
            int see[4] = {kSeeAll, kSeeAll, kSeeAll, kSeeAll};
            if (kMask) {
#pragma unroll
                for (int b = 0; b < 4; ++b) see[b] = seen_run(32 * b, from, to_col);
            }
            auto mask = [&](float (&s)[32], int b) {
                if (!kMask) return;
                if (see[b] == kSeeSome) hide32(s, seen_bits(32 * b, from, to_col), -INFINITY);
                else if (see[b] == kSeeNone) fill32(s, -INFINITY);
            };
            tmem_ld32(tS + 64, s0);
            tmem_ld32(tS + 96, s1);
            tmem_wait_ld();
            mask(s0, 2);
            mask(s1, 3);
            mx[0] = max32(s0);
            mx[1] = max32(s1);
            tmem_ld32(tS, s0);
            tmem_ld32(tS + 32, s1);
            tmem_wait_ld();
            mask(s0, 0);
            mask(s1, 1);
            mx[2] = max32(s0);
            mx[3] = max32(s1);
            const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs);
            // The last product is done where P lies over S, since these scores came behind it
            if (kBeside && i > 0 && !wait(&pv_done, phase ^ 1)) return false;
            if (__any_sync(0xFFFFFFFFu, top - m > kGrow)) {
                if (i > 0) {
                    const float c = top == -INFINITY ? 1.f : ex2(m - top);
                    l0 *= c;
                    l1 *= c;
#pragma unroll 1
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
            auto probs = [&](float (&s)[32], int b) {
                if (kMask && see[b] == kSeeNone) zeros16(tP + 16 * b);
                else probs32(s, cs, neg, l0, l1, tP + 16 * b);
            };
            probs(s0, 0);
            tmem_ld32(tS + 64, s0);
            probs(s1, 1);
            tmem_ld32(tS + 96, s1);
            tmem_wait_ld();
            if (kBeside) signal(&s_free);
            mask(s0, 2);
            mask(s1, 3);
            probs(s0, 2);
            probs(s1, 3);
            tmem_wait_st();
            // Infinities and NaN among the values: before the product that gives the tile back waits for P, or
            // behind it where no tile follows.
            const bool final = i == items - 1;
            if (kMask && !final && !look(i)) return false;
            signal(&p_ready);
            return !(kMask && final) || look(i);
        };
        for (int32_t i = 0; i < items; ++i, phase ^= 1) {
            const bool masked = i == items - 1 || (lo + i) * kRows < full_from;
            if (!(masked ? tile(std::true_type{}, i) : tile(std::false_type{}, i))) break;
        }
        ok = ok && wait(&pv_done, (items - 1) & 1);
        ok = !named_bar_any<1, 128>(!ok);                    // every warp has looked; all go on, or none
        const float l = l0 + l1;
        const float inv = 1.f / l;                           // every row sees its own key; no finite score: 0 / 0
        if (ok && !again) {
            // O through Q's tile and TMA: rows from N on and channels from hd on are not written
#pragma unroll
            for (int b = 0; b < HD / 32; ++b) {
                float f[32];
                tmem_ld32(tO + 32 * b, f);
                tmem_wait_ld();
                tile_put32(sQ, warp * 32 + lane, b, f, inv);
            }
            fence_async_smem();
            softmax_sync();
            if (threadIdx.x == 0) {
                store_head_tile<HD>(&to, sQ, head, row0);
                tma_store_commit();
            }
            if (a.lse != nullptr && n < a.N) a.lse[(int64_t)head * a.N + n] = (m + __log2f(l)) * kLn2;
        } else if (ok) {
            const int32_t r = row0 + warp * 32;
            fwd_rows_again(a, head, r, min(32, a.N - r), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 256);
    }
    if (threadIdx.x == 0) tma_store_wait_read_all();          // O has left shared memory
}

template <int HD>
cudaError_t fwd_hd(const AttnProb& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& to, const AttnTcArgs& a, cudaStream_t st) {
    constexpr uint32_t smem = FwdSmem<HD>::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_fwd_kernel<HD>, smem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)((p.N + kRows - 1) / kRows * p.heads);
    DC_LAUNCH(kAttnTcFwd, st, attn_fwd_kernel<HD><<<grid, kFwdThreads, smem, st>>>(tq, tk, tv, to, a));
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
    CUtensorMap tq, tk, tv, to;
    if (!make_head_map(&tq, q, p.N, p.heads, p.hd, p.qs) || !make_head_map(&tk, k, p.N, p.kvh, p.hd, p.ks) ||
        !make_head_map(&tv, v, p.N, p.kvh, p.hd, p.vs) || !make_head_map(&to, o, p.N, p.heads, p.hd, p.os))
        return cudaErrorInvalidValue;
    AttnTcArgs a = tc_args(p);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.err = err;
    return p.hd <= 64 ? fwd_hd<64>(p, tq, tk, tv, to, a, st) : fwd_hd<128>(p, tq, tk, tv, to, a, st);
}

}  // namespace dynconv
