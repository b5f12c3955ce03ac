// attn_tc_bwd64.cu -- causal attention backward on the tensor cores for heads of up to 64 channels (bf16 storage).
//
// The mathematics, the two kernels and the roundings are those of attn_tc_bwd.cu.  With 64 channels the products
// take half the time and the element work (an exponential and some ten instructions per score) as long as before, so
// the chain of an item's steps and a block's prologue and epilogue (8 of 16 us at 2048 tokens) are what counts.  Two
// blocks therefore share an SM, each with half of TMEM and of shared memory, and one works while the other waits;
// items are 128 rows x 64 columns, so that S, dP and the gradients fit 256 columns:
//   dkv: S 64, dP 64, dV 64, dK 64; P lies over S, dS over dP, dS's remainder behind it
//   dq:  S 64, dP 64, dQ 64, dS two buffers of 32; dS's remainder over S
// Measured at 8 sequences of 2048, 12 heads: dkv 166 us (620 TFLOP/s; 204 us as one block per SM with items of 128 x 128), dq 122 (633; 160);
// an item takes 1.5 and 0.9 us of a block's time, what is outside the items about 8 us per block.  Both loads of scores
// and dP before the exponentials made dq 142; D from tiles by TMA, as the wide kernel does it, 123;
// blocks that walk their tiles, as wide dq's do, 157 (an item 1.06 us: the two blocks of an SM keep in step).  One fused
// kernel would take each exponential once and add 428 MB of dQ here, for which bulk tensor reductions alone take 78 to
// 82 us (5.2 to 5.5 TB/s): untried, its sums would change with the order of the blocks.
//
// Warps: 0-3 the element work (a lane is a row, all 64 columns) and the look for infinities and NaN in masked
// tiles; 4 issues the MMAs; 5 the TMA loads and (dkv) the items' lse and D.
#include <algorithm>
#include <type_traits>

#include "attn_tc_bwd.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {
namespace attn_tc {
namespace {

constexpr int kThreads64 = 192;
constexpr int kCols = 64;                        // tokens of an item's streamed tiles
constexpr uint32_t kHalfAtom = kCols * 128;      // bytes of such a tile

struct Smem64 {
    static constexpr int slots = 4;              // items in flight: two tiles each
    static constexpr uint32_t slot = 2 * kHalfAtom, ring = 2 * kAtom, stats = ring + slots * slot;
    static constexpr uint32_t bytes = 1024 + stats + slots * 2 * kCols * sizeof(float);
    static_assert(2 * (bytes + 2048) <= 233472, "two blocks per SM");
    static_assert(2 * kRows * part_ld<64>() * sizeof(float) <= stats, "partial gradients fit the tiles");
};

// Barriers and TMEM stand once all have come here; the loading warp only arrives.
__device__ __forceinline__ void started_arrive() { asm volatile("bar.arrive 2, 192;" ::: "memory"); }
__device__ __forceinline__ void started_sync() {
    tc_fence_before();
    asm volatile("bar.sync 2, 192;" ::: "memory");
    tc_fence_after();
}
__device__ __forceinline__ void element_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

struct Shared64 {
    uint64_t resident, full[Smem64::slots], empty[Smem64::slots];
    uint64_t s_full, s_free, dp_full, dp_free, p_ready, ds_ready[2], done;
    uint32_t tmem_base;
    int abort_flag, again;
};
// `loads`: arrivals that complete a slot (dkv: its statistics too); thread 0.
__device__ __forceinline__ void init64(Shared64& x, int loads) {
    mbar_init(&x.resident, 1);
    for (int s = 0; s < Smem64::slots; ++s) {
        mbar_init(&x.full[s], loads);
        mbar_init(&x.empty[s], 1);
    }
    mbar_init(&x.s_full, 1);
    mbar_init(&x.s_free, 4);
    mbar_init(&x.dp_full, 1);
    mbar_init(&x.dp_free, 4);
    mbar_init(&x.p_ready, 4);
    mbar_init(&x.ds_ready[0], 4);
    mbar_init(&x.ds_ready[1], 4);
    mbar_init(&x.done, 1);
    x.abort_flag = 0;
    x.again = 0;
    fence_mbar_init();
}

// D (64 columns at `to`) = A B^T: A 128 rows, B 64 rows of 64 channels, both K-major.
__device__ __forceinline__ void product_nt(uint32_t to, uint32_t A, uint32_t B) {
    constexpr uint32_t kId = idesc_bf16(128, kCols, false, false);
#pragma unroll
    for (int c = 0; c < 4; ++c) umma_bf16(to, kmajor_desc(A, c), kmajor_desc(B, c), kId, c != 0);
}
// D (64 columns at `to`) += the bf16 rows at `from` (32 columns of TMEM) X, X 64 rows of 64 channels.
__device__ __forceinline__ void product_ts(uint32_t to, uint32_t from, uint32_t X, bool add) {
    constexpr uint32_t kId = idesc_bf16(128, 64, false, true);
#pragma unroll
    for (int c = 0; c < 4; ++c) umma_ts_bf16(to, from + 8 * c, mnmajor_desc(X, kHalfAtom, 16 * c), kId, add || c > 0);
}

// ---------------------------------------------------------------- dk, dv
__global__ void __launch_bounds__(kThreads64, 2) attn_dkv64_kernel(const __grid_constant__ CUtensorMap tq,
                                                                   const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv,
                                                                   const __grid_constant__ CUtensorMap td,
                                                                   const __grid_constant__ CUtensorMap tdk,
                                                                   const __grid_constant__ CUtensorMap tdv,
                                                                   const AttnTcArgs a) {
    using S = Smem64;
    extern __shared__ uint8_t raw[];
    uint8_t* sK = align1024(raw);
    uint8_t* sV = sK + kAtom;
    uint8_t* ring = sK + S::ring;                            // slot: Q, then dO, of an item
    float* stats = reinterpret_cast<float*>(sK + S::stats);  // slot: -lse (log2 units), then D
    __shared__ Shared64 x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int kv = (int)(blockIdx.x / ranks) % a.kvh;
    const int32_t key0 = tile_of((int32_t)(blockIdx.x / ranks / a.kvh), (a.N + kRows - 1) / kRows,
                                 a.seqlen % kRows ? 0 : a.seqlen / kRows, a.order_k, true) * kRows;
    const int head0 = kv * a.group + rank * a.group / ranks;             // this block's heads
    const int heads = kv * a.group + (rank + 1) * a.group / ranks - head0;
    const int32_t full_to = doc_of(key0, a.seg, a.seqlen).y;             // queries below it see every key of the tile
    const int32_t e_last = doc_of(min(key0 + kRows, a.N) - 1, a.seg, a.seqlen).y;
    const int32_t t0 = key0 / kCols, per_head = (e_last - 1) / kCols - t0 + 1;
    const uint32_t items = (uint32_t)per_head * heads;
    constexpr uint32_t kDP = 64, kDV = 128, kDK = 192;

    if (warp == 5) {
        // loads by lane 0; the statistics of an item, read one item ahead, by the warp
        if (lane == 0) init64(x, 2);
        __syncwarp();
        started_arrive();                                    // the loads need no TMEM
        if (lane == 0) {
            mbar_arrive_expect_tx(&x.resident, 2 * kAtom);
            tma_load_3d(sK, &tk, &x.resident, 0, kv, key0);
            tma_load_3d(sV, &tv, &x.resident, 0, kv, key0);
        }
        int32_t g = 0, t = 0;
        float ls[2], dl[2];
        auto fetch = [&](int32_t h, int32_t tile) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int32_t n = (t0 + tile) * kCols + 2 * lane + e;
                const int64_t at = (int64_t)(head0 + h) * a.N + n;
                ls[e] = n < a.N ? -a.lse[at] * kLog2e : 0.f;
                dl[e] = n < a.N ? a.delta[at] : 0.f;
            }
        };
        fetch(0, 0);
        uint32_t n = 0;
        for (; n < items; ++n) {
            const int s = n % S::slots;
            const uint32_t use = n / S::slots;
            bool ok = true;
            if (use > 0) ok = mbar_wait(&x.empty[s], (use - 1) & 1, &x.abort_flag, a.err);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&x.full[s], S::slot);
                tma_load_3d(ring + s * S::slot, &tq, &x.full[s], 0, head0 + g, (t0 + t) * kCols);
                tma_load_3d(ring + s * S::slot + kHalfAtom, &td, &x.full[s], 0, head0 + g, (t0 + t) * kCols);
            }
            float* st = stats + s * 2 * kCols;
            *reinterpret_cast<float2*>(st + 2 * lane) = make_float2(ls[0], ls[1]);
            *reinterpret_cast<float2*>(st + kCols + 2 * lane) = make_float2(dl[0], dl[1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.full[s]);
            if (++t == per_head) { t = 0; ++g; }
            if (n + 1 < items) fetch(g, t);
        }
        if (lane == 0 && *(volatile int*)&x.abort_flag) {    // no copy may land after the block has gone
            mbar_wait_drain(&x.resident, 0);
            for (uint32_t m = n > S::slots ? n - S::slots : 0; m < n; ++m)
                mbar_wait_drain(&x.full[m % S::slots], (m / S::slots) & 1);
        }
        __syncwarp();
    } else if (warp == 4) {
        tmem_alloc(&x.tmem_base, 256);
        tmem_relinquish();
        started_sync();
        const uint32_t tb = x.tmem_base;
        const uint32_t k_at = smem_u32(sK), v_at = smem_u32(sV), r_at = smem_u32(ring);
        const bool lead = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = mbar_wait(bar, parity, &x.abort_flag, a.err);
            tc_fence_after();
            return got;
        };
        bool ok = wait(&x.resident, 0) && wait(&x.full[0], 0);
        if (ok && lead) {
            product_nt(tb, k_at, r_at);
            umma_commit(&x.s_full);
            product_nt(tb + kDP, v_at, r_at + kHalfAtom);
            umma_commit(&x.dp_full);
        }
        uint32_t phase = 0;
        int32_t t = 0;
        for (uint32_t i = 0; ok && i < items; ++i, phase ^= 1) {
            const uint32_t at = r_at + i % S::slots * S::slot, ns = (i + 1) % S::slots, next = r_at + ns * S::slot;
            const bool more = i + 1 < items;
            ok = wait(&x.p_ready, phase);
            if (ok && lead) product_ts(tb + kDV, tb, at + kHalfAtom, i > 0);
            if (more) {
                ok = ok && wait(&x.full[ns], ((i + 1) / S::slots) & 1);
                if (ok && lead) {
                    product_nt(tb, k_at, next);
                    umma_commit(&x.s_full);
                }
            }
            ok = ok && wait(&x.ds_ready[0], phase);
            if (ok && lead) {
                product_ts(tb + kDK, tb + kDP, at, i > 0);
                if (t < 2) product_ts(tb + kDK, tb + kDP + 32, at, true);        // the diagonal tiles' remainders
                umma_commit(&x.empty[i % S::slots]);
                if (more) {
                    product_nt(tb + kDP, v_at, next + kHalfAtom);
                    umma_commit(&x.dp_full);
                }
            }
            if (++t == per_head) t = 0;
            __syncwarp();
        }
        if (lead) umma_commit(&x.done);                      // every MMA done
        mbar_wait_drain(&x.done, 0);
    } else {
        const int32_t j = key0 + warp * 32 + lane;
        const int32_t end = j < a.N ? doc_of(j, a.seg, a.seqlen).y : 0;
        started_sync();
        const uint32_t at = x.tmem_base + ((uint32_t)(warp * 32) << 16);
        const float cs = a.scale * kLog2e;
        bool ok = true;
        uint32_t phase = 0;
        int32_t t = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = mbar_wait(bar, parity, &x.abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            return ok;
        };
        auto signal = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // One item; two copies of the code, so that the tiles every key is seen by whole pay nothing for masks.
        auto item = [&](auto with_mask, uint32_t i) {
            constexpr bool kMask = decltype(with_mask)::value;
            const int32_t q0 = (t0 + t) * kCols;
            const int from = j - q0, to = end - 1 - q0, slot = i % S::slots;
            const float* st = stats + slot * 2 * kCols;
            int see[2] = {kSeeAll, kSeeAll};
            uint32_t bits[2] = {~0u, ~0u};
            if (kMask) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    see[b] = seen_run(32 * b, from, to);
                    bits[b] = seen_bits(32 * b, from, to);
                }
            }
            float p[2][32], f[2][32];
            if (!wait(&x.full[slot], (i / S::slots) & 1) || !wait(&x.s_full, phase)) return false;
            tmem_ld32(at, p[0]);
            tmem_ld32(at + 32, p[1]);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (kMask && see[b] == kSeeNone) {
                    fill32(p[b], 0.f);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 l = *reinterpret_cast<const float4*>(st + 32 * b + e);
                        fma2v(p[b][e], p[b][e + 1], cs, l.x, l.y);
                        fma2v(p[b][e + 2], p[b][e + 3], cs, l.z, l.w);
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) p[b][e] = ex2(p[b][e]);
                    if (kMask && see[b] == kSeeSome) hide32(p[b], bits[b], 0.f);
                }
                store32(at + 16 * b, p[b]);
            }
            tmem_wait_st();
            signal(&x.p_ready);
            if (!wait(&x.dp_full, phase)) return false;
            tmem_ld32(at + kDP, f[0]);
            tmem_ld32(at + kDP + 32, f[1]);
            tmem_wait_ld();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (kMask && see[b] == kSeeNone) {
                    fill32(f[b], 0.f);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 d = *reinterpret_cast<const float4*>(st + kCols + 32 * b + e);
                        add2(f[b][e], f[b][e + 1], -d.x, -d.y);
                        add2(f[b][e + 2], f[b][e + 3], -d.z, -d.w);
                        mul2v(f[b][e], f[b][e + 1], p[b][e], p[b][e + 1]);
                        mul2v(f[b][e + 2], f[b][e + 3], p[b][e + 2], p[b][e + 3]);
                    }
                    if (kMask && see[b] == kSeeSome) hide32(f[b], bits[b], 0.f);
                }
                store32(at + kDP + 16 * b, f[b]);
                if (kMask && t < 2) {
                    remainder32(f[b]);
                    store32(at + kDP + 32 + 16 * b, f[b]);
                }
            }
            tmem_wait_st();
            // infinities and NaN among Q and dO, before the product that gives the slot back waits for dS
            if (kMask && tile_nonfinite(ring + slot * S::slot + warp * (S::slot / 4), S::slot / 4, lane) && lane == 0)
                x.again = 1;
            signal(&x.ds_ready[0]);
            return true;
        };
        for (uint32_t i = 0; i < items; ++i, phase ^= 1) {
            const bool masked = t < 2 || (t0 + t + 1) * kCols > full_to;
            if (!(masked ? item(std::true_type{}, i) : item(std::false_type{}, i))) break;
            if (++t == per_head) t = 0;
        }
        ok = ok && wait(&x.done, 0);
        ok = !named_bar_any<1, 128>(!ok);                    // every warp has looked; all go on, or none
        if (!ok) x.again = -1;                               // nothing is written then
        const bool write = ok && !x.again;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {                        // dv, dk
            float* row = reinterpret_cast<float*>(sK) + (size_t)(w * kRows + warp * 32 + lane) * part_ld<64>();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float f[32];
                tmem_ld32(at + (w ? kDK : kDV) + 32 * b, f);
                tmem_wait_ld();
                if (ranks > 1) {
                    // this block's part, for the cluster
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(row + 32 * b + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
                } else if (write) {
                    tile_put32(w ? sK : sV, warp * 32 + lane, b, f, w ? a.scale : 1.f);
                }
            }
        }
        if (ranks == 1 && write) {
            fence_async_smem();
            element_sync();
            if (threadIdx.x == 0) {
                store_head_tile<64>(&tdv, sV, kv, key0);
                store_head_tile<64>(&tdk, sK, kv, key0);
                tma_store_commit();
            }
        } else if (ranks == 1 && ok) {
            const int32_t r = key0 + warp * 32;
            dkv_rows_again(a, kv, r, min(32, a.N - r), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(x.tmem_base, 256);
    }
    if (ranks == 1) {
        if (threadIdx.x == 0) tma_store_wait_read_all();      // the gradients have left shared memory
        return;
    }
    join_parts<64, kThreads64, 4>(a, cluster, &x.again, reinterpret_cast<const float*>(sK), kv, key0);
}

// ---------------------------------------------------------------- dq
__global__ void __launch_bounds__(kThreads64, 2) attn_dq64_kernel(const __grid_constant__ CUtensorMap tq,
                                                                  const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv,
                                                                  const __grid_constant__ CUtensorMap td,
                                                                  const __grid_constant__ CUtensorMap tdq,
                                                                  const AttnTcArgs a) {
    using S = Smem64;
    extern __shared__ uint8_t raw[];
    uint8_t* sQ = align1024(raw);
    uint8_t* sO = sQ + kAtom;
    uint8_t* ring = sQ + S::ring;                            // slot: K, then V, of an item
    float* sD = reinterpret_cast<float*>(sQ + S::stats);
    __shared__ Shared64 x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.heads, kv = head / a.group;
    const int32_t tiles = (a.N + kRows - 1) / kRows;
    const int32_t row0 = tile_of((int32_t)(blockIdx.x / a.heads), tiles, a.seqlen % kRows ? 0 : a.seqlen / kRows, a.order_q,
                                 false) * kRows;
    const int32_t last = min(row0 + kRows, a.N) - 1;
    const int32_t lo = doc_of(row0, a.seg, a.seqlen).x / kCols;
    const int32_t full_from = doc_of(last, a.seg, a.seqlen).x;
    const int32_t items = last / kCols - lo + 1, plain = row0 / kCols - lo;      // items before the diagonal's
    constexpr uint32_t kDP = 64, kDQ = 128, kDS = 192;

    if (warp == 5) {
        if (lane == 0) init64(x, 1);
        __syncwarp();
        started_arrive();                                    // the loads need no TMEM
        if (lane == 0) {
            mbar_arrive_expect_tx(&x.resident, 2 * kAtom);
            tma_load_3d(sQ, &tq, &x.resident, 0, head, row0);
            tma_load_3d(sO, &td, &x.resident, 0, head, row0);
            int32_t n = 0;
            for (; n < items; ++n) {
                const int s = n % S::slots, use = n / S::slots;
                if (use > 0 && !mbar_wait(&x.empty[s], (use - 1) & 1, &x.abort_flag, a.err)) break;
                mbar_arrive_expect_tx(&x.full[s], S::slot);
                tma_load_3d(ring + s * S::slot, &tk, &x.full[s], 0, kv, (lo + n) * kCols);
                tma_load_3d(ring + s * S::slot + kHalfAtom, &tv, &x.full[s], 0, kv, (lo + n) * kCols);
            }
            if (*(volatile int*)&x.abort_flag) {             // no copy may land after the block has gone
                mbar_wait_drain(&x.resident, 0);
                for (int32_t m = n > S::slots ? n - S::slots : 0; m < n; ++m)
                    mbar_wait_drain(&x.full[m % S::slots], (m / S::slots) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 4) {
        tmem_alloc(&x.tmem_base, 256);
        tmem_relinquish();
        started_sync();
        const uint32_t tb = x.tmem_base;
        const uint32_t q_at = smem_u32(sQ), o_at = smem_u32(sO), r_at = smem_u32(ring);
        const bool lead = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = mbar_wait(bar, parity, &x.abort_flag, a.err);
            tc_fence_after();
            return got;
        };
        bool ok = wait(&x.resident, 0) && wait(&x.full[0], 0);
        auto scores = [&](uint32_t at) {
            if (lead) {
                product_nt(tb, q_at, at);
                umma_commit(&x.s_full);
            }
        };
        auto products = [&](uint32_t at) {
            if (lead) {
                product_nt(tb + kDP, o_at, at + kHalfAtom);
                umma_commit(&x.dp_full);
            }
        };
        if (ok) {
            scores(r_at);
            products(r_at);
        }
        for (int32_t i = 0; ok && i < items; ++i) {
            const uint32_t at = r_at + i % S::slots * S::slot, ns = (i + 1) % S::slots, next = r_at + ns * S::slot;
            const bool more = i + 1 < items, early = i < plain;      // a diagonal item's remainders lie over S
            if (more) {
                ok = wait(&x.full[ns], ((i + 1) / S::slots) & 1) && wait(&x.s_free, i & 1);
                if (ok && early) scores(next);
                ok = ok && wait(&x.dp_free, i & 1);
                if (ok) products(next);
            }
            ok = ok && wait(&x.ds_ready[i & 1], (i >> 1) & 1);
            if (ok) {
                if (lead) {
                    product_ts(tb + kDQ, tb + kDS + 32 * (i & 1), at, i > 0);
                    if (!early) product_ts(tb + kDQ, tb, at, true);
                    umma_commit(&x.empty[i % S::slots]);
                }
                if (more && !early) scores(next);
            }
            __syncwarp();
        }
        if (lead) umma_commit(&x.done);
        mbar_wait_drain(&x.done, 0);
    } else {
        const int row = warp * 32 + lane;
        const int32_t n = row0 + row;
        const float cs = a.scale * kLog2e;
        {
            // D = dO . O: eight lanes per row, all loads in flight together
            uint4 u[8], v[8];
            const int c = 8 * (lane & 7);
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int64_t m = row0 + 32 * warp + 4 * it + (lane >> 3);
                const bool real = m < a.N && c < a.hd;
                u[it] = v[it] = make_uint4(0, 0, 0, 0);
                if (real) {
                    u[it] = __ldg(reinterpret_cast<const uint4*>(a.o + m * a.os + (int64_t)head * a.hd + c));
                    v[it] = __ldg(reinterpret_cast<const uint4*>(a.d_o + m * a.dos + (int64_t)head * a.hd + c));
                }
            }
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                float d = bf16_lo(u[it].x) * bf16_lo(v[it].x);
                d = fmaf(bf16_hi(u[it].x), bf16_hi(v[it].x), d);
                d = fmaf(bf16_lo(u[it].y), bf16_lo(v[it].y), d);
                d = fmaf(bf16_hi(u[it].y), bf16_hi(v[it].y), d);
                d = fmaf(bf16_lo(u[it].z), bf16_lo(v[it].z), d);
                d = fmaf(bf16_hi(u[it].z), bf16_hi(v[it].z), d);
                d = fmaf(bf16_lo(u[it].w), bf16_lo(v[it].w), d);
                d = fmaf(bf16_hi(u[it].w), bf16_hi(v[it].w), d);
#pragma unroll
                for (int o = 4; o; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
                if ((lane & 7) == 0) sD[32 * warp + 4 * it + (lane >> 3)] = d;
            }
            __syncwarp();
        }
        const int32_t start = n < a.N ? doc_of(n, a.seg, a.seqlen).x : INT32_MAX;
        const float ls = n < a.N ? -a.lse[(int64_t)head * a.N + n] * kLog2e : 0.f;
        float dl = -sD[row];
        started_sync();
        const uint32_t at = x.tmem_base + ((uint32_t)(warp * 32) << 16), ds_at = at + kDS;
        bool ok = true;
        uint32_t phase = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = mbar_wait(bar, parity, &x.abort_flag, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            return ok;
        };
        auto signal = [&](uint64_t* bar) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto item = [&](auto with_mask, int32_t i) {
            constexpr bool kMask = decltype(with_mask)::value;
            const int32_t c0 = (lo + i) * kCols;
            const int from = start - c0, to = n - c0;
            int see[2] = {kSeeAll, kSeeAll};
            uint32_t bits[2] = {~0u, ~0u};
            if (kMask) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    see[b] = seen_run(32 * b, from, to);
                    bits[b] = seen_bits(32 * b, from, to);
                }
            }
            float p[2][32], f[2][32];
            if (!wait(&x.s_full, phase)) return false;
            tmem_ld32(at, p[0]);
            tmem_ld32(at + 32, p[1]);
            tmem_wait_ld();
            signal(&x.s_free);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (kMask && see[b] == kSeeNone) {
                    fill32(p[b], 0.f);
                    continue;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    fma2(p[b][e], p[b][e + 1], cs, ls);
                    p[b][e] = ex2(p[b][e]);
                    p[b][e + 1] = ex2(p[b][e + 1]);
                }
                if (kMask && see[b] == kSeeSome) hide32(p[b], bits[b], 0.f);
            }
            if (!wait(&x.dp_full, phase)) return false;
            tmem_ld32(at + kDP, f[0]);
            tmem_ld32(at + kDP + 32, f[1]);
            tmem_wait_ld();
            signal(&x.dp_free);
            if (kMask) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    if (see[b] == kSeeSome) hide32(f[b], bits[b], 0.f);
                    else if (see[b] == kSeeNone) fill32(f[b], 0.f);
                }
                // D of a row that sees no other item
                float y = 0.f, z = 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    y = fmaf(p[0][e], f[0][e], y);
                    z = fmaf(p[1][e], f[1][e], z);
                }
                if (start >= c0 && n < c0 + kCols) dl = -(y + z);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (!(kMask && see[b] == kSeeNone)) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        add2(f[b][e], f[b][e + 1], dl, dl);
                        mul2v(f[b][e], f[b][e + 1], p[b][e], p[b][e + 1]);
                    }
                }
                store32(ds_at + 32 * (i & 1) + 16 * b, f[b]);
                if (kMask && i >= plain) {
                    remainder32(f[b]);
                    store32(at + 16 * b, f[b]);
                }
            }
            tmem_wait_st();
            if (kMask) {
                // infinities and NaN among the keys, before the product that gives the slot back waits for dS
                const int slot = i % S::slots;
                if (!wait(&x.full[slot], (i / S::slots) & 1)) return false;
                if (tile_nonfinite(ring + slot * S::slot + warp * (kHalfAtom / 4), kHalfAtom / 4, lane) && lane == 0) x.again = 1;
            }
            signal(&x.ds_ready[i & 1]);
            return true;
        };
        for (int32_t i = 0; i < items; ++i, phase ^= 1) {
            const bool masked = i >= plain || (lo + i) * kCols < full_from;
            if (!(masked ? item(std::true_type{}, i) : item(std::false_type{}, i))) break;
        }
        if (n < a.N) a.delta[(int64_t)head * a.N + n] = -dl;
        ok = ok && wait(&x.done, 0);
        ok = !named_bar_any<1, 128>(!ok);                    // every warp has looked; all go on, or none
        if (ok && !x.again) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float f[32];
                tmem_ld32(at + kDQ + 32 * b, f);
                tmem_wait_ld();
                tile_put32(sQ, row, b, f, a.scale);
            }
            fence_async_smem();
            element_sync();
            if (threadIdx.x == 0) {
                store_head_tile<64>(&tdq, sQ, head, row0);
                tma_store_commit();
            }
        } else if (ok) {
            const int32_t r = row0 + warp * 32;
            dq_rows_again(a, head, r, min(32, a.N - r), lane);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(x.tmem_base, 256);
    }
    if (threadIdx.x == 0) tma_store_wait_read_all();          // dq has left shared memory
}

}  // namespace

cudaError_t bwd_narrow(const AttnProb& p, const BwdMaps& m, const AttnTcArgs& a, cudaStream_t st) {
    constexpr uint32_t smem = Smem64::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_dkv64_kernel, smem);
    if (e == cudaSuccess) e = DC_SMEM_LIMIT(attn_dq64_kernel, smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + kRows - 1) / kRows;
    DC_LAUNCH(kAttnTcDq, st, attn_dq64_kernel<<<(unsigned)(tiles * p.heads), kThreads64, smem, st>>>(m.q, m.k64, m.v64, m.d,
                                                                                                    m.dq, a));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int ranks = dkv_ranks(p, tiles * p.kvh);
    DC_LAUNCH(kAttnTcDkv, st, e = launch_ranks(attn_dkv64_kernel, ranks, (unsigned)(tiles * p.kvh * ranks), kThreads64, smem,
                                               st, m.q64, m.k, m.v, m.d64, m.dk, m.dv, a));
    return e;
}

}  // namespace attn_tc
}  // namespace dynconv
