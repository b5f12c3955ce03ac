// attn_tc_bwd.cu -- causal attention backward on the tensor cores (bf16 storage), heads of 72 to 128 channels (narrow
// ones: attn_tc_bwd64.cu).
//
//   P = exp(scale S - lse),  dP = dO V^T,  dS = P (dP - D)
//   dV = P^T dO,  dK = scale dS^T Q   (over every query of the document, every head of the group)
//   dQ = scale dS K                   (over every key the query sees)
//
// Two kernels, each with its sums in TMEM for its whole run and written once: attn_dkv_kernel takes 128
// keys of one key/value head and walks the query tiles of every head of the group; attn_dq_kernel takes 128
// queries of one head and walks the key tiles.  S and dP are computed in both (7 products of a tile pair
// where one fused kernel needs 5), because the fused kernel would add a 128 x 128 fp32 tile of dQ into global
// memory for every tile pair, in an order that changes from run to run.  Here nothing is added atomically and results
// repeat bitwise.  What that costs is open: bulk tensor reductions alone run at 4.6 (a block per SM) to 5.1 TB/s (two)
// for the 1141 MB that 8 sequences of 2048, 16 heads of 128 would add (224 to 248 us, as long as either kernel takes).
//
// No operand passes through shared memory by hand: the transposed scores S^T = K Q^T put keys on the TMEM
// lanes, P^T and dS^T are written back to TMEM as bf16 and are the A operands of dV and dK; in attn_dq_kernel
// dS is the A operand of dQ.  P and dS are rounded to bf16 because the tensor cores take them so; dS is
// computed from the fp32 P.  In the diagonal tile, where the rows of few keys are whose gradients are the
// largest, dS goes in as two bf16 (value and remainder).
//
// attn_dq_kernel runs first and leaves D for the other.  D = dO . O takes the O that the forward rounded; for
// rows that see no key outside the diagonal tile it is taken as sum_j P dP instead, which is the same without
// that rounding (dP - D cancels most where a row sees few keys).
//
// attn_dq_kernel is a block per SM that walks its share of the (head, tile) pairs, because a block that came for
// one pair spent 8 us outside its items (launch, barriers and TMEM, the first loads, the last store) and ~1.4 us on
// each: now Q of the next pair is loaded once this one's last scores are done, its first scores follow at once,
// and dO, through whose tile dQ is stored, comes while they are read (16384 tokens, 16 heads of 128: 272 -> 249 us in
// sequences of 2048, 193 -> 175 in sequences of 1024; writing dQ from the registers, so that dO could come earlier,
// too: 262 and 185).
//
// With few key tiles and large groups the heads of a group are shared out over a cluster of blocks, whose partial
// dK and dV are added through distributed shared memory in the order of their ranks.
//
// Warps: 0-7 the element work (a lane is a row; warps 0-3 take columns 0-63, 4-7 columns 64-127, each
// writing its bf16 results over columns that it alone has read), 8 MMA issue, 9 TMA, 10 infinities and NaN in
// masked tiles (see attn_tc_fwd.cu), 11 (dkv) the rows' lse and D, (dq) the store of dQ.
//
// What bounds them is the chain from one item (tile pair) to the next, so every wait on it is moved off:
// the next scores are computed into S as soon as the element warps hold this item's in registers, the
// exponentials run before the wait for dP, and the two halves of an item have ring places of their own,
// given back as soon as their last product is done (both loads of an item together, released together, left the
// tensor cores waiting for L2: 4250 cycles per item instead of ~2500).
//   dkv: S(i+1) | dV(i) | dK(i) dP(i+1)    P and dS lie in the columns of dP, read into registers before
//   dq:  S(i+1) | dP(i+1) | dQ(i)          dS has two buffers of its own
// Measured at 16384 tokens, 16 heads of 128 over 4, in sequences of 2048: dkv 260 us (1057 TFLOP/s of its four products,
// 1.8 us per item), dq 249 (828 of its three, 1.4 us per item); 9 documents of 346 to 2716 tokens: 199 and 157.
#include <algorithm>
#include <type_traits>

#include "attn_tc_bwd.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {
namespace attn_tc {
namespace {

constexpr int HD = 128;                          // channels that fit; narrower heads are padded by zeros
constexpr int kBwdThreads = 384;
// Barriers and TMEM stand once all have come here; the loading warp only arrives.
__device__ __forceinline__ void started_arrive() { asm volatile("bar.arrive 2, 384;" ::: "memory"); }
__device__ __forceinline__ void started_sync() {
    tc_fence_before();
    asm volatile("bar.sync 2, 384;" ::: "memory");
    tc_fence_after();
}
// The element warps' barrier (256 threads).
__device__ __forceinline__ void element_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Shared memory: two resident tiles, a ring of tiles, the statistics of two items, the barriers.  No slack for
// alignment: the dynamic part starts on a 1024-byte boundary, since these kernels have no static part (checked).
struct BwdSmem {
    static constexpr uint32_t tile = kAtom * (HD / 64);
    static constexpr int slots = 5;
    static constexpr uint32_t ring = 2 * tile, stats = ring + slots * tile, shared = stats + 2 * 2 * kRows * sizeof(float);
    // a block's partial dV and dK for its cluster, in the memory of the tiles
    static_assert(2 * kRows * part_ld<HD>() * sizeof(float) <= stats, "partial gradients fit the tiles");
    struct Shared {
        uint64_t resident, full[slots], empty[slots], stat_full[2], stat_free[2];
        uint64_t s_full, s_free, dp_full, dp_free, p_ready, ds_ready[2], d_done, done, scanned;
        uint64_t q_free, o_full, o_free, staged, drained;             // dq
        uint32_t tmem_base;
        int abort_flag, again;
    };
    static constexpr uint32_t bytes = shared + sizeof(Shared);
    static_assert(bytes <= 232448, "fits an SM");
};
// The tiles' swizzle needs 1024-byte alignment: true for the whole grid alike, and reported, where it does not hold.
__device__ __forceinline__ bool misplaced(const void* sm, uint32_t* err) {
    if ((smem_u32(sm) & 1023u) == 0) return false;
    if (threadIdx.x == 0) atomicOr(err, kErrWaitTimeout);
    return true;
}
// Barriers of either kernel; one thread.
__device__ __forceinline__ void bwd_init(BwdSmem::Shared& x) {
    mbar_init(&x.resident, 1);
    for (int s = 0; s < BwdSmem::slots; ++s) {
        mbar_init(&x.full[s], 1);
        mbar_init(&x.empty[s], 2);                           // the last product, the look for infinities
    }
    for (int s = 0; s < 2; ++s) {
        mbar_init(&x.stat_full[s], 1);
        mbar_init(&x.stat_free[s], 8);
    }
    mbar_init(&x.s_full, 1);
    mbar_init(&x.s_free, 8);
    mbar_init(&x.dp_full, 1);
    mbar_init(&x.dp_free, 8);
    mbar_init(&x.p_ready, 8);
    mbar_init(&x.ds_ready[0], 8);
    mbar_init(&x.ds_ready[1], 8);
    mbar_init(&x.d_done, 8);
    mbar_init(&x.done, 1);
    mbar_init(&x.scanned, 1);
    mbar_init(&x.q_free, 1);
    mbar_init(&x.o_full, 1);
    mbar_init(&x.o_free, 1);
    mbar_init(&x.staged, 8);
    mbar_init(&x.drained, 1);
    x.abort_flag = 0;
    x.again = 0;
    fence_mbar_init();
}
// Place n of the ring: its slot, and the parity of its use of that slot.
struct Spot {
    int slot;
    uint32_t parity;
    __device__ __forceinline__ explicit Spot(uint32_t n)
        : slot((int)(n % BwdSmem::slots)), parity((n / BwdSmem::slots) & 1) {}
};
// TMA of the ring's places 0 .. count - 1 by one thread: load(place, destination, barrier).  After an abort no
// copy may land once the block has gone.
template <typename Load>
__device__ __forceinline__ void feed_ring(uint8_t* ring, BwdSmem::Shared& x, uint32_t count, uint32_t* err,
                                          Load load) {
    using S = BwdSmem;
    uint32_t n = 0;
    for (; n < count; ++n) {
        const Spot at(n);
        if (n >= S::slots && !mbar_wait(&x.empty[at.slot], at.parity ^ 1, &x.abort_flag, err)) break;
        mbar_arrive_expect_tx(&x.full[at.slot], S::tile);
        load(n, ring + at.slot * S::tile, &x.full[at.slot]);
    }
    if (*(volatile int*)&x.abort_flag) {
        mbar_wait_drain(&x.resident, 0);
        for (uint32_t m = n > S::slots ? n - S::slots : 0; m < n; ++m) {
            const Spot at(m);
            mbar_wait_drain(&x.full[at.slot], at.parity);
        }
    }
}

// ---------------------------------------------------------------- dk, dv
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dkv_kernel(const __grid_constant__ CUtensorMap tq,
                                                                  const __grid_constant__ CUtensorMap tk,
                                                                  const __grid_constant__ CUtensorMap tv,
                                                                  const __grid_constant__ CUtensorMap td,
                                                                  const __grid_constant__ CUtensorMap tdk,
                                                                  const __grid_constant__ CUtensorMap tdv,
                                                                  const AttnTcArgs a) {
    using S = BwdSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* sK = sm;
    uint8_t* sV = sm + S::tile;
    uint8_t* ring = sm + S::ring;                            // place 2 i: Q of item i, 2 i + 1: its dO
    float* stats = reinterpret_cast<float*>(sm + S::stats);
    S::Shared& x = *reinterpret_cast<S::Shared*>(sm + S::shared);
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
    const int32_t t0 = key0 / kRows, per_head = (e_last - 1) / kRows - t0 + 1;
    const uint32_t items = (uint32_t)per_head * heads;
    if (misplaced(sm, a.err)) return;
    constexpr uint32_t kDP = 128, kDV = 256, kDK = 256 + HD;

    if (warp == 9) {
        if (lane == 0) bwd_init(x);
        __syncwarp();
        started_arrive();                                    // the loads need no TMEM
        if (lane == 0) {
            mbar_arrive_expect_tx(&x.resident, 2 * S::tile);
            load_head_tile<HD>(sK, &tk, &x.resident, kv, key0);
            load_head_tile<HD>(sV, &tv, &x.resident, kv, key0);
            int32_t g = 0, t = 0;
            feed_ring(ring, x, 2 * items, a.err, [&](uint32_t n, uint8_t* to, uint64_t* bar) {
                load_head_tile<HD>(to, n & 1 ? &td : &tq, bar, head0 + g, (t0 + t) * kRows);
                if ((n & 1) && ++t == per_head) { t = 0; ++g; }
            });
        }
        __syncwarp();
    } else if (warp == 8) {
        tmem_alloc(&x.tmem_base, 512);
        tmem_relinquish();
        started_sync();
        const uint32_t tb = x.tmem_base;
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdG = idesc_bf16(128, HD, false, true);
        const uint32_t k_at = smem_u32(sK), v_at = smem_u32(sV), r_at = smem_u32(ring);
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
        // D (128 columns at `to`) += the bf16 rows at `from` (columns 0-63 and 64-127 of the tile 64 columns apart) X
        auto grad = [&](uint32_t to, uint32_t from, uint32_t X, bool add) {
            if (lead) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    umma_ts_bf16(tb + to, tb + from + (c < 4 ? 8 * c : 64 + 8 * (c - 4)), mnmajor_desc(X, kAtom, 16 * c),
                                 kIdG, add || c > 0);
            }
        };
        // A wait that finds its barrier complete still takes some 100 cycles, in which the tensor cores run dry: the
        // two loads of the next item are asked after together, and tiles that TMA brought need no tcgen05 fence.
        auto landed = [&](const Spot& p, const Spot& q) {
            const bool u = mbar_try_wait(&x.full[p.slot], p.parity), v = mbar_try_wait(&x.full[q.slot], q.parity);
            return (u && v) || (mbar_wait(&x.full[p.slot], p.parity, &x.abort_flag, a.err) &&
                                mbar_wait(&x.full[q.slot], q.parity, &x.abort_flag, a.err));
        };
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = mbar_wait(bar, parity, &x.abort_flag, a.err);
            tc_fence_after();
            return got;
        };
        bool ok = wait(&x.resident, 0) && wait(&x.full[0], 0);
        if (ok) nt(0, k_at, r_at, &x.s_full);
        ok = ok && wait(&x.full[1], 0);
        if (ok) nt(kDP, v_at, r_at + S::tile, &x.dp_full);
        uint32_t phase = 0;
        int32_t t = 0;
        for (uint32_t i = 0; ok && i < items; ++i, phase ^= 1) {
            const Spot q(2 * i), d(2 * i + 1), q1(2 * i + 2), d1(2 * i + 3);
            const bool more = i + 1 < items;
            auto next_scores = [&]() {
                ok = ok && landed(q1, d1) && wait(&x.s_free, phase);
                if (ok) nt(0, k_at, r_at + q1.slot * S::tile, &x.s_full);
            };
            if (more && t > 0) next_scores();
            ok = ok && wait(&x.p_ready, phase);
            if (ok) {
                grad(kDV, kDP, r_at + d.slot * S::tile, i > 0);
                if (lead) umma_commit(&x.empty[d.slot]);
            }
            ok = ok && wait(&x.ds_ready[0], phase);
            if (ok) {
                grad(kDK, kDP + 32, r_at + q.slot * S::tile, i > 0);
                // the diagonal tile's remainders lie in the columns of S: the next scores come after them
                if (t == 0) grad(kDK, 0, r_at + q.slot * S::tile, true);
                if (lead) umma_commit(&x.empty[q.slot]);
            }
            if (more && t == 0) next_scores();
            if (more && ok) nt(kDP, v_at, r_at + d1.slot * S::tile, &x.dp_full);
            if (++t == per_head) t = 0;
            __syncwarp();
        }
        if (lead) umma_commit(&x.done);                      // every MMA done
        mbar_wait_drain(&x.done, 0);
    } else if (warp == 10) {
        started_sync();
        bool ok = true;
        int32_t t = 0;
        for (uint32_t n = 0; ok && n < 2 * items; ++n) {
            const Spot at(n);
            ok = mbar_wait(&x.full[at.slot], at.parity, &x.abort_flag, a.err);
            if (!ok) break;
            if ((t == 0 || (t0 + t + 1) * kRows > full_to) && tile_nonfinite(ring + at.slot * S::tile, S::tile, lane) &&
                lane == 0)
                x.again = 1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.empty[at.slot]);
            if ((n & 1) && ++t == per_head) t = 0;
        }
        if (lane == 0) mbar_arrive(&x.scanned);
    } else if (warp == 11) {
        // lse (log2 units, negated) and D of each item's queries: read ahead, four per lane
        int32_t g = 0, t = 0;
        float ls[4], dl[4];
        auto fetch = [&]() {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int32_t n = (t0 + t) * kRows + 4 * lane + e;
                const int64_t at = (int64_t)(head0 + g) * a.N + n;
                ls[e] = n < a.N ? -a.lse[at] * kLog2e : 0.f;
                dl[e] = n < a.N ? a.delta[at] : 0.f;
            }
            if (++t == per_head) { t = 0; ++g; }
        };
        started_sync();
        fetch();
        for (uint32_t i = 0; i < items; ++i) {
            const int b = i & 1;
            if (i >= 2 && !mbar_wait(&x.stat_free[b], ((i >> 1) - 1) & 1, &x.abort_flag, a.err)) break;
            float4* st = reinterpret_cast<float4*>(stats + b * 2 * kRows);
            st[lane] = make_float4(ls[0], ls[1], ls[2], ls[3]);
            st[32 + lane] = make_float4(dl[0], dl[1], dl[2], dl[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.stat_full[b]);
            if (i + 1 < items) fetch();
        }
    } else {
        const int w = warp >> 2;                             // columns 64 w .. 64 w + 63
        const int32_t j = key0 + (warp & 3) * 32 + lane;
        const float cs = a.scale * kLog2e;
        const int32_t end = j < a.N ? doc_of(j, a.seg, a.seqlen).y : 0;
        started_sync();
        const uint32_t tb = x.tmem_base;
        const uint32_t at = tb + ((uint32_t)((warp & 3) * 32) << 16) + 64 * w;
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
            const int32_t q0 = (t0 + t) * kRows;
            const int from = j - q0 - 64 * w, to = end - 1 - q0 - 64 * w;
            const float* st = stats + (i & 1) * 2 * kRows + 64 * w;
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
            if (!wait(&x.stat_full[i & 1], (i >> 1) & 1)) return false;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (kMask && see[b] == kSeeNone) {
                    fill32(p[b], 0.f);
                    continue;
                }
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
            if (!wait(&x.dp_full, phase)) return false;
            tmem_ld32(at + kDP, f[0]);
            tmem_ld32(at + kDP + 32, f[1]);
            tmem_wait_ld();
            store32(at + kDP, p[0]);
            store32(at + kDP + 16, p[1]);
            tmem_wait_st();
            signal(&x.p_ready);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (kMask && see[b] == kSeeNone) {
                    fill32(f[b], 0.f);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 d = *reinterpret_cast<const float4*>(st + kRows + 32 * b + e);
                        add2(f[b][e], f[b][e + 1], -d.x, -d.y);
                        add2(f[b][e + 2], f[b][e + 3], -d.z, -d.w);
                        mul2v(f[b][e], f[b][e + 1], p[b][e], p[b][e + 1]);
                        mul2v(f[b][e + 2], f[b][e + 3], p[b][e + 2], p[b][e + 3]);
                    }
                    if (kMask && see[b] == kSeeSome) hide32(f[b], bits[b], 0.f);
                }
                store32(at + kDP + 32 + 16 * b, f[b]);
                if (kMask && t == 0) {
                    remainder32(f[b]);
                    store32(at + 16 * b, f[b]);
                }
            }
            tmem_wait_st();
            signal(&x.ds_ready[0]);
            if (lane == 0) mbar_arrive(&x.stat_free[i & 1]);
            return true;
        };
        for (uint32_t i = 0; i < items; ++i, phase ^= 1) {
            const bool masked = t == 0 || (t0 + t + 1) * kRows > full_to;
            if (!(masked ? item(std::true_type{}, i) : item(std::false_type{}, i))) break;
            if (++t == per_head) t = 0;
        }
        ok = ok && wait(&x.done, 0) && wait(&x.scanned, 0);
        ok = !named_bar_any<1, 256>(!ok);                    // all warps go on, or none
        if (!ok) x.again = -1;                               // nothing is written then
        if (ranks > 1) {
            // this block's part, for the cluster: warps 0-3 dv, warps 4-7 dk
            float* row = reinterpret_cast<float*>(sm) + (size_t)(w * kRows + (warp & 3) * 32 + lane) * part_ld<HD>();
            const uint32_t src = tb + ((uint32_t)((warp & 3) * 32) << 16) + (w ? kDK : kDV);
#pragma unroll
            for (int b = 0; b < HD / 32; ++b) {
                float f[32];
                tmem_ld32(src + 32 * b, f);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(row + 32 * b + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
        } else if (ok && !x.again) {
            // warps 0-3 dv, warps 4-7 dk, through the resident tiles and TMA
            const uint32_t src = tb + ((uint32_t)((warp & 3) * 32) << 16) + (w ? kDK : kDV);
#pragma unroll
            for (int b = 0; b < HD / 32; ++b) {
                float f[32];
                tmem_ld32(src + 32 * b, f);
                tmem_wait_ld();
                tile_put32(w ? sK : sV, (warp & 3) * 32 + lane, b, f, w ? a.scale : 1.f);
            }
            fence_async_smem();
            element_sync();
            if (threadIdx.x == 0) {
                store_head_tile<HD>(&tdv, sV, kv, key0);
                store_head_tile<HD>(&tdk, sK, kv, key0);
                tma_store_commit();
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
        tmem_dealloc(x.tmem_base, 512);
    }
    if (ranks == 1) {
        if (threadIdx.x == 0) tma_store_wait_read_all();      // the gradients have left shared memory
        return;
    }
    join_parts<HD, kBwdThreads, 8>(a, cluster, &x.again, reinterpret_cast<const float*>(sm), kv, key0);
}

// ---------------------------------------------------------------- dq
__global__ void __launch_bounds__(kBwdThreads, 1) attn_dq_kernel(const __grid_constant__ CUtensorMap tq,
                                                                 const __grid_constant__ CUtensorMap tk,
                                                                 const __grid_constant__ CUtensorMap tv,
                                                                 const __grid_constant__ CUtensorMap td,
                                                                 const __grid_constant__ CUtensorMap to,
                                                                 const __grid_constant__ CUtensorMap tdq,
                                                                 const AttnTcArgs a) {
    using S = BwdSmem;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint8_t* sQ = sm;
    uint8_t* sO = sm + S::tile;
    uint8_t* ring = sm + S::ring;                            // place 0: O, 2 i + 1: K of item i, 2 i + 2: its V
    float* sX = reinterpret_cast<float*>(sm + S::stats);     // [2][128] halves of a sum over a row
    S::Shared& x = *reinterpret_cast<S::Shared*>(sm + S::shared);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t tiles = (a.N + kRows - 1) / kRows, total = tiles * a.heads;
    // The block's tiles: forwards through one stretch of the order (most work first), backwards through the next.
    struct Tile {
        int head;
        int32_t row0, lo, items;
    };
    auto tile_at = [&](int32_t t, Tile& c) {
        const int32_t g = (int32_t)gridDim.x, b = (int32_t)blockIdx.x, u = t * g + (t & 1 ? g - 1 - b : b);
        if (u >= total) return false;
        c.head = u % a.heads;
        c.row0 = tile_of(u / a.heads, tiles, a.seqlen % kRows ? 0 : a.seqlen / kRows, a.order_q, false) * kRows;
        c.lo = doc_of(c.row0, a.seg, a.seqlen).x / kRows;
        c.items = c.row0 / kRows - c.lo + 1;
        return true;
    };
    Tile c;
    if (misplaced(sm, a.err)) return;
    constexpr uint32_t kDP = 128, kDQ = 256, kDS = 384;      // dS: two buffers of 64 columns, a barrier each

    if (warp == 9) {
        if (lane == 0) bwd_init(x);
        __syncwarp();
        started_arrive();                                    // the loads need no TMEM
        if (lane == 0) {
            uint32_t n = 0;                                  // places of the ring
            int32_t t = 0, qs = 0, os = 0;                   // tiles begun, Q and dO loaded
            bool ok = true;
            auto put = [&](const CUtensorMap* map, int h, int32_t token) {
                const Spot at(n);
                if (n >= S::slots && !mbar_wait(&x.empty[at.slot], at.parity ^ 1, &x.abort_flag, a.err)) return false;
                mbar_arrive_expect_tx(&x.full[at.slot], S::tile);
                load_head_tile<HD>(ring + at.slot * S::tile, map, &x.full[at.slot], h, token);
                ++n;
                return true;
            };
            for (; ok && tile_at(t, c); ++t) {
                if (t > 0) ok = mbar_wait(&x.q_free, (t - 1) & 1, &x.abort_flag, a.err);
                if (!ok) break;
                mbar_arrive_expect_tx(&x.resident, S::tile);
                load_head_tile<HD>(sQ, &tq, &x.resident, c.head, c.row0);
                ++qs;
                const int kv = c.head / a.group;
                ok = put(&to, c.head, c.row0);
                for (int32_t i = 0; ok && i < c.items; ++i) {
                    ok = put(&tk, kv, (c.lo + i) * kRows) && put(&tv, kv, (c.lo + i) * kRows);
                    if (i == 0) {
                        if (t > 0) ok = ok && mbar_wait(&x.o_free, (t - 1) & 1, &x.abort_flag, a.err);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&x.o_full, S::tile);
                        load_head_tile<HD>(sO, &td, &x.o_full, c.head, c.row0);
                        ++os;
                    }
                }
            }
            if (*(volatile int*)&x.abort_flag) {             // no copy may land after the block has gone
                if (qs > 0) mbar_wait_drain(&x.resident, (qs - 1) & 1);
                if (os > 0) mbar_wait_drain(&x.o_full, (os - 1) & 1);
                for (uint32_t m = n > S::slots ? n - S::slots : 0; m < n; ++m)
                    mbar_wait_drain(&x.full[Spot(m).slot], Spot(m).parity);
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        tmem_alloc(&x.tmem_base, 512);
        tmem_relinquish();
        started_sync();
        const uint32_t tb = x.tmem_base;
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdG = idesc_bf16(128, HD, false, true);
        const uint32_t q_at = smem_u32(sQ), o_at = smem_u32(sO), r_at = smem_u32(ring);
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
        auto landed = [&](const Spot& p) { return mbar_wait(&x.full[p.slot], p.parity, &x.abort_flag, a.err); };
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = mbar_wait(bar, parity, &x.abort_flag, a.err);
            tc_fence_after();
            return got;
        };
        bool ok = true;
        uint32_t n = 0, g = 0;                               // places of the ring, items
        for (int32_t t = 0; ok && tile_at(t, c); ++t, n += 2 * c.items + 1) {
            auto scores = [&](int32_t i) {
                const Spot k(n + 2 * i + 1);
                nt(0, q_at, r_at + k.slot * S::tile, &x.s_full);
                if (lead && i == c.items - 1) umma_commit(&x.q_free);
            };
            auto products = [&](int32_t i) {
                const Spot v(n + 2 * i + 2);
                nt(kDP, o_at, r_at + v.slot * S::tile, &x.dp_full);
                if (lead) umma_commit(&x.empty[v.slot]);
            };
            // item i: its tile of K or V is there, and the item before has been read out of the columns
            auto k_there = [&](int32_t i) {
                return landed(Spot(n + 2 * i + 1)) && (g == 0 && i == 0 || wait(&x.s_free, (g + i - 1) & 1));
            };
            auto v_there = [&](int32_t i) {
                return landed(Spot(n + 2 * i + 2)) && (g == 0 && i == 0 || wait(&x.dp_free, (g + i - 1) & 1));
            };
            ok = wait(&x.resident, t & 1) && k_there(0);
            if (ok) scores(0);
            ok = ok && wait(&x.o_full, t & 1) && v_there(0);
            if (ok) products(0);
            for (int32_t i = 0; ok && i < c.items; ++i) {
                if (i + 1 < c.items) {
                    ok = k_there(i + 1);
                    if (ok) scores(i + 1);
                    ok = ok && v_there(i + 1);
                    if (ok) products(i + 1);
                }
                const uint32_t b = (g + i) & 1;
                ok = ok && wait(&x.ds_ready[b], ((g + i) >> 1) & 1);
                if (ok && lead) {
                    const Spot k(n + 2 * i + 1);
                    const uint32_t at = r_at + k.slot * S::tile;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        umma_ts_bf16(tb + kDQ, tb + kDS + 64 * b + 8 * e, mnmajor_desc(at, kAtom, 16 * e), kIdG, i > 0 || e > 0);
                    if (i == c.items - 1) {
                        // the remainders of the diagonal tile, over the last scores
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            umma_ts_bf16(tb + kDQ, tb + (e < 4 ? 8 * e : 64 + 8 * (e - 4)), mnmajor_desc(at, kAtom, 16 * e),
                                         kIdG, 1);
                    }
                    umma_commit(&x.empty[k.slot]);
                    if (i == c.items - 1) umma_commit(&x.done);
                }
                __syncwarp();
            }
            g += c.items;
        }
        if (!ok) {                                           // no product may run on in freed TMEM
            if (lead) umma_commit(&x.drained);
            mbar_wait_drain(&x.drained, 0);
        }
    } else if (warp == 10) {
        started_sync();
        bool ok = true;
        uint32_t n = 0;
        for (int32_t t = 0; ok && tile_at(t, c); ++t) {
            const int32_t full_from = doc_of(min(c.row0 + kRows, a.N) - 1, a.seg, a.seqlen).x;
            ok = mbar_wait(&x.d_done, t & 1, &x.abort_flag, a.err);
            if (!ok) break;
            if (lane == 0) {
                x.again = 0;                                 // every warp has read the last tile's
                mbar_arrive(&x.empty[Spot(n).slot]);         // O has been read
                mbar_arrive(&x.empty[Spot(n).slot]);
            }
            __syncwarp();
            ++n;
            for (int32_t i = 0; ok && i < 2 * c.items; ++i, ++n) {
                const Spot at(n);
                ok = mbar_wait(&x.full[at.slot], at.parity, &x.abort_flag, a.err);
                if (!ok) break;
                if (!(i & 1) && (i >> 1 == c.items - 1 || (c.lo + (i >> 1)) * kRows < full_from) &&
                    tile_nonfinite(ring + at.slot * S::tile, S::tile, lane) && lane == 0)
                    x.again = 1;
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.empty[at.slot]);
            }
            if (ok && lane == 0) mbar_arrive(&x.scanned);
        }
    } else if (warp < 8) {
        const int w = warp >> 2, row = (warp & 3) * 32 + lane;
        const float cs = a.scale * kLog2e;
        started_sync();
        const uint32_t tb = x.tmem_base;
        const uint32_t at = tb + ((uint32_t)((warp & 3) * 32) << 16) + 64 * w;
        const uint32_t ds_at = tb + ((uint32_t)((warp & 3) * 32) << 16) + kDS + 32 * w;
        bool ok = true, met;
        uint32_t phase = 0, g = 0, place = 0;                // items, places of the ring before this tile
        int32_t t = 0, n, start, full_from;
        float ls, dl;
        // a row's tile: its token, where its document starts, its lse (log2 units, negated)
        auto begin = [&]() {
            n = c.row0 + row;
            start = n < a.N ? doc_of(n, a.seg, a.seqlen).x : INT32_MAX;
            ls = n < a.N ? -a.lse[(int64_t)c.head * a.N + n] * kLog2e : 0.f;
            full_from = doc_of(min(c.row0 + kRows, a.N) - 1, a.seg, a.seqlen).x;
        };
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
        // D = dO . O
        auto row_sum = [&]() {
            const Spot o(place);
            if (!wait(&x.o_full, t & 1) || !wait(&x.full[o.slot], o.parity)) return false;
            const uint8_t* so = ring + o.slot * S::tile;
            dl = -(row_dot(sO, so, row) + row_dot(sO + kAtom, so + kAtom, row));
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.d_done);
            return true;
        };
        auto item = [&](auto with_mask, int32_t i) {
            constexpr bool kMask = decltype(with_mask)::value;
            const int32_t c0 = (c.lo + i) * kRows;
            const bool final = kMask && i == c.items - 1;
            const int from = start - c0 - 64 * w, to = n - c0 - 64 * w;
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
            if (i == 0 && !row_sum()) return false;          // while the tiles' loads and products run
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
            }
            if (final) {
                // D of the rows that see no other tile
                float y = 0.f, z = 0.f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    y = fmaf(p[0][e], f[0][e], y);
                    z = fmaf(p[1][e], f[1][e], z);
                }
                sX[w * kRows + row] = y + z;
                element_sync();
                met = true;
                if (start >= c0) dl = -(sX[row] + sX[kRows + row]);
                if (w == 0 && n < a.N) a.delta[(int64_t)c.head * a.N + n] = -dl;
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
                store32(ds_at + 64 * ((g + i) & 1) + 16 * b, f[b]);
                if (final) {
                    remainder32(f[b]);
                    store32(at + 16 * b, f[b]);
                }
            }
            tmem_wait_st();
            signal(&x.ds_ready[(g + i) & 1]);
            return true;
        };
        bool more = tile_at(0, c);
        if (more) begin();
        while (more) {
            met = false;
            for (int32_t i = 0; i < c.items; ++i, phase ^= 1) {
                const bool masked = i == c.items - 1 || (c.lo + i) * kRows < full_from;
                if (!(masked ? item(std::true_type{}, i) : item(std::false_type{}, i))) break;
            }
            if (!met) element_sync();                        // after an abort: the other warps may wait there
            const Tile now = c;
            g += c.items;
            place += 2 * c.items + 1;
            more = tile_at(t + 1, c);
            if (more) begin();
            ok = ok && wait(&x.done, t & 1) && wait(&x.scanned, t & 1);
            ok = !named_bar_any<1, 256>(!ok);                // all warps go on, or none
            if (!ok) break;
            if (!x.again) {
                // each half of the warps takes half of the channels, through dO's tile
#pragma unroll
                for (int b = w * (HD / 64); b < (w + 1) * (HD / 64); ++b) {
                    float f[32];
                    tmem_ld32(tb + ((uint32_t)((warp & 3) * 32) << 16) + kDQ + 32 * b, f);
                    tmem_wait_ld();
                    tile_put32(sO, row, b, f, a.scale);
                }
                fence_async_smem();
            } else {
                const int32_t r = now.row0 + warp * 16;
                dq_rows_again(a, now.head, r, min(16, a.N - r), lane);
            }
            signal(&x.staged);
            ++t;
        }
    } else {
        // the store of a tile's dQ, and dO's tile given back
        started_sync();
        bool ok = true;
        for (int32_t t = 0; ok && tile_at(t, c); ++t) {
            ok = mbar_wait(&x.staged, t & 1, &x.abort_flag, a.err);
            if (ok && lane == 0) {
                if (!*(volatile int*)&x.again) {
                    store_head_tile<HD>(&tdq, sO, c.head, c.row0);
                    tma_store_commit();
                    tma_store_wait_read_all();
                }
                mbar_arrive(&x.o_free);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(x.tmem_base, 512);
    }
}

cudaError_t bwd_wide(const AttnProb& p, const BwdMaps& m, const AttnTcArgs& a, cudaStream_t st) {
    constexpr uint32_t smem = BwdSmem::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_dkv_kernel, smem);
    if (e == cudaSuccess) e = DC_SMEM_LIMIT(attn_dq_kernel, smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + kRows - 1) / kRows;
    DC_LAUNCH(kAttnTcDq, st, attn_dq_kernel<<<(unsigned)std::min<int64_t>(tiles * p.heads, num_sms()), kBwdThreads, smem, st>>>(m.q, m.k, m.v, m.d, m.o,
                                                                                                   m.dq, a));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int ranks = dkv_ranks(p, tiles * p.kvh);
    DC_LAUNCH(kAttnTcDkv, st, e = launch_ranks(attn_dkv_kernel, ranks, (unsigned)(tiles * p.kvh * ranks), kBwdThreads,
                                               smem, st, m.q, m.k, m.v, m.d, m.dk, m.dv, a));
    return e;
}

}  // namespace
}  // namespace attn_tc

cudaError_t attn_tc_bwd(const AttnProb& p, const void* d_o, const void* q, const void* k, const void* v,
                        const void* o, const float* lse, float* delta, void* dq, void* dk, void* dv, uint32_t* err,
                        cudaStream_t st) {
    using namespace attn_tc;
    BwdMaps m;
    if (!make_head_map(&m.q, q, p.N, p.heads, p.hd, p.qs) || !make_head_map(&m.k, k, p.N, p.kvh, p.hd, p.ks) ||
        !make_head_map(&m.v, v, p.N, p.kvh, p.hd, p.vs) || !make_head_map(&m.d, d_o, p.N, p.heads, p.hd, p.dos) ||
        !make_head_map(&m.dq, dq, p.N, p.heads, p.hd, p.dqs) || !make_head_map(&m.dk, dk, p.N, p.kvh, p.hd, p.dks) ||
        !make_head_map(&m.dv, dv, p.N, p.kvh, p.hd, p.dvs) || !make_head_map(&m.o, o, p.N, p.heads, p.hd, p.os))
        return cudaErrorInvalidValue;
    if (p.hd <= 64 &&
        (!make_head_map(&m.q64, q, p.N, p.heads, p.hd, p.qs, 64) || !make_head_map(&m.k64, k, p.N, p.kvh, p.hd, p.ks, 64) ||
         !make_head_map(&m.v64, v, p.N, p.kvh, p.hd, p.vs, 64) || !make_head_map(&m.d64, d_o, p.N, p.heads, p.hd, p.dos, 64)))
        return cudaErrorInvalidValue;
    AttnTcArgs a = tc_args(p);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.d_o = static_cast<const __nv_bfloat16*>(d_o);
    a.o = const_cast<__nv_bfloat16*>(static_cast<const __nv_bfloat16*>(o));
    a.dq = static_cast<__nv_bfloat16*>(dq);
    a.dk = static_cast<__nv_bfloat16*>(dk);
    a.dv = static_cast<__nv_bfloat16*>(dv);
    a.lse = const_cast<float*>(lse);
    a.delta = delta;
    a.err = err;
    return p.hd <= 64 ? bwd_narrow(p, m, a, st) : bwd_wide(p, m, a, st);
}

}  // namespace dynconv
