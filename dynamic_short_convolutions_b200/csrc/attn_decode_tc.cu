// attn_decode_tc.cu -- a serving step over a cache on the tensor cores, for steps with many rows (drafted trees,
// large groups; bf16): the rows of a sequence's tokens and a group's heads share every key and value read.
//
// A block takes 128 rows r = m * group + g of one key/value head of one sequence and one run of its cached rows, as
// the forward of attn_tc_fwd.cu with keys and values by TMA from the cache and 512 columns of TMEM for itself: two
// buffers of scores, P beside them, O.  The rotated q goes in as value and remainder (two products: nothing else
// rounds it).  Rows of the last tile behind the cached ones hold whatever the cache holds there: their scores are
// masked and their values set to zero in shared memory.  The drafted rows are one more tile, filled from k and v
// and written to the cache by the block of the last run; infinities and NaN among their values are left out of
// the product (0 x NaN would reach rows that do not see them) and added to the rows that see them.
//
// The blocks of a cache's runs are a cluster: each leaves its result in shared memory, and all join them, a share of
// the rows each, in the order of the runs.
//
// Warps: 0-3 softmax (a row per thread); 4-7 the drafted tile, meanwhile; both rotate q before; 8 issues the MMAs;
// 9 the TMA loads.
//
// Measured: 8 sequences of ~2200 rows, trees of 24 tokens, 16 heads of 128 over 4: 25.7 us (1.5 TB/s; 48 with mma.sync and
// a join through memory).  About 10 us are the set-up, q's rotation and the join; a tile of 128 rows takes 2 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "attn_decode.cuh"
#include "attn_tc.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {

using namespace attn_dec;
using namespace attn_tc;

namespace {

namespace cg = cooperative_groups;

constexpr int kBlock = 320, kWorkers = 256;

template <int HD>
struct DecTcSmem {
    static constexpr uint32_t tile = kAtom * (HD / 64);
    static constexpr int slots = HD == 128 ? 4 : 8;
    static constexpr int ld = HD + 4;                            // a row of the result, padded
    static constexpr uint32_t bytes = 1024 + tile * (2 + slots);
    // the result uses the tiles' memory
    static_assert(kRows * ld * 4 <= tile * (2 + slots), "results fit the tiles");
};

// Barriers of the eight working warps, and of the four that fill the drafted tile.
__device__ __forceinline__ void work_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ void fill_sync() { asm volatile("bar.sync 3, 128;" ::: "memory"); }
// Byte offset of 16-byte chunk c (8 channels) of row r in a tile of 64-channel atoms.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(c / 8) * kAtom + sw128_off(r, c % 8); }

template <int HD>
__global__ void __launch_bounds__(kBlock, 1) attn_decode_tc_kernel(const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv,
                                                                   const __nv_bfloat16* __restrict__ q,
                                                                   const __nv_bfloat16* __restrict__ k,
                                                                   const __nv_bfloat16* __restrict__ v,
                                                                   __nv_bfloat16* k_cache, __nv_bfloat16* v_cache,
                                                                   __nv_bfloat16* __restrict__ o, const DecArgs a) {
    using S = DecTcSmem<HD>;
    constexpr int C = HD / 8;                                    // 16-byte chunks per row
    constexpr uint32_t kP = 256, kO = 320;                       // TMEM columns; S at 0 and 128
    extern __shared__ uint8_t raw[];
    uint8_t* sQ = align1024(raw);                                // q, then its remainder
    uint8_t* ring = sQ + 2 * S::tile;                            // place 2 i: K of tile i, 2 i + 1: its V
    __shared__ uint64_t q_full, full[S::slots], empty[S::slots], s_full[2], s_free[2], p_ready, pv_done, room, drained;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, poison;
    __shared__ uint64_t seen[64];
    __shared__ const float* turn[64];
    __shared__ float smax[kRows], ssum[kRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cg::cluster_group cluster = cg::this_cluster();
    Place p = place_of<kRows>(a, kRows);                         // p.split is the block's rank
    if (!p.idle && !look_up(a, p, seen, turn)) {
        p.idle = true;
        if (threadIdx.x == 0) atomicOr(a.err, kErrRopePos);
    }
    if (p.idle) {
        zero_rows<__nv_bfloat16, kRows>(a, p, o);
        return;
    }
    const int64_t slot = (p.b * a.kvh + p.kv) * a.max_len;       // the cache's first row
    const int tiles = (int)((p.to - p.from + kRows - 1) / kRows), items = tiles + (p.tail ? 1 : 0);
    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        for (int s = 0; s < S::slots; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {                            // of either buffer of scores
            mbar_init(&s_full[b], 1);
            mbar_init(&s_free[b], 4);
        }
        mbar_init(&p_ready, 4);
        mbar_init(&pv_done, 1);
        mbar_init(&room, 1);
        mbar_init(&drained, 1);
        abort_flag = 0;
        poison = 0;
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
        if (lane == 0) {
            const int32_t cache = (int32_t)(p.b * a.kvh + p.kv);
            int n = 0;
            for (; n < 2 * tiles; ++n) {
                const int s = n % S::slots, use = n / S::slots;
                if (use > 0 && !mbar_wait(&empty[s], (use - 1) & 1, &abort_flag, a.err)) break;
                mbar_arrive_expect_tx(&full[s], S::tile);
                const int32_t row = (int32_t)p.from + (n >> 1) * kRows;
#pragma unroll
                for (int c = 0; c < HD / 64; ++c)
                    tma_load_3d(ring + s * S::tile + c * kAtom, n & 1 ? &tv : &tk, &full[s], 64 * c, row, cache);
            }
            // The drafted tile takes the next two places.  This thread has followed the slots' phases: others that waited
            // on them from afar could take the parity of an earlier phase for the one they mean.
            bool got = n == 2 * tiles;
            for (int e = n; got && p.tail && e < n + 2; ++e)
                got = e < S::slots || mbar_wait(&empty[e % S::slots], (e / S::slots - 1) & 1, &abort_flag, a.err);
            if (got) mbar_arrive(&room);
            if (*(volatile int*)&abort_flag)                     // no copy may land after the block has gone
                for (int m = n > S::slots ? n - S::slots : 0; m < n; ++m)
                    mbar_wait_drain(&full[m % S::slots], (m / S::slots) & 1);
        }
        __syncwarp();
    } else if (warp == 8) {
        constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
        constexpr uint32_t kIdO = idesc_bf16(128, HD, false, true);
        const uint32_t q_at = smem_u32(sQ), r_at = smem_u32(ring);
        const bool lead = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = mbar_wait(bar, parity, &abort_flag, a.err);
            tc_fence_after();
            return got;
        };
        auto scores = [&](int i) {
            const int n = 2 * i, s = n % S::slots;
            if (!wait(&full[s], (n / S::slots) & 1)) return false;
            if (lead) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
                    if (part == 0 || a.rot)
#pragma unroll
                        for (int c = 0; c < HD / 16; ++c)
                            umma_bf16(tb + 128 * (i & 1), kmajor_desc(q_at + part * S::tile + (c / 4) * kAtom, c % 4),
                                      kmajor_desc(r_at + s * S::tile + (c / 4) * kAtom, c % 4), kIdS, part + c != 0);
                umma_commit(&s_full[i & 1]);
                umma_commit(&empty[s]);
            }
            return true;
        };
        bool ok = items == 0 || (wait(&q_full, 0) && scores(0));
        for (int i = 0; ok && i < items; ++i) {
            const int n = 2 * i + 1, s = n % S::slots;
            // the buffer of the next scores was read two tiles ago
            if (i + 1 < items) ok = (i == 0 || wait(&s_free[(i - 1) & 1], ((i - 1) >> 1) & 1)) && scores(i + 1);
            ok = ok && wait(&full[s], (n / S::slots) & 1) && wait(&p_ready, i & 1);
            if (ok && lead) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    umma_ts_bf16(tb + kO, tb + kP + 8 * c, mnmajor_desc(r_at + s * S::tile, kAtom, 16 * c), kIdO,
                                 i > 0 || c > 0);
                umma_commit(&pv_done);
                umma_commit(&empty[s]);
            }
            __syncwarp();
        }
        if (lead) umma_commit(&drained);                         // every MMA done before TMEM is freed
        mbar_wait_drain(&drained, 0);
    } else {
        bool ok = true;
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
        const int r = threadIdx.x, row = p.tile * kRows + r;     // a softmax thread's row
        const int token = r < kRows && row < a.rows ? row / a.group : -1;
        // ---- q
        const int units = units_of(a, a.hd / 8);
#pragma unroll 2
        for (int i = threadIdx.x; i < kRows * units; i += kWorkers) {
            const int t = i / units, u = i - t * units, at = p.tile * kRows + t;
            if (at >= a.rows) continue;
            const int m = at / a.group, g = at - m * a.group;
            turn_unit(a, q + (p.b * a.M + m) * a.qs + ((int64_t)p.kv * a.group + g) * a.hd, u, turn[m],
                      [&](int c, const float (&x)[8]) {
                          uint32_t hi[4], lo[4];
#pragma unroll
                          for (int e = 0; e < 4; ++e) {
                              hi[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
                              lo[e] = pack_bf16(x[2 * e] - bf16_lo(hi[e]), x[2 * e + 1] - bf16_hi(hi[e]));
                          }
                          *reinterpret_cast<uint4*>(sQ + chunk_at(t, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                          if (a.rot) *reinterpret_cast<uint4*>(sQ + S::tile + chunk_at(t, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                      });
        }
        // rows and channels that are none: zeros
        const int real = min(kRows, a.rows - p.tile * kRows);
        for (int i = threadIdx.x; i < kRows * C; i += kWorkers) {
            const int t = i / C, c = i % C;
            if (t < real && c * 8 < a.hd) continue;
            *reinterpret_cast<uint4*>(sQ + chunk_at(t, c)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(sQ + S::tile + chunk_at(t, c)) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        work_sync();
        if (threadIdx.x == 0) mbar_arrive(&q_full);
        float m = -INFINITY, l0 = 0.f, l1 = 0.f;                 // running maximum (log2 units), halves of the sum
        // ---- the drafted tile
        auto draft = [&]() {
            const int n = 2 * tiles;
            uint8_t* kt = ring + n % S::slots * S::tile;
            uint8_t* vt = ring + (n + 1) % S::slots * S::tile;
            wait(&room, 0);
            bool bad = false;
            const int at = threadIdx.x - kThreads;
            if (ok) {
                for (int i = at; i < a.M * units; i += kThreads) {
                    const int t = i / units, u = i - t * units;
                    turn_unit(a, k + (p.b * a.M + t) * a.ks + (int64_t)p.kv * a.hd, u, turn[t], [&](int c, const float (&f)[8]) {
                        const uint4 x = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                                   pack_bf16(f[6], f[7]));
                        *reinterpret_cast<uint4*>(kt + chunk_at(t, c)) = x;
                        if (p.tile == 0) *reinterpret_cast<uint4*>(k_cache + (slot + p.len + t) * a.hd + c * 8) = x;
                    });
                }
#pragma unroll 4
                for (int i = at; i < kRows * C; i += kThreads) {
                    const int t = i / C, c = i % C;
                    uint4 y = make_uint4(0, 0, 0, 0);
                    if (t < a.M && c * 8 < a.hd) {
                        y = __ldg(reinterpret_cast<const uint4*>(v + (p.b * a.M + t) * a.vs + (int64_t)p.kv * a.hd + c * 8));
                        if (p.tile == 0) *reinterpret_cast<uint4*>(v_cache + (slot + p.len + t) * a.hd + c * 8) = y;
                        uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t odd = nonfinite_bits(w[e]);
                            bad = bad || odd;
                            w[e] &= ~((odd & 0x8000u ? 0xFFFFu : 0u) | (odd & 0x80000000u ? 0xFFFF0000u : 0u));
                        }
                    } else {
                        *reinterpret_cast<uint4*>(kt + chunk_at(t, c)) = y;
                    }
                    *reinterpret_cast<uint4*>(vt + chunk_at(t, c)) = y;
                }
            }
            if (bad) poison = 1;
            fence_async_smem();
            fill_sync();
            if (threadIdx.x == kThreads && ok) {
                mbar_arrive(&full[n % S::slots]);
                mbar_arrive(&full[(n + 1) % S::slots]);
            }
        };
        if (warp >= 4 && p.tail) draft();
        // ---- softmax
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const uint32_t tP = tb + lanes + kP, tO = tb + lanes + kO;
        const float cs = a.scale * kLog2e;
        // One tile; two copies of the code, so that whole cached tiles pay nothing for masks.
        auto tile = [&](auto with_mask, int i) {
            constexpr bool kMask = decltype(with_mask)::value;
            const uint32_t tS = tb + lanes + 128 * (i & 1);
            const int64_t left = i < tiles ? p.to - p.from - (int64_t)i * kRows : 0;       // cached rows of the tile
            uint32_t bits[4];
            if (i == tiles) {
                const uint64_t s = token >= 0 ? seen[token] : 0;
                bits[0] = (uint32_t)s;
                bits[1] = (uint32_t)(s >> 32);
                bits[2] = bits[3] = 0;
            } else {
#pragma unroll
                for (int b = 0; b < 4; ++b) bits[b] = seen_bits(32 * b, 0, (int)left - 1);
            }
            if (!wait(&s_full[i & 1], (i >> 1) & 1)) return false;
            float s0[32], s1[32], mx[4];
            tmem_ld32(tS + 64, s0);
            tmem_ld32(tS + 96, s1);
            tmem_wait_ld();
            if (kMask) hide32(s0, bits[2], -INFINITY);
            if (kMask) hide32(s1, bits[3], -INFINITY);
            mx[0] = max32(s0);
            mx[1] = max32(s1);
            tmem_ld32(tS, s0);
            tmem_ld32(tS + 32, s1);
            tmem_wait_ld();
            if (kMask) hide32(s0, bits[0], -INFINITY);
            if (kMask) hide32(s1, bits[1], -INFINITY);
            mx[2] = max32(s0);
            mx[3] = max32(s1);
            const float top = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs);
            if (i > 0 && !wait(&pv_done, (i - 1) & 1)) return false;
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
            const float neg = m == -INFINITY ? 0.f : -m;         // a row that has seen no key yet
            probs32(s0, cs, neg, l0, l1, tP);
            probs32(s1, cs, neg, l0, l1, tP + 16);
            tmem_ld32(tS + 64, s0);
            tmem_ld32(tS + 96, s1);
            tmem_wait_ld();
            signal(&s_free[i & 1]);
            if (kMask) hide32(s0, bits[2], -INFINITY);
            if (kMask) hide32(s1, bits[3], -INFINITY);
            probs32(s0, cs, neg, l0, l1, tP + 32);
            probs32(s1, cs, neg, l0, l1, tP + 48);
            tmem_wait_st();
            if (kMask && i < tiles) {
                // values behind the cached rows: zeros
                const int n = 2 * i + 1;
                if (!wait(&full[n % S::slots], (n / S::slots) & 1)) return false;
                if (r >= left)
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        *reinterpret_cast<uint4*>(ring + n % S::slots * S::tile + chunk_at(r, c)) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
            }
            signal(&p_ready);
            return true;
        };
        for (int i = 0; warp < 4 && i < items; ++i) {
            const bool masked = i == tiles || p.to - p.from - (int64_t)i * kRows < kRows;
            if (!(masked ? tile(std::true_type{}, i) : tile(std::false_type{}, i))) break;
        }
        if (warp < 4) ok = ok && (items == 0 || wait(&pv_done, (items - 1) & 1));
        ok = !named_bar_any<1, kWorkers>(!ok);                   // all go on, or none: the tiles' memory is free
        float* so = reinterpret_cast<float*>(sQ);
        if (ok && warp < 4) {
            const uint64_t bad = poison && p.tail && token >= 0 ? seen[token] : 0;
#pragma unroll 1
            for (int b = 0; b < HD / 32; ++b) {
                float f[32];
                if (items > 0) {
                    tmem_ld32(tO + 32 * b, f);
                    tmem_wait_ld();
                } else {
                    fill32(f, 0.f);
                }
                if (bad != 0)
                    for (int j = 0; j < a.M; ++j)
                        if (bad >> j & 1)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (32 * b + e < a.hd) {
                                    const float x = __bfloat162float(v[(p.b * a.M + j) * a.vs + (int64_t)p.kv * a.hd + 32 * b + e]);
                                    if (!(fabsf(x) < INFINITY)) f[e] += x;
                                }
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(so + r * S::ld + 32 * b + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
            }
            if (l0 + l1 == 0.f && sees_nothing(a, p, seen, row)) m = 0.f, l0 = 1.f;
            smax[r] = m;
            ssum[r] = l0 + l1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tb, 512);
    }
    // Every thread of every block of the cluster comes here (idle slots left together), whatever became of its waits.
    cluster.sync();
    const float* so = reinterpret_cast<const float*>(sQ);
    const int rows = min(kRows, a.rows - p.tile * kRows);
    for (int i = threadIdx.x; i < (rows - p.split + a.n_split - 1) / a.n_split * (HD / 4); i += kBlock) {
        const int t = i / (HD / 4) * a.n_split + p.split, c = i % (HD / 4) * 4;
        if (c >= a.hd) continue;
        float mx = -INFINITY, l = 0.f;
        for (int n = 0; n < a.n_split; ++n) mx = fmaxf(mx, cluster.map_shared_rank(smax, n)[t]);
        const float use = mx == -INFINITY ? 0.f : mx;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int n = 0; n < a.n_split; ++n) {
            const float w = ex2(cluster.map_shared_rank(smax, n)[t] - use);
            const float4 x = *reinterpret_cast<const float4*>(cluster.map_shared_rank(so, n) + t * S::ld + c);
            s.x += w * x.x; s.y += w * x.y; s.z += w * x.z; s.w += w * x.w;
            l += w * cluster.map_shared_rank(ssum, n)[t];
        }
        const int at = p.tile * kRows + t, m = at / a.group, g = at - m * a.group;
        const float inv = 1.f / l;
        *reinterpret_cast<uint2*>(o + (p.b * a.M + m) * a.os + ((int64_t)p.kv * a.group + g) * a.hd + c) =
            make_uint2(pack_bf16(s.x * inv, s.y * inv), pack_bf16(s.z * inv, s.w * inv));
    }
    cluster.sync();                                              // no block leaves while its result is read
}

template <int HD>
cudaError_t launch_tc(const CUtensorMap& tk, const CUtensorMap& tv, const DecArgs& a, unsigned grid, const void* q,
                      const void* k, const void* v, void* kc, void* vc, void* o, cudaStream_t st) {
    using B = __nv_bfloat16;
    constexpr uint32_t smem = DecTcSmem<HD>::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_decode_tc_kernel<HD>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.n_split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DC_LAUNCH(kAttnDecodeTc, st, e = cudaLaunchKernelEx(&cfg, attn_decode_tc_kernel<HD>, tk, tv, static_cast<const B*>(q),
                                                        static_cast<const B*>(k), static_cast<const B*>(v),
                                                        static_cast<B*>(kc), static_cast<B*>(vc), static_cast<B*>(o), a));
    return e;
}

}  // namespace

cudaError_t attn_decode_tc(const DecodeProb& p, const DecArgs& a, unsigned grid, const void* q, const void* k,
                           const void* v, void* k_cache, void* v_cache, void* o, cudaStream_t st) {
    CUtensorMap tk, tv;
    if (!make_cache_map(&tk, k_cache, p, kRows) || !make_cache_map(&tv, v_cache, p, kRows))
        return cudaErrorInvalidValue;
    return p.hd <= 64 ? launch_tc<64>(tk, tv, a, grid, q, k, v, k_cache, v_cache, o, st)
                      : launch_tc<128>(tk, tv, a, grid, q, k, v, k_cache, v_cache, o, st);
}

}  // namespace dynconv
