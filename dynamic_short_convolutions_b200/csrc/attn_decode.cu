// attn_decode.cu -- attention of new or drafted tokens over a key/value cache, one launch per step:
// rotation of q and k at their positions, appending to the caches, and
//   o_m = softmax(scale q_m . k_j) v_j   over the cached rows j < L and the drafted rows m may see.
//
// Memory-bound for single tokens: the cache is read once.  A block takes one key/value head of one
// sequence, so all heads of the group and all its tokens (rows r = m * group + g) share each key and value
// read, and one of n_split runs of the cached rows, because batch x kv_heads alone would not fill the GPU;
// runs follow the sequence's own length.  Tiles of K and V come through a ring of 16-byte asynchronous
// copies (rows beyond L are zero-filled, never read; the 8-row kernel's and the tcgen05 kernel's TMA boxes do read
// them, mask their scores and set their values to zero).  The drafted rows are a last tile that the block
// of the last run fills from k and v (rotated, rounded to the storage type as the cache holds them) and also
// writes to the cache.  Partial results of the runs are joined in their order by the block that finishes
// last (a counter per head and sequence, reset by it), so results repeat bitwise.
//
// bf16, up to 8 rows (single tokens): the products are turned round, S^T = K Q^T and O^T = V^T P^T, so that the rows
// are the 8 columns of an mma.sync and none of it is empty but for missing rows (half the instructions of 16-row
// tiles); each warp walks slices of 16 cached rows by itself, with a TMA ring of its own, and no barrier.
// bf16, up to 32 rows: mma.sync m16n8k16 (a tcgen05 tile of 128 rows would be mostly empty; more rows run in
// attn_decode_tc.cu); P is rounded to bf16 because the tensor cores take it so, its sum is taken before; the rotated
// q is kept as two bf16 (value and remainder), since nothing else rounds it.  fp32: FMAs, a warp per four rows.
//
// Measured: 64 sequences of ~3000 rows, 16 heads of 128 over 4, one token: 71 us, 5.6 TB/s (0.85 of the copy rate; 88
// on 16-row tiles); 64 of 3000, 4 tokens (16 rows): 75 us, 5.3 TB/s; 8 tokens (32 rows): 99 us, 4.0 TB/s, where the
// barriers of a tile and 255 registers tell; one of ~700 rows, 12 heads of 64: 8.3 us, the chain length, rows, softmax,
// join.  fp32: the first 154 us (5.1 TB/s, 0.78), the second 11.3, 13 of ~560 rows with 3 tokens and 4 heads a group 14.9.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_decode.cuh"
#include "prof.h"
#include "smem_limit.h"

namespace dynconv {

using namespace attn_dec;

namespace {

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// ---------------------------------------------------------------- bf16
constexpr int kTok = 64;                             // tokens per tile
constexpr int kStages = 3;

// Byte offset of 16-byte chunk c of row r in a tile of HD bf16 per row: chunks permuted within a row's
// 128-byte half so that the eight rows of an ldmatrix fall in different banks.
template <int HD>
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * HD * 2 + ((c ^ (r & 7)) << 4)); }

template <int HD>
struct DecSmem {
    static constexpr uint32_t half = kTok * HD * 2;              // K or V of a tile
    static constexpr uint32_t bytes = kStages * 2 * half;        // the parts and q use the ring's memory
};

template <int HD, int RW>
__global__ void __launch_bounds__(kThreads) attn_decode_kernel(const __nv_bfloat16* __restrict__ q,
                                                               const __nv_bfloat16* __restrict__ k,
                                                               const __nv_bfloat16* __restrict__ v,
                                                               __nv_bfloat16* k_cache, __nv_bfloat16* v_cache,
                                                               __nv_bfloat16* __restrict__ o, const DecArgs a) {
    using S = DecSmem<HD>;
    constexpr int ROWS = 16 * RW, TW = 4 / RW;                   // a warp: 16 rows, 64 / TW tokens of each tile,
    constexpr int NT = RW == 1 ? 16 : 32, GROUPS = kTok / TW / NT;   // in groups of NT
    constexpr int C = HD / 8;                                    // 16-byte chunks per row
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float smax[TW * ROWS], ssum[TW * ROWS];
    __shared__ uint64_t seen[64];
    __shared__ const float* turn[64];
    __shared__ float scratch[4][16][NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rw = warp % RW, tw = warp / RW;
    Place p = place_of<ROWS>(a, kTok);
    const int64_t slot = (p.b * a.kvh + p.kv) * a.max_len;
    const uint32_t ring = smem_at(sm);
    const int tiles = (int)((p.to - p.from + kTok - 1) / kTok);

    auto fetch = [&](int t) {                                    // cached tile t of this run
        if (t < tiles) {
            const int64_t r0 = p.from + (int64_t)t * kTok;
            const uint32_t at = ring + (t % kStages) * 2 * S::half;
            for (int i = threadIdx.x; i < kTok * C; i += kThreads) {
                const int r = i / C, c = i % C;
                const bool real = r0 + r < p.to && c * 8 < a.hd;
                const int64_t src = (slot + (real ? r0 + r : 0)) * a.hd + (real ? c * 8 : 0);
                copy16(at + swz<HD>(r, c), k_cache + src, real);
                copy16(at + S::half + swz<HD>(r, c), v_cache + src, real);
            }
        }
        copies_close();
    };
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) fetch(t);
    if (!p.idle && !look_up(a, p, seen, turn)) {
        p.idle = true;
        if (threadIdx.x == 0) atomicOr(a.err, kErrRopePos);
    }
    if (p.idle) {
        copies_wait<0>();
        zero_rows<__nv_bfloat16, ROWS>(a, p, o);
        return;
    }
    // q, rotated, as value and remainder, through the last stage of the ring
    uint8_t* sq = sm + (kStages - 1) * 2 * S::half;
#pragma unroll 4
    for (int i = threadIdx.x; i < ROWS * C; i += kThreads) {
        const int r = i / C, c = i % C, row = p.tile * ROWS + r;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (row < a.rows && c * 8 < a.hd) {
            const int m = row / a.group, g = row - m * a.group;
            turned(q + (p.b * a.M + m) * a.qs + ((int64_t)p.kv * a.group + g) * a.hd, c * 8, turn[m], a.rot, a.half, x);
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = pack2(x[2 * e], x[2 * e + 1]);
            lo[e] = pack2(x[2 * e] - __uint_as_float(hi[e] << 16), x[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
        *reinterpret_cast<uint4*>(sq + swz<HD>(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sq + ROWS * HD * 2 + swz<HD>(r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();
    uint32_t qh[HD / 16][4], ql[HD / 16][4];
#pragma unroll
    for (int c = 0; c < HD / 16; ++c) {
        const uint32_t at = smem_at(sq) + swz<HD>(16 * rw + (lane & 15), 2 * c + (lane >> 4));
        ldsm4(qh[c], at);
        ldsm4(ql[c], at + ROWS * HD * 2);
    }
    __syncthreads();

    float acc[HD / 8][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < HD / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    const float cs = a.scale * kLog2e;
    const int total = tiles + (p.tail ? 1 : 0);
    for (int t = 0; t < total; ++t) {
        const bool draft = t == tiles;
        uint8_t* tile = sm + (t % kStages) * 2 * S::half;
        bool poison = false;                                     // infinities or NaN among the drafted values
        if (!draft) {
            fetch(t + kStages - 1);
            copies_wait<kStages - 1>();
            __syncthreads();
        } else {
            copies_wait<0>();
            __syncthreads();
            bool bad = false;
            const bool write = p.tile == 0;
#pragma unroll 2
            for (int i = threadIdx.x; i < kTok * C; i += kThreads) {
                const int r = i / C, c = i % C;
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (r < a.M && c * 8 < a.hd) {
                    float f[8];
                    turned(k + (p.b * a.M + r) * a.ks + (int64_t)p.kv * a.hd, c * 8, turn[r], a.rot, a.half, f);
                    x = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                    y = __ldg(reinterpret_cast<const uint4*>(v + (p.b * a.M + r) * a.vs + (int64_t)p.kv * a.hd + c * 8));
                    // an exponent of ones in either half of a word
                    auto odd = [](uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; };
                    bad = bad || (odd(y.x) | odd(y.y) | odd(y.z) | odd(y.w));
                    if (write) {
                        *reinterpret_cast<uint4*>(k_cache + (slot + p.len + r) * a.hd + c * 8) = x;
                        *reinterpret_cast<uint4*>(v_cache + (slot + p.len + r) * a.hd + c * 8) = y;
                    }
                }
                *reinterpret_cast<uint4*>(tile + swz<HD>(r, c)) = x;
                *reinterpret_cast<uint4*>(tile + S::half + swz<HD>(r, c)) = y;
            }
            poison = __syncthreads_or(bad) != 0;
        }
        const uint32_t kt = smem_at(tile), vt = kt + S::half;
        const int64_t left = draft ? a.M : p.to - p.from - (int64_t)t * kTok;     // real rows of the tile
#pragma unroll 1
        for (int gi = 0; gi < GROUPS; ++gi) {
            const int c0 = NT * (GROUPS * tw + gi);              // first of NT tokens
            if (c0 >= left || p.tile * ROWS + 16 * rw >= a.rows) continue;
            float s[NT / 8][4];
#pragma unroll
            for (int n = 0; n < NT / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) {
#pragma unroll
                for (int n = 0; n < NT / 16; ++n) {
                    uint32_t b[4];
                    ldsm4(b, kt + swz<HD>(c0 + 16 * n + (lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1)));
                    mma16816(s[2 * n], qh[c], b[0], b[1]);
                    mma16816(s[2 * n + 1], qh[c], b[2], b[3]);
                    if (a.rot) {
                        mma16816(s[2 * n], ql[c], b[0], b[1]);
                        mma16816(s[2 * n + 1], ql[c], b[2], b[3]);
                    }
                }
            }
            // rows 16 rw + lane / 4 (e 0, 1) and + 8 (e 2, 3), tokens c0 + 8 n + 2 (lane % 4) + (e & 1)
            uint32_t hidden = 0;
            if (draft || left < kTok) {
#pragma unroll
                for (int n = 0; n < NT / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int tok = c0 + 8 * n + 2 * (lane & 3) + (e & 1);
                        const int row = p.tile * ROWS + 16 * rw + (lane >> 2) + 8 * (e >> 1);
                        const bool see = tok < left && (!draft || (row < a.rows && (seen[row / a.group] >> tok & 1)));
                        if (!see) {
                            s[n][e] = -INFINITY;
                            hidden |= 1u << (4 * n + e);
                        }
                    }
            }
            uint32_t pa[NT / 16][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < NT / 8; ++n) top = fmaxf(top, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                const float now = fmaxf(mx[h], top * cs), use = now == -INFINITY ? 0.f : now;
                const float corr = exp2f(mx[h] - use);
                mx[h] = now;
                float add = 0.f;
#pragma unroll
                for (int n = 0; n < NT / 8; ++n) {
                    s[n][2 * h] = exp2f(fmaf(s[n][2 * h], cs, -use));
                    s[n][2 * h + 1] = exp2f(fmaf(s[n][2 * h + 1], cs, -use));
                    add += s[n][2 * h] + s[n][2 * h + 1];
                    pa[n / 2][2 * (n & 1) + h] = pack2(s[n][2 * h], s[n][2 * h + 1]);
                }
                sum[h] = sum[h] * corr + add;
                if (corr != 1.f) {
#pragma unroll
                    for (int n = 0; n < HD / 8; ++n) {
                        acc[n][2 * h] *= corr;
                        acc[n][2 * h + 1] *= corr;
                    }
                }
            }
            if (!poison) {
#pragma unroll
                for (int n = 0; n < HD / 16; ++n)
#pragma unroll
                    for (int x = 0; x < NT / 16; ++x) {
                        uint32_t b[4];
                        ldsm4t(b, vt + swz<HD>(c0 + 16 * x + (lane & 15), 2 * n + (lane >> 4)));
                        mma16816(acc[2 * n], pa[x], b[0], b[1]);
                        mma16816(acc[2 * n + 1], pa[x], b[2], b[3]);
                    }
            } else {
                // term by term, without the masked ones (0 x NaN would be NaN); a masked place is marked by -1
                __syncwarp();
#pragma unroll
                for (int n = 0; n < NT / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        scratch[warp][(lane >> 2) + 8 * (e >> 1)][8 * n + 2 * (lane & 3) + (e & 1)] =
                            hidden >> (4 * n + e) & 1 ? -1.f : s[n][e];
                __syncwarp();
#pragma unroll 1
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int n = 0; n < HD / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float w = scratch[warp][(lane >> 2) + 8 * (e >> 1)][c];
                            const int d = 2 * (lane & 3) + (e & 1);
                            if (w != -1.f)
                                acc[n][e] = fmaf(w, __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                                                        tile + S::half + swz<HD>(c0 + c, n) + 2 * d)), acc[n][e]);
                        }
            }
        }
        __syncthreads();                                         // the tile's stage is filled again
    }
    copies_wait<0>();
    __syncthreads();
    // parts of the TW token groups, in the ring's memory
    float* so = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], 1);
        sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], 2);
        const int r = tw * ROWS + 16 * rw + (lane >> 2) + 8 * h;
        if ((lane & 3) == 0) {
            const bool none = sees_nothing(a, p, seen, p.tile * ROWS + r - tw * ROWS);
            smax[r] = none ? 0.f : mx[h];
            ssum[r] = none ? 1.f : sum[h];
        }
#pragma unroll
        for (int n = 0; n < HD / 8; ++n)
            *reinterpret_cast<float2*>(so + r * HD + 8 * n + 2 * (lane & 3)) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
    }
    __syncthreads();
    finish<__nv_bfloat16, HD, ROWS, TW>(a, p, so, smax, ssum, so + TW * ROWS * HD, o);
}

// ---------------------------------------------------------------- bf16, up to 8 rows
constexpr int kSlice = 16;                           // cached rows a warp takes at a time

template <int HD>
struct Dec8Smem {
    static constexpr uint32_t half = kSlice * HD * 2, atom = kSlice * 128;   // K or V of a slice; 64 channels of it
    static constexpr int stages = HD == 128 ? 3 : 6;
    static constexpr uint32_t bytes = 1024 + 4 * stages * 2 * half;
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two blocks per SM, which is what its ring leaves room for (without the bound the compiler takes 128 registers and
// holds back loads of the join: 64 sequences of ~3000 rows 74.3 us for 73.2).
template <int HD>
__global__ void __launch_bounds__(kThreads, 2) attn_decode8_kernel(const __grid_constant__ CUtensorMap tk,
                                                                   const __grid_constant__ CUtensorMap tv,
                                                                   const __nv_bfloat16* __restrict__ q,
                                                                   const __nv_bfloat16* __restrict__ k,
                                                                   const __nv_bfloat16* __restrict__ v,
                                                                   __nv_bfloat16* k_cache, __nv_bfloat16* v_cache,
                                                                   __nv_bfloat16* __restrict__ o, const DecArgs a) {
    using S = Dec8Smem<HD>;
    constexpr int ROWS = 8, C = HD / 8, kPitch = HD * 2 + 16;    // q rows padded: an ldmatrix's eight fall in other banks
    extern __shared__ uint8_t raw[];
    uint8_t* ring = tc::align1024(raw);
    __shared__ __align__(16) uint8_t sq[2 * ROWS * kPitch];      // q, its remainder
    __shared__ uint64_t full[4][S::stages];
    __shared__ float smax[4 * ROWS], ssum[4 * ROWS];
    __shared__ uint64_t seen[64];
    __shared__ const float* turn[64];
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Place p = place_of<ROWS>(a, 4 * kSlice);
    if (threadIdx.x == 0) {
        for (int w = 0; w < 4; ++w)
            for (int s = 0; s < S::stages; ++s) tc::mbar_init(&full[w][s], 1);
        abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (!p.idle && !look_up(a, p, seen, turn)) {                 // its barrier: the mbarriers too are ready
        p.idle = true;
        if (threadIdx.x == 0) atomicOr(a.err, kErrRopePos);
    }
    if (p.idle) {
        zero_rows<__nv_bfloat16, ROWS>(a, p, o);
        return;
    }
    const int64_t slot = (p.b * a.kvh + p.kv) * a.max_len;
    const int32_t cache = (int32_t)(p.b * a.kvh + p.kv);
    const int slices = (int)((p.to - p.from + kSlice - 1) / kSlice);
    const int mine = slices > warp ? (slices - warp + 3) / 4 : 0;            // slices warp, warp + 4, ...
    uint8_t* own = ring + warp * S::stages * 2 * S::half;
    auto fetch = [&](int i) {                                    // one lane: this warp's slice i
        uint8_t* to = own + i % S::stages * 2 * S::half;
        uint64_t* bar = &full[warp][i % S::stages];
        const int32_t row = (int32_t)p.from + (warp + 4 * i) * kSlice;
        tc::mbar_arrive_expect_tx(bar, 2 * S::half);
#pragma unroll
        for (int c = 0; c < HD / 64; ++c) {
            attn_tc::tma_load_3d(to + c * S::atom, &tk, bar, 64 * c, row, cache);
            attn_tc::tma_load_3d(to + S::half + c * S::atom, &tv, bar, 64 * c, row, cache);
        }
    };
    if (lane == 0)
        for (int i = 0; i < mine && i < S::stages; ++i) fetch(i);
    // q, rotated, as value and remainder
    for (int i = threadIdx.x; i < ROWS * C; i += kThreads) {
        const int r = i / C, c = i % C;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r < a.rows && c * 8 < a.hd) {
            const int m = r / a.group, g = r - m * a.group;
            turned(q + (p.b * a.M + m) * a.qs + ((int64_t)p.kv * a.group + g) * a.hd, c * 8, turn[m], a.rot, a.half, x);
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = pack2(x[2 * e], x[2 * e + 1]);
            lo[e] = pack2(x[2 * e] - __uint_as_float(hi[e] << 16), x[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
        *reinterpret_cast<uint4*>(sq + r * kPitch + c * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sq + (ROWS + r) * kPitch + c * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __syncthreads();
    uint32_t qh[HD / 32][4], ql[HD / 32][4];                     // B operands of two steps of 16 channels each
#pragma unroll
    for (int c = 0; c < HD / 32; ++c) {
        const uint32_t at = smem_at(sq) + (lane & 7) * kPitch + (4 * c + (lane >> 3)) * 16;
        ldsm4(qh[c], at);
        ldsm4(ql[c], at + ROWS * kPitch);
    }
    float acc[HD / 16][4], mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < HD / 16; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
    const float cs = a.scale * kLog2e;
    // Rows r0, r0 + 1 and tokens lane / 4 (values 0, 1) and lane / 4 + 8 (2, 3) of a slice are this thread's.
    const int r0 = 2 * (lane & 3);
    auto chunk = [](int row, int c) { return (uint32_t)(c / 8) * Dec8Smem<HD>::atom + tc::sw128_off(row, c % 8); };
    // One slice; hidden: a bit per value of this thread that its row does not see.
    auto slice = [&](const uint8_t* at, uint32_t hidden) {
        const uint32_t kt = smem_at(at), vt = kt + S::half;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) {
            uint32_t x[4];
            ldsm4(x, kt + chunk(lane & 15, 2 * c + (lane >> 4)));
            mma16816(s, x, qh[c / 2][2 * (c & 1)], qh[c / 2][2 * (c & 1) + 1]);
            if (a.rot) mma16816(t, x, ql[c / 2][2 * (c & 1)], ql[c / 2][2 * (c & 1) + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = hidden >> e & 1 ? -INFINITY : s[e] + t[e];
        float p2[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float top = fmaxf(s[h], s[2 + h]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            const float now = fmaxf(mx[h], top * cs), use = now == -INFINITY ? 0.f : now;
            const float corr = exp2f(mx[h] - use);
            mx[h] = now;
            p2[h] = exp2f(fmaf(s[h], cs, -use));
            p2[2 + h] = exp2f(fmaf(s[2 + h], cs, -use));
            sum[h] = sum[h] * corr + (p2[h] + p2[2 + h]);
            if (corr != 1.f) {
#pragma unroll
                for (int n = 0; n < HD / 16; ++n) {
                    acc[n][h] *= corr;
                    acc[n][2 + h] *= corr;
                }
            }
        }
        const uint32_t b0 = transposed(pack2(p2[0], p2[1])), b1 = transposed(pack2(p2[2], p2[3]));
#pragma unroll
        for (int n = 0; n < HD / 16; ++n) {
            uint32_t x[4];
            ldsm4t(x, vt + chunk((lane & 7) + ((lane >> 4) << 3), 2 * n + ((lane >> 3) & 1)));
            mma16816(acc[n], x, b0, b1);
        }
    };
    bool ok = true;
    int done = 0;
    for (; done < mine; ++done) {
        uint8_t* at = own + done % S::stages * 2 * S::half;
        ok = tc::mbar_wait(&full[warp][done % S::stages], (done / S::stages) & 1, &abort_flag, a.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const int64_t left = p.to - p.from - (int64_t)(warp + 4 * done) * kSlice;     // cached rows of the slice
        uint32_t hidden = 0;
        if (left < kSlice) {
            // rows behind the cached ones: scores masked, values zero (they may hold anything)
            if ((lane >> 2) >= left) hidden |= 3u;
            if ((lane >> 2) + 8 >= left) hidden |= 12u;
            for (int i = lane; i < (kSlice - (int)left) * C; i += 32)
                *reinterpret_cast<uint4*>(at + S::half + chunk((int)left + i / C, i % C)) = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        slice(at, hidden);
        __syncwarp();
        if (lane == 0 && done + S::stages < mine) fetch(done + S::stages);
    }
    if (!ok && lane == 0)                                        // no copy may land after the block has gone
        for (int i = done; i < mine && i < done + S::stages; ++i)
            tc::mbar_wait_drain(&full[warp][i % S::stages], (i / S::stages) & 1);
    // ---- the drafted tokens: a slice of the last warp (its ring is empty)
    if (p.tail && warp == 3 && ok) {
        bool bad = false;
        for (int i = lane; i < kSlice * C; i += 32) {
            const int t = i / C, c = i % C;
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (t < a.M && c * 8 < a.hd) {
                float f[8];
                turned(k + (p.b * a.M + t) * a.ks + (int64_t)p.kv * a.hd, c * 8, turn[t], a.rot, a.half, f);
                x = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                y = __ldg(reinterpret_cast<const uint4*>(v + (p.b * a.M + t) * a.vs + (int64_t)p.kv * a.hd + c * 8));
                *reinterpret_cast<uint4*>(k_cache + (slot + p.len + t) * a.hd + c * 8) = x;
                *reinterpret_cast<uint4*>(v_cache + (slot + p.len + t) * a.hd + c * 8) = y;
                // infinities and NaN stay out of the product (0 x NaN) and are added to the rows that see them
                uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t odd = attn_tc::nonfinite_bits(w[e]);
                    bad = bad || odd;
                    w[e] &= ~((odd & 0x8000u ? 0xFFFFu : 0u) | (odd & 0x80000000u ? 0xFFFF0000u : 0u));
                }
            }
            *reinterpret_cast<uint4*>(own + chunk(t, c)) = x;
            *reinterpret_cast<uint4*>(own + S::half + chunk(t, c)) = y;
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        uint64_t see[2];
        uint32_t hidden = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            see[h] = r0 + h < a.rows ? seen[(r0 + h) / a.group] : 0;
            if (!(see[h] >> (lane >> 2) & 1)) hidden |= 1u << h;
            if (!(see[h] >> ((lane >> 2) + 8) & 1)) hidden |= 4u << h;
            if (p.len == 0 && see[h] == 0) mx[h] = 0.f, sum[h] = 1.f;    // as sees_nothing says
        }
        slice(own, hidden);
        if (bad)
            for (int j = 0; j < a.M; ++j)
#pragma unroll
                for (int n = 0; n < HD / 16; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int d = 16 * n + (lane >> 2) + 8 * (e >> 1);
                        if (d < a.hd && (see[e & 1] >> j & 1)) {
                            const float x = __bfloat162float(v[(p.b * a.M + j) * a.vs + (int64_t)p.kv * a.hd + d]);
                            if (!(fabsf(x) < INFINITY)) acc[n][e] += x;
                        }
                    }
    }
    __syncthreads();
    float* so = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[h] += __shfl_xor_sync(0xFFFFFFFFu, sum[h], x);
        const int r = warp * ROWS + r0 + h;
        if (lane < 4) {
            smax[r] = mx[h];
            ssum[r] = sum[h];
        }
#pragma unroll
        for (int n = 0; n < HD / 16; ++n) {
            so[r * HD + 16 * n + (lane >> 2)] = acc[n][h];
            so[r * HD + 16 * n + (lane >> 2) + 8] = acc[n][2 + h];
        }
    }
    __syncthreads();
    finish<__nv_bfloat16, HD, ROWS, 4>(a, p, so, smax, ssum, so + 4 * ROWS * HD, o);
}

// ---------------------------------------------------------------- fp32
constexpr int kTokF = 32;

// Four rows per warp; TW warps share the tokens of a tile where the rows do not fill the block (64 x 3000 cached rows,
// 16 heads of 128 over 4, one token: 345 us where one warp of four worked, 173 with TW = 4).  The probabilities go
// to the value loop through shared memory, four rows in a load: 154 us, with shuffles and a test per row 173.
template <int HD, int TW>
__global__ void __launch_bounds__(kThreads) attn_decode_f32_kernel(const float* __restrict__ q,
                                                                   const float* __restrict__ k,
                                                                   const float* __restrict__ v, float* k_cache,
                                                                   float* v_cache, float* __restrict__ o,
                                                                   const DecArgs a) {
    constexpr int C = HD / 4, E = HD / 32;                       // 16-byte chunks per row; channels per lane
    constexpr int ROWS = TW == 1 ? 16 : 8, NT = kTokF / TW;      // rows of a block; tokens of a warp per tile
    constexpr uint32_t kHalf = kTokF * HD * 4;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ __align__(16) float sq[ROWS][HD];
    __shared__ float4 sp[kThreads / 32][NT];                     // a tile's probabilities
    __shared__ float smax[TW * ROWS], ssum[TW * ROWS];
    __shared__ uint64_t seen[64];
    __shared__ const float* turn[64];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tw = TW == 1 ? 0 : warp % TW, r0 = warp / TW * 4;  // a warp's share of the tokens; its rows
    // scores: a lane's token, its part of the channels
    const int tok = TW == 1 ? lane : tw * NT + lane % NT, part = TW == 1 ? 0 : lane / NT;
    Place p = place_of<ROWS>(a, kTokF);
    const int64_t slot = (p.b * a.kvh + p.kv) * a.max_len;
    const uint32_t ring = smem_at(sm);
    const int tiles = (int)((p.to - p.from + kTokF - 1) / kTokF);
    auto place = [](int r, int c) { return (uint32_t)(r * HD * 4 + ((c ^ (r & 7)) << 4)); };
    auto fetch = [&](int t) {
        if (t < tiles) {
            const int64_t r0 = p.from + (int64_t)t * kTokF;
            const uint32_t at = ring + (t % kStages) * 2 * kHalf;
            for (int i = threadIdx.x; i < kTokF * C; i += kThreads) {
                const int r = i / C, c = i % C;
                const bool real = r0 + r < p.to && c * 4 < a.hd;
                const int64_t src = (slot + (real ? r0 + r : 0)) * a.hd + (real ? c * 4 : 0);
                copy16(at + place(r, c), k_cache + src, real);
                copy16(at + kHalf + place(r, c), v_cache + src, real);
            }
        }
        copies_close();
    };
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) fetch(t);
    if (!p.idle && !look_up(a, p, seen, turn)) {
        p.idle = true;
        if (threadIdx.x == 0) atomicOr(a.err, kErrRopePos);
    }
    if (p.idle) {
        copies_wait<0>();
        zero_rows<float, ROWS>(a, p, o);
        return;
    }
#pragma unroll 4
    for (int i = threadIdx.x; i < ROWS * C; i += kThreads) {
        const int r = i / C, c = i % C, row = p.tile * ROWS + r;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (row < a.rows && c * 4 < a.hd) {
            const int m = row / a.group, g = row - m * a.group;
            turned(q + (p.b * a.M + m) * a.qs + ((int64_t)p.kv * a.group + g) * a.hd, c * 4, turn[m], a.rot, a.half, x);
        }
        *reinterpret_cast<float4*>(&sq[r][c * 4]) = make_float4(x[0], x[1], x[2], x[3]);
    }
    __syncthreads();
    float acc[4][E], mx[4], sum[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        mx[r] = -INFINITY;
        sum[r] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = 0.f;
    }
    const float cs = a.scale * kLog2e;
    const int rows_left = a.rows - p.tile * ROWS - r0;           // real rows of this warp
    const int drafts = p.tail ? (a.M + kTokF - 1) / kTokF : 0;
    for (int t = 0; t < tiles + drafts; ++t) {
        const bool draft = t >= tiles;
        const int d0 = draft ? (t - tiles) * kTokF : 0;          // first drafted token of the tile
        uint8_t* tile = sm + (t % kStages) * 2 * kHalf;
        if (!draft) {
            fetch(t + kStages - 1);
            copies_wait<kStages - 1>();
            __syncthreads();
        } else {
            copies_wait<0>();
            __syncthreads();
            const bool write = p.tile == 0;
#pragma unroll 4
            for (int i = threadIdx.x; i < kTokF * C; i += kThreads) {
                const int r = i / C, c = i % C, m = d0 + r;
                float x[4] = {0.f, 0.f, 0.f, 0.f};
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (m < a.M && c * 4 < a.hd) {
                    turned(k + (p.b * a.M + m) * a.ks + (int64_t)p.kv * a.hd, c * 4, turn[m], a.rot, a.half, x);
                    y = __ldg(reinterpret_cast<const float4*>(v + (p.b * a.M + m) * a.vs + (int64_t)p.kv * a.hd + c * 4));
                    if (write) {
                        *reinterpret_cast<float4*>(k_cache + (slot + p.len + m) * a.hd + c * 4) = make_float4(x[0], x[1], x[2], x[3]);
                        *reinterpret_cast<float4*>(v_cache + (slot + p.len + m) * a.hd + c * 4) = y;
                    }
                }
                *reinterpret_cast<float4*>(tile + place(r, c)) = make_float4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<float4*>(tile + kHalf + place(r, c)) = y;
            }
            __syncthreads();
        }
        const int left = (int)min((int64_t)kTokF, draft ? (int64_t)(a.M - d0) : p.to - p.from - (int64_t)t * kTokF);
        if (rows_left > 0) {
            // scores: TW lanes per token, four rows
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int c = part; c < C; c += TW) {
                const float4 x = *reinterpret_cast<const float4*>(tile + place(tok, c));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 y = *reinterpret_cast<const float4*>(&sq[r0 + r][4 * c]);
                    s[r] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[r]))));
                }
            }
            uint32_t see[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int x = NT; x < 32; x <<= 1) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], x);
                const int row = min(p.tile * ROWS + r0 + r, a.rows - 1);
                const bool mine = tok < left && (!draft || (seen[row / a.group] >> (d0 + tok) & 1));
                see[r] = __ballot_sync(0xFFFFFFFFu, mine);
                float top = mine ? s[r] * cs : -INFINITY;
#pragma unroll
                for (int x = NT / 2; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                const float now = fmaxf(mx[r], top), use = now == -INFINITY ? 0.f : now;
                const float corr = exp2f(mx[r] - use);
                mx[r] = now;
                s[r] = mine ? exp2f(fmaf(s[r], cs, -use)) : 0.f;
                sum[r] = sum[r] * corr + s[r];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[r][e] *= corr;
            }
            // values: a lane per E channels; a masked token's value is not touched
            if (part == 0) sp[warp][lane % NT] = make_float4(s[0], s[1], s[2], s[3]);
            __syncwarp();
            const int count = min(NT, left - tw * NT), ch = lane * E;
            auto values = [&](auto with_mask) {
#pragma unroll 8
                for (int n = 0; n < count; ++n) {
                    const float* row = reinterpret_cast<const float*>(tile + kHalf + place(tw * NT + n, ch / 4)) + ch % 4;
                    const float4 w4 = sp[warp][n];
                    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
                    float x[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = row[e];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (!decltype(with_mask)::value || (see[r] >> n & 1))
#pragma unroll
                            for (int e = 0; e < E; ++e) acc[r][e] = fmaf(w[r], x[e], acc[r][e]);
                }
            };
            if (draft) values(std::true_type{});
            else values(std::false_type{});
            __syncwarp();                                        // the probabilities are read
        }
        __syncthreads();
    }
    copies_wait<0>();
    __syncthreads();
    float* so = reinterpret_cast<float*>(sm);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int x = NT / 2; x; x >>= 1) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], x);
        if (lane == 0) {
            const bool none = sees_nothing(a, p, seen, p.tile * ROWS + r0 + r);
            smax[tw * ROWS + r0 + r] = none ? 0.f : mx[r];
            ssum[tw * ROWS + r0 + r] = none ? 1.f : sum[r];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) so[(tw * ROWS + r0 + r) * HD + lane * E + e] = acc[r][e];
    }
    __syncthreads();
    finish<float, HD, ROWS, TW>(a, p, so, smax, ssum, so + TW * ROWS * HD, o);
}

// Rows a block takes: 8, 16 or 32 where they are all there are (its warps then share out the tokens), else the 128 of
// the tcgen05 kernel; fp32: 8 or 16.
int tile_rows(const DecodeProb& p) {
    const int64_t rows = (int64_t)p.M * p.group;
    if (p.dtype == 0) return rows <= 8 ? 8 : 16;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : kTcTile;
}

template <typename T, typename F>
cudaError_t launch(std::atomic<uint64_t>& limit, F* f, size_t smem, unsigned grid, const void* q, const void* k,
                   const void* v, void* kc, void* vc, void* o, const DecArgs& a, cudaStream_t st) {
    cudaError_t e = smem_limit(limit, reinterpret_cast<const void*>(f), smem);
    if (e != cudaSuccess) return e;
    DC_LAUNCH(kAttnDecode, st, f<<<grid, kThreads, smem, st>>>(static_cast<const T*>(q), static_cast<const T*>(k),
                                                               static_cast<const T*>(v), static_cast<T*>(kc),
                                                               static_cast<T*>(vc), static_cast<T*>(o), a));
    return cudaGetLastError();
}
template <int HD, int TW>
cudaError_t launch_tw(unsigned grid, const void* q, const void* k, const void* v, void* kc, void* vc, void* o,
                       const DecArgs& a, cudaStream_t st) {
    static std::atomic<uint64_t> limit{0};
    return launch<float>(limit, attn_decode_f32_kernel<HD, TW>, kStages * 2 * kTokF * HD * 4, grid, q, k, v, kc, vc, o, a, st);
}
template <int HD>
cudaError_t launch_f32(unsigned grid, const void* q, const void* k, const void* v, void* kc, void* vc, void* o,
                       const DecArgs& a, cudaStream_t st) {
    return a.rows <= 4   ? launch_tw<HD, 4>(grid, q, k, v, kc, vc, o, a, st)
           : a.rows <= 8 ? launch_tw<HD, 2>(grid, q, k, v, kc, vc, o, a, st)
                         : launch_tw<HD, 1>(grid, q, k, v, kc, vc, o, a, st);
}
template <int HD>
cudaError_t launch_8(const DecodeProb& p, unsigned grid, const void* q, const void* k, const void* v, void* kc, void* vc,
                     void* o, const DecArgs& a, cudaStream_t st) {
    using B = __nv_bfloat16;
    CUtensorMap tk, tv;
    if (!make_cache_map(&tk, kc, p, kSlice) || !make_cache_map(&tv, vc, p, kSlice)) return cudaErrorInvalidValue;
    constexpr uint32_t smem = Dec8Smem<HD>::bytes;
    cudaError_t e = DC_SMEM_LIMIT(attn_decode8_kernel<HD>, smem);
    if (e != cudaSuccess) return e;
    DC_LAUNCH(kAttnDecode, st, attn_decode8_kernel<HD><<<grid, kThreads, smem, st>>>(
                                   tk, tv, static_cast<const B*>(q), static_cast<const B*>(k), static_cast<const B*>(v),
                                   static_cast<B*>(kc), static_cast<B*>(vc), static_cast<B*>(o), a));
    return cudaGetLastError();
}
template <int HD, int RW>
cudaError_t launch_bf16(unsigned grid, const void* q, const void* k, const void* v, void* kc, void* vc, void* o,
                        const DecArgs& a, cudaStream_t st) {
    static std::atomic<uint64_t> limit{0};
    return launch<__nv_bfloat16>(limit, attn_decode_kernel<HD, RW>, DecSmem<HD>::bytes, grid, q, k, v, kc, vc, o, a, st);
}

}  // namespace

int64_t attn_decode_groups(const DecodeProb& p) {
    const int rows = tile_rows(p);
    return p.batch * p.kvh * (((int64_t)p.M * p.group + rows - 1) / rows);
}

// Runs the cache is split into: as many as keep all blocks on the GPU at once (two per SM; one of the tcgen05
// kernel, whose runs are the blocks of a cluster: 1, 2, 4 or 8), but none of a full cache shorter than a few tiles.
// Measured: one sequence of 12 heads over ~700 rows takes 8.3 us with runs of at least 128 rows, 8.9 with 256, 10.7
// with 64; 64 sequences x 4 heads over ~3000 rows 73 us with 1 or 2 runs, 75 with 3, 80 with 6.
int attn_decode_splits(const DecodeProb& p) {
    const int64_t groups = std::max<int64_t>(1, attn_decode_groups(p));
    const bool tc = tile_rows(p) == kTcTile;
    const int64_t shortest = tc ? 2 * kTcTile : p.dtype == 0 ? 4 * kTokF : tile_rows(p) == 8 ? 8 * kSlice : 4 * kTok;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>({(tc ? 148 : 2 * 148) / groups, (p.max_len + shortest - 1) / shortest, 64}));
    if (!tc) return (int)most;
    int ranks = 1;
    while (ranks < 8 && ranks * 2 <= most) ranks *= 2;
    return ranks;
}

size_t attn_decode_part_bytes(const DecodeProb& p) {
    const int n = attn_decode_splits(p), hd = p.hd <= 64 ? 64 : 128;
    return n == 1 || tile_rows(p) == kTcTile ? 0 : (size_t)attn_decode_groups(p) * n * tile_rows(p) * (hd + 2) * sizeof(float);
}

cudaError_t attn_decode(const DecodeProb& p, const void* q, const void* k, const void* v, void* kc, void* vc,
                        const int32_t* lens, const uint64_t* tree, void* o, uint32_t* err, uint32_t* count, float* part,
                        cudaStream_t st) {
    DecArgs a{p.M, p.heads, p.kvh, p.group, p.hd, p.M * p.group, attn_decode_splits(p), p.max_len, p.qs, p.ks, p.vs, p.os,
              p.rot, p.half, p.max_pos, p.cs, lens, tree, p.scale, part, count, err};
    const unsigned grid = (unsigned)(attn_decode_groups(p) * a.n_split);
    if (p.dtype == 0)
        return p.hd <= 64 ? launch_f32<64>(grid, q, k, v, kc, vc, o, a, st) : launch_f32<128>(grid, q, k, v, kc, vc, o, a, st);
    const int rows = tile_rows(p);
    if (rows == kTcTile) return attn_decode_tc(p, a, grid, q, k, v, kc, vc, o, st);
    if (rows == 8)
        return p.hd <= 64 ? launch_8<64>(p, grid, q, k, v, kc, vc, o, a, st) : launch_8<128>(p, grid, q, k, v, kc, vc, o, a, st);
    if (p.hd <= 64)
        return rows == 16 ? launch_bf16<64, 1>(grid, q, k, v, kc, vc, o, a, st) : launch_bf16<64, 2>(grid, q, k, v, kc, vc, o, a, st);
    return rows == 16 ? launch_bf16<128, 1>(grid, q, k, v, kc, vc, o, a, st) : launch_bf16<128, 2>(grid, q, k, v, kc, vc, o, a, st);
}

}  // namespace dynconv
