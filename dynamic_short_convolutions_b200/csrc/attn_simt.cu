// attn_simt.cu -- causal attention on the CUDA cores, forward and backward: fp32 storage (never
// rounded to a tensor-core input type) and the bf16 shapes the tensor-core kernels do not take.
//
//   o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i.k_j - lse_i),  s(i) <= j <= i
//   dp_ij = do_i.v_j,  ds_ij = p_ij (dp_ij - D_i),  D_i = do_i.o_i
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij do_i
//
// A block takes 64 query rows (forward, dq) or 64 keys (dk, dv) of one head and walks the 64-row
// tiles of the other side; tiles follow the packed token index, so documents need no list of
// work: a row's first visible key is its document's start, and only the tiles that a diagonal or a
// document start crosses are masked.  256 threads each hold a 4 x 4 block of the 64 x 64 scores
// (rows 4 ty + i, columns tx + 16 j) and 4 rows x HD / 16 channels of the accumulators; operands
// are fp32 in shared memory, rows padded to HD + 4 floats so that the 16 column rows of a warp's
// 16-byte loads fall in different banks.  Products of scores run as packed FMAs (two channels each).
//
// Measured (fp32, 5 documents of about 550, 8 heads of 64 over 2): forward 100 us, dk and dv 174, dq 121.  A pair of tiles
// takes a multiprocessor 5.2 us in the forward where its FMAs alone would take 2.15 (pipe 0.49 busy, shared memory
// 0.71, issue 0.57): four warps per scheduler do not cover the latency of the loads.  Lanes as 4 x 8 instead of 2 x 16
// of the grid, which halves the distinct rows a warp reads, changed nothing; two blocks of dk and dv per
// multiprocessor at 128 registers neither.
//
// The backward takes p again from the lse, which the forward rounded to fp32, and D from the o it rounded: two roundings
// more than a form that keeps p.  They show where a row sees few keys and dp - D cancels: dq of documents of 2 tokens is
// off by 4.4e-7 rel-L2 (a plain fp32 form 1.9e-7), of 8 by 2.8e-7 (1.4e-7), of 64 by 2.7e-7 (2.4e-7).
//
// Masked places: the score is replaced before the maximum, and in masked tiles a product with a
// masked probability is not added at all (0 x NaN would be NaN).
#include <cooperative_groups.h>

#include <algorithm>

#include "attn.h"
#include "attn_places.cuh"
#include "common.cuh"
#include "prof.h"
#include "smem_limit.h"
#include "tmap.h"

namespace dynconv {
namespace {

namespace cg = cooperative_groups;

constexpr int kTile = kSimtTile;
constexpr int kThreads = 256;
constexpr int kLdP = kTile + 4;

template <int HD>
constexpr int ld_of() { return HD + 4; }
// Stages of the forward's and dq's ring: two where two blocks still fit an SM.
template <int HD>
constexpr int stages_of() { return HD == 64 ? 2 : 1; }

struct SimtArgs {
    int32_t N, seqlen;
    int heads, kvh, group, hd;
    int64_t qs, ks, vs, os, dos, dqs, dks, dvs;
    float scale;
    const int2* seg;
    const int32_t *order_q, *order_k;
};

// rows row0 .. row0 + 63 of one head (channels hd, zero beyond hd and beyond N) into fp32 shared memory
template <typename T, int HD>
__device__ __forceinline__ void load_tile(float* dst, const T* __restrict__ src, int64_t stride, int32_t row0, int32_t N,
                                          int hd, bool vec) {
    constexpr int LD = ld_of<HD>();
    if (vec) {
        for (int i = threadIdx.x; i < kTile * (HD / 4); i += kThreads) {
            const int r = i / (HD / 4), c = (i % (HD / 4)) * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row0 + r < N && c < hd) {
                const T* p = src + (int64_t)(row0 + r) * stride + c;
                if (sizeof(T) == 4) {
                    f = *reinterpret_cast<const float4*>(p);
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(p);
                    f = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                                    __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
                }
            }
            *reinterpret_cast<float4*>(dst + r * LD + c) = f;
        }
    } else {
        for (int i = threadIdx.x; i < kTile * HD; i += kThreads) {
            const int r = i / HD, c = i % HD;
            dst[r * LD + c] = row0 + r < N && c < hd ? to_f32(src[(int64_t)(row0 + r) * stride + c]) : 0.f;
        }
    }
}

__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// load_tile, fp32 rows on 16-byte boundaries as asynchronous copies (complete after copies_wait and a barrier).
template <typename T, int HD>
__device__ __forceinline__ void fetch_tile(float* dst, const T* __restrict__ src, int64_t stride, int32_t row0, int32_t N,
                                           int hd, bool vec) {
    if (sizeof(T) != 4 || !vec) {
        load_tile<T, HD>(dst, src, stride, row0, N, hd, vec);
        return;
    }
    constexpr int LD = ld_of<HD>();
#pragma unroll
    for (int i = threadIdx.x; i < kTile * (HD / 4); i += kThreads) {
        const int r = i / (HD / 4), c = (i % (HD / 4)) * 4;
        const bool real = row0 + r < N && c < hd;
        const T* p = src + (real ? (int64_t)(row0 + r) * stride + c : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst + r * LD + c)),
                     "l"(p), "r"(real ? 16 : 0)
                     : "memory");
    }
}

// Two fp32 lanes at once: d += a * b, each lane one fused multiply-add (the packed fp32 FMA of sm_100).
__device__ __forceinline__ void pair_fma(uint64_t& d, uint64_t a, uint64_t b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// acc[i][j] = A[4 ty + i] . B[tx + 16 j] over HD channels; even and odd channels summed apart (packed FMAs: half the
// instructions of a kernel that the issue rate bounds)
template <int HD>
__device__ __forceinline__ void tile_nt(const float* A, const float* B, float (&acc)[4][4], int ty, int tx) {
    constexpr int LD = ld_of<HD>();
    uint64_t sum[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = 0;
#pragma unroll 4
    for (int c = 0; c < HD; c += 4) {
        ulonglong2 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(A + (4 * ty + i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * j) * LD + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pair_fma(sum[i][j], a[i].x, b[j].x);
                pair_fma(sum[i][j], a[i].y, b[j].y);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(sum[i][j]));
            acc[i][j] = lo + hi;
        }
}

// Whether a tile holds an infinity or a NaN: the block's answer (a barrier).  A masked place has probability 0, so
// without them the plain products serve masked tiles too; with them tile_nn leaves masked terms out.
template <int HD>
__device__ __forceinline__ bool tile_odd(const float* X, bool ask) {
    constexpr int LD = ld_of<HD>();
    bool odd = false;
    if (ask)
        for (int i = threadIdx.x; i < kTile * (HD / 4); i += kThreads) {
            const float4 f = *reinterpret_cast<const float4*>(X + i / (HD / 4) * LD + i % (HD / 4) * 4);
            odd = odd || !(fabsf(f.x) < INFINITY && fabsf(f.y) < INFINITY && fabsf(f.z) < INFINITY && fabsf(f.w) < INFINITY);
        }
    return __syncthreads_or(odd) != 0;
}

// acc[i][4 jj + e] += sum_c P[4 ty + i][c] X[c][4 tx + 64 jj + e]; with MASK only over c in [lo_i, hi_i]
template <int HD, bool MASK>
__device__ __forceinline__ void tile_nn(const float* P, const float* X, float (&acc)[4][HD / 16], int ty, int tx,
                                        const int (&lo)[4], const int (&hi)[4]) {
    constexpr int LD = ld_of<HD>();
    constexpr int NJ = HD / 64;
#pragma unroll 2
    for (int c = 0; c < kTile; c += 4) {
        float p[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(P + (4 * ty + i) * kLdP + c);
            p[i][0] = f.x; p[i][1] = f.y; p[i][2] = f.z; p[i][3] = f.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int jj = 0; jj < NJ; ++jj) {
                const float4 x = *reinterpret_cast<const float4*>(X + (c + e) * LD + 4 * tx + 64 * jj);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (MASK && (c + e < lo[i] || c + e > hi[i])) continue;
                    acc[i][4 * jj + 0] = fmaf(p[i][e], x.x, acc[i][4 * jj + 0]);
                    acc[i][4 * jj + 1] = fmaf(p[i][e], x.y, acc[i][4 * jj + 1]);
                    acc[i][4 * jj + 2] = fmaf(p[i][e], x.z, acc[i][4 * jj + 2]);
                    acc[i][4 * jj + 3] = fmaf(p[i][e], x.w, acc[i][4 * jj + 3]);
                }
            }
    }
}

// reductions over the 16 lanes (tx) of a row
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// A thread's part of an accumulator row into shared memory.
template <int HD>
__device__ __forceinline__ void put_row(float* row, const float (&acc)[HD / 16], int tx) {
#pragma unroll
    for (int jj = 0; jj < HD / 64; ++jj)
        *reinterpret_cast<float4*>(row + 4 * tx + 64 * jj) =
            make_float4(acc[4 * jj], acc[4 * jj + 1], acc[4 * jj + 2], acc[4 * jj + 3]);
}

template <typename T, int HD>
__device__ __forceinline__ void store_rows(T* dst, int64_t stride, int32_t row0, int32_t N, int hd,
                                           const float (&acc)[4][HD / 16], const float (&mul)[4], int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t n = row0 + 4 * ty + i;
        if (n >= N) continue;
        T* p = dst + (int64_t)n * stride;
#pragma unroll
        for (int jj = 0; jj < HD / 64; ++jj)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = 4 * tx + 64 * jj + e;
                if (c < hd) p[c] = from_f32<T>(acc[i][4 * jj + e] * mul[i]);
            }
    }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) attn_fwd_simt_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                                 const T* __restrict__ v, T* __restrict__ o,
                                                                 float* __restrict__ lse, SimtArgs a, int vec) {
    constexpr int LD = ld_of<HD>(), NS = stages_of<HD>();
    extern __shared__ float sm[];
    float* sQ = sm;
    float* ring = sQ + kTile * LD;         // stage s: K at ring + 2 s tiles, V behind it
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int head = (int)(blockIdx.x / ranks) % a.heads, kv = head / a.group;
    const int32_t tiles = (a.N + kTile - 1) / kTile;
    const int32_t row0 = tile_of((int32_t)(blockIdx.x / ranks / a.heads), tiles, a.seqlen % kTile ? 0 : a.seqlen / kTile,
                                 a.order_q, false) * kTile;
    q += (int64_t)head * a.hd;
    o += (int64_t)head * a.hd;
    k += (int64_t)kv * a.hd;
    v += (int64_t)kv * a.hd;
    load_tile<T, HD>(sQ, q, a.qs, row0, a.N, a.hd, vec);
    const int32_t last = min(row0 + kTile, a.N) - 1;
    const int32_t first_key = doc_of(row0, a.seg, a.seqlen).x;
    const int32_t full_from = doc_of(last, a.seg, a.seqlen).x;
    int32_t start[4];
    float m[4], l[4], acc[4][HD / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        start[i] = doc_of(min(row0 + 4 * ty + i, a.N - 1), a.seg, a.seqlen).x;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) acc[i][c] = 0.f;
    }
    const float cs = a.scale * kLog2e;
    auto fetch = [&](int32_t k0, int at) {
        if (k0 <= last) {
            fetch_tile<T, HD>(ring + 2 * at * kTile * LD, k, a.ks, k0, a.N, a.hd, vec);
            fetch_tile<T, HD>(ring + (2 * at + 1) * kTile * LD, v, a.vs, k0, a.N, a.hd, vec);
        }
        copies_close();
    };
    // this block's tiles of keys: every ranks-th
    const int32_t k_first = (first_key / kTile + rank) * kTile, step = ranks * kTile;
    if (NS == 2) fetch(k_first, 0);
    int at = 0;
    for (int32_t k0 = k_first; k0 <= last; k0 += step, at ^= NS - 1) {
        __syncthreads();                   // the stage fetched into now is read
        fetch(NS == 2 ? k0 + step : k0, NS == 2 ? at ^ 1 : 0);
        copies_wait<NS - 1>();
        __syncthreads();
        const float* sK = ring + 2 * at * kTile * LD;
        const float* sV = sK + kTile * LD;
        float* sP = ring + 2 * at * kTile * LD;      // the keys are read before the probabilities are written
        float s[4][4];
        tile_nt<HD>(sQ, sK, s, ty, tx);
        const bool masked = k0 + kTile - 1 > row0 || k0 < full_from;
        int lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = start[i] - k0;
            hi[i] = row0 + 4 * ty + i - k0;
            float mx = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j;
                if (masked && (c < lo[i] || c > hi[i])) s[i][j] = -INFINITY;
                mx = fmaxf(mx, s[i][j] * cs);
            }
            mx = row_max(mx);
            const float use = mx == -INFINITY ? 0.f : mx;     // a row that has seen no key yet
            const float corr = exp2f(m[i] - use);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = exp2f(fmaf(s[i][j], cs, -use));
                sum += s[i][j];
            }
            l[i] = l[i] * corr + sum;
            m[i] = mx;
#pragma unroll
            for (int c = 0; c < HD / 16; ++c) acc[i][c] *= corr;
        }
        const bool odd = tile_odd<HD>(sV, masked);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sP[(4 * ty + i) * kLdP + tx + 16 * j] = s[i][j];
        __syncthreads();
        if (odd) tile_nn<HD, true>(sP, sV, acc, ty, tx, lo, hi);
        else tile_nn<HD, false>(sP, sV, acc, ty, tx, lo, hi);
    }
    if (ranks > 1) {
        // partial rows of the cluster's blocks, joined in the order of their ranks, each block a share of the rows
        copies_wait<0>();
        __syncthreads();
        float* stat = sQ + kTile * LD;                       // in the ring: m, then l of a row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            l[i] = row_sum(l[i]);
            put_row<HD>(sQ + (4 * ty + i) * LD, acc[i], tx);
            if (tx == 0) {
                stat[4 * ty + i] = m[i];
                stat[kTile + 4 * ty + i] = l[i];
            }
        }
        cluster.sync();
        const int per = kTile / ranks;
        for (int i = threadIdx.x; i < per * HD; i += kThreads) {
            const int r = rank * per + i / HD, c = i % HD;
            float mx = -INFINITY, sum = 0.f, x = 0.f;
            for (int n = 0; n < ranks; ++n) mx = fmaxf(mx, cluster.map_shared_rank(stat, n)[r]);
            const float use = mx == -INFINITY ? 0.f : mx;
            for (int n = 0; n < ranks; ++n) {
                const float* part = cluster.map_shared_rank(sQ, n);
                const float w = exp2f(part[kTile * LD + r] - use);
                sum = fmaf(w, part[kTile * LD + kTile + r], sum);
                x = fmaf(w, part[r * LD + c], x);
            }
            const int32_t n = row0 + r;
            if (n >= a.N) continue;
            if (c < a.hd) o[(int64_t)n * a.os + c] = from_f32<T>(x * (1.f / sum));
            if (lse != nullptr && c == 0) lse[(int64_t)head * a.N + n] = (mx + log2f(sum)) * kLn2;
        }
        cluster.sync();                    // no block leaves while its part is read
        return;
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        l[i] = row_sum(l[i]);
        inv[i] = 1.f / l[i];               // every row sees its own key; no finite score: 0 / 0
        const int32_t n = row0 + 4 * ty + i;
        if (lse != nullptr && tx == 0 && n < a.N) lse[(int64_t)head * a.N + n] = (m[i] + log2f(l[i])) * kLn2;
    }
    store_rows<T, HD>(o, a.os, row0, a.N, a.hd, acc, inv, ty, tx);
}

// dq of 64 query rows of one head: the tiles of keys walked as in the forward.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) attn_dq_simt_kernel(const T* __restrict__ d_o, const T* __restrict__ q,
                                                                const T* __restrict__ k, const T* __restrict__ v,
                                                                const float* __restrict__ lse,
                                                                const float* __restrict__ delta, T* __restrict__ dq,
                                                                SimtArgs a, int vec) {
    constexpr int LD = ld_of<HD>(), NS = stages_of<HD>();
    extern __shared__ float sm[];
    float* sQ = sm;
    float* sO = sQ + kTile * LD;
    float* ring = sO + kTile * LD;         // stage s: K at ring + 2 s tiles, V behind it
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int head = (int)(blockIdx.x / ranks) % a.heads, kv = head / a.group;
    const int32_t tiles = (a.N + kTile - 1) / kTile;
    const int32_t row0 = tile_of((int32_t)(blockIdx.x / ranks / a.heads), tiles, a.seqlen % kTile ? 0 : a.seqlen / kTile,
                                 a.order_q, false) * kTile;
    load_tile<T, HD>(sQ, q + (int64_t)head * a.hd, a.qs, row0, a.N, a.hd, vec);
    load_tile<T, HD>(sO, d_o + (int64_t)head * a.hd, a.dos, row0, a.N, a.hd, vec);
    k += (int64_t)kv * a.hd;
    v += (int64_t)kv * a.hd;
    const int32_t last = min(row0 + kTile, a.N) - 1;
    const int32_t first_key = doc_of(row0, a.seg, a.seqlen).x;
    const int32_t full_from = doc_of(last, a.seg, a.seqlen).x;
    int32_t start[4];
    float ls[4], dl[4], acc[4][HD / 16], mul[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t n = min(row0 + 4 * ty + i, a.N - 1);
        start[i] = doc_of(n, a.seg, a.seqlen).x;
        ls[i] = lse[(int64_t)head * a.N + n] * kLog2e;
        dl[i] = delta[(int64_t)head * a.N + n];
        mul[i] = a.scale;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) acc[i][c] = 0.f;
    }
    const float cs = a.scale * kLog2e;
    auto fetch = [&](int32_t k0, int at) {
        if (k0 <= last) {
            fetch_tile<T, HD>(ring + 2 * at * kTile * LD, k, a.ks, k0, a.N, a.hd, vec);
            fetch_tile<T, HD>(ring + (2 * at + 1) * kTile * LD, v, a.vs, k0, a.N, a.hd, vec);
        }
        copies_close();
    };
    // this block's tiles of keys: every ranks-th
    const int32_t k_first = (first_key / kTile + rank) * kTile, step = ranks * kTile;
    if (NS == 2) fetch(k_first, 0);
    int at = 0;
    for (int32_t k0 = k_first; k0 <= last; k0 += step, at ^= NS - 1) {
        __syncthreads();                   // the stage fetched into now is read
        fetch(NS == 2 ? k0 + step : k0, NS == 2 ? at ^ 1 : 0);
        copies_wait<NS - 1>();
        __syncthreads();
        const float* sK = ring + 2 * at * kTile * LD;
        const float* sV = sK + kTile * LD;
        float* sD = ring + (2 * at + 1) * kTile * LD;        // the values are read before ds is written
        float s[4][4], dp[4][4];
        tile_nt<HD>(sQ, sK, s, ty, tx);
        tile_nt<HD>(sO, sV, dp, ty, tx);
        const bool masked = k0 + kTile - 1 > row0 || k0 < full_from;
        int lo[4], hi[4];
        const bool odd = tile_odd<HD>(sK, masked);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = start[i] - k0;
            hi[i] = row0 + 4 * ty + i - k0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j;
                const float p = exp2f(fmaf(s[i][j], cs, -ls[i]));
                const bool hide = masked && (c < lo[i] || c > hi[i]);
                sD[(4 * ty + i) * kLdP + c] = hide ? 0.f : p * (dp[i][j] - dl[i]);
            }
        }
        __syncthreads();
        if (odd) tile_nn<HD, true>(sD, sK, acc, ty, tx, lo, hi);
        else tile_nn<HD, false>(sD, sK, acc, ty, tx, lo, hi);
    }
    dq += (int64_t)head * a.hd;
    if (ranks == 1) {
        store_rows<T, HD>(dq, a.dqs, row0, a.N, a.hd, acc, mul, ty, tx);
        return;
    }
    // partial sums of the cluster's blocks, as in the forward
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) put_row<HD>(sQ + (4 * ty + i) * LD, acc[i], tx);
    cluster.sync();
    const int per = kTile / ranks;
    for (int i = threadIdx.x; i < per * HD; i += kThreads) {
        const int r = rank * per + i / HD, c = i % HD;
        float x = 0.f;
        for (int n = 0; n < ranks; ++n) x += cluster.map_shared_rank(sQ, n)[r * LD + c];
        if (row0 + r < a.N && c < a.hd) dq[(int64_t)(row0 + r) * a.dqs + c] = from_f32<T>(x * a.scale);
    }
    cluster.sync();
}

// dk and dv of 64 keys of one key/value head: every head of the group, every tile of queries that sees
// a key of the tile, in order (no atomics).  Scores are held transposed: rows are keys.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) attn_dkv_simt_kernel(const T* __restrict__ d_o, const T* __restrict__ q,
                                                                 const T* __restrict__ k, const T* __restrict__ v,
                                                                 const float* __restrict__ lse,
                                                                 const float* __restrict__ delta, T* __restrict__ dk,
                                                                 T* __restrict__ dv, SimtArgs a, int vec) {
    constexpr int LD = ld_of<HD>();
    extern __shared__ float sm[];
    float* sK = sm;
    float* sV = sK + kTile * LD;
    float* sQ = sV + kTile * LD;
    float* sO = sQ + kTile * LD;
    float* sP = sO + kTile * LD;
    float* sD = sP + kTile * kLdP;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int kv = (int)(blockIdx.x / ranks) % a.kvh;
    const int32_t row0 = tile_of((int32_t)(blockIdx.x / ranks / a.kvh), (a.N + kTile - 1) / kTile,
                                 a.seqlen % kTile ? 0 : a.seqlen / kTile, a.order_k, true) * kTile;
    fetch_tile<T, HD>(sK, k + (int64_t)kv * a.hd, a.ks, row0, a.N, a.hd, vec);
    fetch_tile<T, HD>(sV, v + (int64_t)kv * a.hd, a.vs, row0, a.N, a.hd, vec);
    const int32_t last = min(row0 + kTile, a.N) - 1;
    const int32_t first_end = doc_of(row0, a.seg, a.seqlen).y;
    const int32_t e_last = doc_of(last, a.seg, a.seqlen).y;               // queries end with the last key's document
    int32_t end[4];
    float acck[4][HD / 16], accv[4][HD / 16], mk[4], mv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        end[i] = doc_of(min(row0 + 4 * ty + i, a.N - 1), a.seg, a.seqlen).y;
        mk[i] = a.scale;
        mv[i] = 1.f;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c) acck[i][c] = accv[i][c] = 0.f;
    }
    const float cs = a.scale * kLog2e;
    // this block's (head, tile of queries) pairs: every ranks-th
    int head = kv * a.group;
    int32_t q0 = row0 + rank * kTile;
    const int32_t rows = (e_last - row0 + kTile - 1) / kTile * kTile;
    auto settle = [&]() {
        while (q0 >= row0 + rows) {
            q0 -= rows;
            ++head;
        }
    };
    for (settle(); head < (kv + 1) * a.group; q0 += ranks * kTile, settle()) {
        __syncthreads();
        fetch_tile<T, HD>(sQ, q + (int64_t)head * a.hd, a.qs, q0, a.N, a.hd, vec);
        fetch_tile<T, HD>(sO, d_o + (int64_t)head * a.hd, a.dos, q0, a.N, a.hd, vec);
        copies_close();
        float ls[4], dl[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int32_t n = min(q0 + tx + 16 * j, a.N - 1);
            ls[j] = lse[(int64_t)head * a.N + n] * kLog2e;
            dl[j] = delta[(int64_t)head * a.N + n];
        }
        copies_wait<0>();
        __syncthreads();
        float s[4][4], dp[4][4];
        tile_nt<HD>(sK, sQ, s, ty, tx);
        tile_nt<HD>(sV, sO, dp, ty, tx);
        const bool masked = q0 < row0 + kTile || q0 + kTile > first_end;
        int lo[4], hi[4];
        bool odd = false;
        if (masked) {
            odd = tile_odd<HD>(sQ, true);
            odd = tile_odd<HD>(sO, true) || odd;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = row0 + 4 * ty + i - q0;
            hi[i] = end[i] - 1 - q0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = tx + 16 * j;
                const float p = exp2f(fmaf(s[i][j], cs, -ls[j]));
                const bool hide = masked && (c < lo[i] || c > hi[i]);
                sP[(4 * ty + i) * kLdP + c] = hide ? 0.f : p;
                sD[(4 * ty + i) * kLdP + c] = hide ? 0.f : p * (dp[i][j] - dl[j]);
            }
        }
        __syncthreads();
        if (odd) {
            tile_nn<HD, true>(sP, sO, accv, ty, tx, lo, hi);
            tile_nn<HD, true>(sD, sQ, acck, ty, tx, lo, hi);
        } else {
            tile_nn<HD, false>(sP, sO, accv, ty, tx, lo, hi);
            tile_nn<HD, false>(sD, sQ, acck, ty, tx, lo, hi);
        }
    }
    dk += (int64_t)kv * a.hd;
    dv += (int64_t)kv * a.hd;
    if (ranks == 1) {
        store_rows<T, HD>(dk, a.dks, row0, a.N, a.hd, acck, mk, ty, tx);
        store_rows<T, HD>(dv, a.dvs, row0, a.N, a.hd, accv, mv, ty, tx);
        return;
    }
    // partial sums of the cluster's blocks, added in the order of their ranks, each block a share of the rows
    copies_close();
    copies_wait<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        put_row<HD>(sQ + (4 * ty + i) * LD, acck[i], tx);
        put_row<HD>(sO + (4 * ty + i) * LD, accv[i], tx);
    }
    cluster.sync();
    const int per = kTile / ranks;
    for (int i = threadIdx.x; i < per * HD; i += kThreads) {
        const int r = rank * per + i / HD, c = i % HD;
        float x = 0.f, y = 0.f;
        for (int n = 0; n < ranks; ++n) {
            x += cluster.map_shared_rank(sQ, n)[r * LD + c];
            y += cluster.map_shared_rank(sO, n)[r * LD + c];
        }
        if (row0 + r < a.N && c < a.hd) {
            dk[(int64_t)(row0 + r) * a.dks + c] = from_f32<T>(x * a.scale);
            dv[(int64_t)(row0 + r) * a.dvs + c] = from_f32<T>(y);
        }
    }
    cluster.sync();                        // no block leaves while its part is read
}

// A warp per (token, head); lanes over the channels.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_delta_kernel(const T* __restrict__ d_o, const T* __restrict__ o,
                                                              int64_t dos, int64_t os, int64_t N, int heads, int hd,
                                                              float* __restrict__ delta) {
    const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    const int64_t n = w / heads;
    if (n >= N) return;
    const int h = (int)(w - n * heads);
    float s = 0.f;
    for (int c = lane; c < hd; c += 32)
        s = fmaf(to_f32(d_o[n * dos + (int64_t)h * hd + c]), to_f32(o[n * os + (int64_t)h * hd + c]), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    if (lane == 0) delta[(int64_t)h * N + n] = s;
}

SimtArgs args_of(const AttnProb& p) {
    return SimtArgs{(int32_t)p.N, (int32_t)p.seqlen, p.heads, p.kvh, p.group, p.hd, p.qs, p.ks, p.vs,
                    p.os, p.dos, p.dqs, p.dks, p.dvs, p.scale, p.seg, p.order_q, p.order_k};
}

// 16-byte (fp32) or 8-byte (bf16) loads of four channels: head starts and rows on such boundaries
int vec_ok(const AttnProb& p, bool bwd) {
    return p.hd % 4 == 0 && p.qs % 4 == 0 && p.ks % 4 == 0 && p.vs % 4 == 0 && (!bwd || p.dos % 4 == 0);
}

// Blocks of a cluster that share the work of one tile: a power of two up to 8, while the grid has fewer blocks than
// `halves` / 2 per multiprocessor: 3 for the forward and dq, two of whose blocks fit a multiprocessor, 1.5 for dk and
// dv, where one does.  Measured (fp32, 64 channels; one block a tile, then by this rule; forward / dk and dv / dq, us):
// one sequence of 1024, 4 heads 93 / 157 / 126, 46 / 65 / 57; of 2048, 4 heads over 2: 178 / 308 / 243, 99 / 177 / 130;
// 5 documents of about 550, 8 over 2: dq 134, 121.  With twice the limit: 116 / 222 / 149 at the second.
int ranks_of(int64_t blocks, int halves) {
    int ranks = 1;
    while (ranks < 8 && 2 * blocks * ranks < halves * num_sms()) ranks *= 2;
    return ranks;
}
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), int64_t blocks, int ranks, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int HD>
cudaError_t fwd_t(const AttnProb& p, const void* q, const void* k, const void* v, void* o, float* lse,
                  cudaStream_t st) {
    constexpr size_t smem = sizeof(float) * (1 + 2 * stages_of<HD>()) * kTile * ld_of<HD>();
    cudaError_t e = DC_SMEM_LIMIT((attn_fwd_simt_kernel<T, HD>), smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (p.N + kTile - 1) / kTile * p.heads;
    DC_LAUNCH(kAttnSimtFwd, st, e = launch(attn_fwd_simt_kernel<T, HD>, blocks, ranks_of(blocks, 6), smem, st,
                                           static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
                                           static_cast<T*>(o), lse, args_of(p), vec_ok(p, false)));
    return e;
}

template <typename T, int HD>
cudaError_t bwd_t(const AttnProb& p, const void* d_o, const void* q, const void* k, const void* v, const float* lse,
                  const float* delta, void* dq, void* dk, void* dv, cudaStream_t st) {
    constexpr size_t smem_q = sizeof(float) * (2 + 2 * stages_of<HD>()) * kTile * ld_of<HD>();
    constexpr size_t smem_kv = sizeof(float) * (4 * kTile * ld_of<HD>() + 2 * kTile * kLdP);
    cudaError_t e = DC_SMEM_LIMIT((attn_dq_simt_kernel<T, HD>), smem_q);
    if (e == cudaSuccess) e = DC_SMEM_LIMIT((attn_dkv_simt_kernel<T, HD>), smem_kv);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (p.N + kTile - 1) / kTile;
    const T *td = static_cast<const T*>(d_o), *tq = static_cast<const T*>(q), *tk = static_cast<const T*>(k),
            *tv = static_cast<const T*>(v);
    DC_LAUNCH(kAttnSimtDkv, st, e = launch(attn_dkv_simt_kernel<T, HD>, tiles * p.kvh, ranks_of(tiles * p.kvh, 3),
                                           smem_kv, st, td, tq, tk, tv, lse, delta, static_cast<T*>(dk),
                                           static_cast<T*>(dv), args_of(p), vec_ok(p, true)));
    if (e != cudaSuccess) return e;
    DC_LAUNCH(kAttnSimtDq, st, e = launch(attn_dq_simt_kernel<T, HD>, tiles * p.heads, ranks_of(tiles * p.heads, 6), smem_q,
                                          st, td, tq, tk, tv, lse, delta, static_cast<T*>(dq), args_of(p),
                                          vec_ok(p, true)));
    return e;
}

}  // namespace

cudaError_t attn_simt_fwd(const AttnProb& p, const void* q, const void* k, const void* v, void* o, float* lse,
                          cudaStream_t st) {
    if (p.dtype == 0)
        return p.hd <= 64 ? fwd_t<float, 64>(p, q, k, v, o, lse, st) : fwd_t<float, 128>(p, q, k, v, o, lse, st);
    return p.hd <= 64 ? fwd_t<__nv_bfloat16, 64>(p, q, k, v, o, lse, st)
                      : fwd_t<__nv_bfloat16, 128>(p, q, k, v, o, lse, st);
}

cudaError_t attn_simt_bwd(const AttnProb& p, const void* d_o, const void* q, const void* k, const void* v,
                          const float* lse, const float* delta, void* dq, void* dk, void* dv, cudaStream_t st) {
    if (p.dtype == 0)
        return p.hd <= 64 ? bwd_t<float, 64>(p, d_o, q, k, v, lse, delta, dq, dk, dv, st)
                          : bwd_t<float, 128>(p, d_o, q, k, v, lse, delta, dq, dk, dv, st);
    return p.hd <= 64 ? bwd_t<__nv_bfloat16, 64>(p, d_o, q, k, v, lse, delta, dq, dk, dv, st)
                      : bwd_t<__nv_bfloat16, 128>(p, d_o, q, k, v, lse, delta, dq, dk, dv, st);
}

cudaError_t attn_delta(const AttnProb& p, const void* d_o, const void* o, float* delta, cudaStream_t st) {
    const int64_t warps = p.N * p.heads;
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    if (p.dtype == 0)
        DC_LAUNCH(kAttnDelta, st, attn_delta_kernel<float><<<grid, kThreads, 0, st>>>(
                                      static_cast<const float*>(d_o), static_cast<const float*>(o), p.dos, p.os, p.N,
                                      p.heads, p.hd, delta));
    else
        DC_LAUNCH(kAttnDelta, st, attn_delta_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(
                                      static_cast<const __nv_bfloat16*>(d_o), static_cast<const __nv_bfloat16*>(o),
                                      p.dos, p.os, p.N, p.heads, p.hd, delta));
    return cudaGetLastError();
}

}  // namespace dynconv
