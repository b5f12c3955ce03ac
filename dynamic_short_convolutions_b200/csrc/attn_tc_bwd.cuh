// attn_tc_bwd.cuh -- what the tensor-core backward kernels of wide and narrow heads share: bf16 remainders, rows
// computed again one by one, the sum of a cluster's partial gradients.
#pragma once

#include <cooperative_groups.h>

#include <algorithm>

#include "attn_tc.cuh"

namespace dynconv {
namespace attn_tc {
namespace {

namespace cg = cooperative_groups;

// What bf16 rounding leaves of 32 values.
__device__ __forceinline__ void remainder32(float (&f)[32]) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const uint32_t w = pack_bf16(f[e], f[e + 1]);
        f[e] -= bf16_lo(w);
        f[e + 1] -= bf16_hi(w);
    }
}
__device__ __forceinline__ void store32(uint32_t to, const float (&f)[32]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
    tmem_st16(to, w);
}
// dk and dv of `count` keys from key0 on (all below N), key by key over the queries that see it.
__device__ __noinline__ void dkv_rows_again(const AttnTcArgs& a, int kv, int32_t key0, int count, int lane) {
    const float cs = a.scale * kLog2e;
    for (int r = 0; r < count; ++r) {
        const int32_t j = key0 + r;
        const int32_t end = doc_of(j, a.seg, a.seqlen).y;
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
        const float ls = a.lse[(int64_t)head * a.N + n] * kLog2e;
        const float dl = warp_dot(d, row4(a.o + (int64_t)n * a.os + (int64_t)head * a.hd, lane, a.hd));
        if (lane == 0) a.delta[(int64_t)head * a.N + n] = dl;
        float4 dq = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int32_t j = doc_of(n, a.seg, a.seqlen).x; j <= n; ++j) {
            const float4 k = row4(a.k + (int64_t)j * a.ks + (int64_t)kv * a.hd, lane, a.hd);
            const float4 v = row4(a.v + (int64_t)j * a.vs + (int64_t)kv * a.hd, lane, a.hd);
            const float p = exp2f(fmaf(warp_dot(q, k), cs, -ls));
            axpy4(dq, p * (warp_dot(d, v) - dl), k);
        }
        put4(a.dq + (int64_t)n * a.dqs + (int64_t)head * a.hd, lane, a.hd,
             make_float4(dq.x * a.scale, dq.y * a.scale, dq.z * a.scale, dq.w * a.scale));
    }
}

// Row `row` of two tiles of 64 channels, as TMA laid them out: the sum of their products.
__device__ __forceinline__ float row_dot(const uint8_t* x, const uint8_t* y, uint32_t row) {
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + sw128_off(row, c));
        const uint4 v = *reinterpret_cast<const uint4*>(y + sw128_off(row, c));
        d0 = fmaf(bf16_lo(u.x), bf16_lo(v.x), d0);
        d1 = fmaf(bf16_hi(u.x), bf16_hi(v.x), d1);
        d0 = fmaf(bf16_lo(u.y), bf16_lo(v.y), d0);
        d1 = fmaf(bf16_hi(u.y), bf16_hi(v.y), d1);
        d0 = fmaf(bf16_lo(u.z), bf16_lo(v.z), d0);
        d1 = fmaf(bf16_hi(u.z), bf16_hi(v.z), d1);
        d0 = fmaf(bf16_lo(u.w), bf16_lo(v.w), d0);
        d1 = fmaf(bf16_hi(u.w), bf16_hi(v.w), d1);
    }
    return d0 + d1;
}

// Row length of a block's partial gradients in shared memory: padded by 16 bytes, so that a lane per row writes
// without bank conflicts.
template <int HD>
constexpr int part_ld() { return HD + 4; }

// The partial gradients of a cluster's blocks (`part`: dv, then dk, [2][128][part_ld] of each block), added in the
// order of the ranks, each block a share of the rows; `again`: a block's 1 (a masked place held an infinity or NaN:
// its rows one by one) or -1 (a wait ran out: nothing is written).  Every thread of every block calls this, whatever
// became of its waits, so the cluster's barriers end.
template <int HD, int THREADS, int WARPS>
__device__ __forceinline__ void join_parts(const AttnTcArgs& a, cg::cluster_group& cluster, int* again, const float* part,
                                           int kv, int32_t key0) {
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    cluster.sync();
    int bad = 0;
    for (int r = 0; r < ranks; ++r) {
        const int f = *cluster.map_shared_rank(again, r);
        bad = f < 0 || bad < 0 ? -1 : bad | f;
    }
    const int per = kRows / ranks, r0 = rank * per;          // the rows this block adds up
    if (bad == 0) {
        for (int i = threadIdx.x; i < 2 * per * (HD / 8); i += THREADS) {
            const int c = i % (HD / 8) * 8, r = i / (HD / 8) % per, w = i / (HD / 8) / per;
            const int32_t j = key0 + r0 + r;
            float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
            for (int n = 0; n < ranks; ++n) {
                const float4* p = reinterpret_cast<const float4*>(
                    cluster.map_shared_rank(part, n) + (size_t)(w * kRows + r0 + r) * part_ld<HD>() + c);
                const float4 u = p[0], v = p[1];
                lo.x += u.x; lo.y += u.y; lo.z += u.z; lo.w += u.w;
                hi.x += v.x; hi.y += v.y; hi.z += v.z; hi.w += v.w;
            }
            if (j >= a.N || c >= a.hd) continue;
            const float m = w ? a.scale : 1.f;
            __nv_bfloat16* to = (w ? a.dk + (int64_t)j * a.dks : a.dv + (int64_t)j * a.dvs) + (int64_t)kv * a.hd + c;
            *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16(lo.x * m, lo.y * m), pack_bf16(lo.z * m, lo.w * m),
                                                       pack_bf16(hi.x * m, hi.y * m), pack_bf16(hi.z * m, hi.w * m));
        }
    } else if (bad > 0 && warp < WARPS) {
        const int32_t n = (per + WARPS - 1) / WARPS, r = key0 + r0 + warp * n;
        dkv_rows_again(a, kv, r, min(min(n, per - warp * n), a.N - r), lane);
    }
    cluster.sync();                                          // no block leaves while its part is read
}

// Blocks that share the heads of a group, a power of two up to 8, while key tiles are few.  Measured at HD = 128:
// 312 tiles of documents of many lengths 205 us with 2, 283 with 1, 301 with 4; 512 equal ones 451 with 1, 503 with 2.
// At 64 channels, two blocks per multiprocessor: 32 tiles, groups of 8: 99 us with 8, 601 with 1; 96, groups of 4: 72
// with 4, 160 with 1; 128: 85 with 4, 97 with 2; 256: 131 with 2, 171 with 1, 153 with 4; 512: 230 with 1, 225 with 2.
inline int dkv_ranks(const AttnProb& p, int64_t blocks) {
    int ranks = 1;
    while (ranks * 2 <= std::min(p.group, 8) && blocks * ranks < 3 * num_sms()) ranks *= 2;
    return ranks;
}
// A launch in clusters of `ranks` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_ranks(void (*kernel)(KArgs...), int ranks, unsigned grid, int threads, size_t smem, cudaStream_t st,
                         Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace

// Tensor maps of a backward call: boxes of 128 tokens, and of 64 for the tiles that narrow heads stream.
struct BwdMaps {
    CUtensorMap q, k, v, d, o, dq, dk, dv, q64, k64, v64, d64;
};
// Head widths up to 64 (attn_tc_bwd64.cu).
cudaError_t bwd_narrow(const AttnProb& p, const BwdMaps& m, const AttnTcArgs& a, cudaStream_t st);

}  // namespace attn_tc
}  // namespace dynconv
