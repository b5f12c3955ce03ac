// attn_prep.cu -- what the attention kernels want to know of packed documents, one launch before them: the check
// of cu_seqlens, every token's document (a load where a binary search of dependent loads took 1-2 us at the
// start of each block), and the tiles in descending order of their work (documents differ in length, and with the
// long tiles last most SMs wait for a few blocks).  7.6 us between events
// around the launch for 9 documents, 9967 tokens, some 5 of them the events' and the launch's own; cu_seqlens in shared
// memory changed nothing.  The order alone took dk and dv of these from 278 to 205 us.
#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "prof.h"

namespace dynconv {
namespace {

constexpr int kThreads = 1024;
constexpr int kBins = kThreads;                  // a thread per bin

// Block 0 checks cu_seqlens and sorts the query tiles, block 1 the key tiles (a counting sort; the order within a
// bin is not fixed and touches no result), the others write the documents of 1024 tokens each.
__global__ void __launch_bounds__(kThreads) attn_prep_kernel(const int32_t* __restrict__ cu, int32_t n_docs, int32_t N,
                                                             int32_t tile, int2* __restrict__ seg,
                                                             int32_t* __restrict__ order, uint32_t* err) {
    if (blockIdx.x >= 2) {
        const int64_t n = (int64_t)(blockIdx.x - 2) * kThreads + threadIdx.x;
        if (n < N) {
            int32_t s, e;
            seg_bounds32((int32_t)n, cu, n_docs, 0, N, s, e);
            seg[n] = make_int2(s, e);
        }
        return;
    }
    const bool keys = blockIdx.x == 1;
    if (!keys) {
        bool bad = false;
        for (int32_t i = threadIdx.x; i < n_docs; i += kThreads) bad = bad || cu[i] > cu[i + 1];
        if (threadIdx.x == 0) bad = bad || cu[0] != 0 || cu[n_docs] != N;
        if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(err, kErrBadSeqlens);
    }
    __shared__ int32_t place[kBins];
    const int32_t tiles = (N - 1) / tile + 1;
    int shift = 0;
    while ((tiles - 1) >> shift >= kBins) ++shift;
    auto bin_of = [&](int32_t t) {           // 0: the most work
        int32_t s, e, work;
        if (keys) {
            seg_bounds32((int32_t)min((int64_t)(t + 1) * tile, (int64_t)N) - 1, cu, n_docs, 0, N, s, e);
            work = (e - 1) / tile - t;       // tiles of queries behind the key tile's own
        } else {
            work = t - seg_start32(t * tile, cu, n_docs, 0) / tile;
        }
        return kBins - 1 - (work >> shift);
    };
    for (int i = threadIdx.x; i < kBins; i += kThreads) place[i] = 0;
    __syncthreads();
    for (int32_t t = threadIdx.x; t < tiles; t += kThreads) atomicAdd(&place[bin_of(t)], 1);
    __syncthreads();
    // exclusive sums of the bins: within warps, then over the warps' sums
    __shared__ int32_t sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t own = place[threadIdx.x];
    int32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int32_t all = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xFFFFFFFFu, all, o);
            if (lane >= o) all += x;
        }
        sums[lane] = all - sums[lane];
    }
    __syncthreads();
    place[threadIdx.x] = sums[warp] + sum - own;
    __syncthreads();
    for (int32_t t = threadIdx.x; t < tiles; t += kThreads) order[(keys ? tiles : 0) + atomicAdd(&place[bin_of(t)], 1)] = t;
}

}  // namespace

cudaError_t attn_prep(const AttnProb& p, int tile, int2* seg, int32_t* order, uint32_t* err, cudaStream_t st) {
    const unsigned grid = 2 + (unsigned)((p.N + kThreads - 1) / kThreads);
    DC_LAUNCH(kAttnPrep, st, attn_prep_kernel<<<grid, kThreads, 0, st>>>(p.cu, (int32_t)p.n_docs, (int32_t)p.N, tile, seg,
                                                                         order, err));
    return cudaGetLastError();
}

}  // namespace dynconv
