// attn_decode.cuh -- what the cache-attention kernels share: arguments, a block's place, the rotation of 16 bytes,
// the drafted tokens' view, and joining the results of the runs a cache is split into.
#pragma once

#include <algorithm>

#include "attn.h"
#include "attn_tc.cuh"
#include "common.cuh"

namespace dynconv {
namespace attn_dec {

constexpr int kThreads = 128;

struct DecArgs {
    int M, heads, kvh, group, hd, rows, n_split;     // rows = M * group
    int64_t max_len, qs, ks, vs, os;
    int rot, half;
    int64_t max_pos;
    const float* cs;
    const int32_t* lens;
    const uint64_t* tree;
    float scale;
    float* part;                                     // per [batch, kvh, row tile]: o [n_split][rows][HD], then maximum and
                                                     // sum [n_split][rows][2]
    uint32_t* count;                                 // [batch, kvh, row tiles]
    uint32_t* err;
};

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes to shared memory; zeros where !real (the address is not read then)
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Which drafted tokens token m sees, as bits, and its depth below the cached tokens.
__device__ __forceinline__ uint64_t seen_by(const DecArgs& a, int64_t b, int m) {
    if (a.tree != nullptr) {
        const uint64_t t = __ldg(reinterpret_cast<const unsigned long long*>(a.tree) + b * a.M + m);
        return a.M < 64 ? t & ((uint64_t(1) << a.M) - 1) : t;
    }
    return m == 63 ? ~uint64_t(0) : (uint64_t(2) << m) - 1;
}
__device__ __forceinline__ int depth_of(uint64_t seen, int m) { return __popcll(seen & ~(uint64_t(1) << m)); }

// The 16 bytes of channels from c on of a head's row x, rotated by the table row f (nullptr: as they are).
template <typename T>
__device__ __forceinline__ void turned(const T* x, int c, const float* f, int rot, int half, float (&out)[16 / sizeof(T)]) {
    constexpr int V = 16 / sizeof(T);
    T own[V];
    *reinterpret_cast<uint4*>(own) = __ldg(reinterpret_cast<const uint4*>(x + c));
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = to_f32(own[e]);
    if (f == nullptr || c >= rot) return;
    if (!half) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            if (c + e >= rot) break;
            const float2 z = __ldg(reinterpret_cast<const float2*>(f + c + e));
            const float u = out[e], w = out[e + 1];
            out[e] = u * z.x - w * z.y;
            out[e + 1] = u * z.y + w * z.x;
        }
        return;
    }
    const int hr = rot / 2;
    if (hr % V == 0) {
        const bool first = c < hr;
        T other[V];
        *reinterpret_cast<uint4*>(other) = __ldg(reinterpret_cast<const uint4*>(x + (first ? c + hr : c - hr)));
        const float2* z = reinterpret_cast<const float2*>(f) + (first ? c : c - hr);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 y = __ldg(z + e);
            const float w = to_f32(other[e]);
            out[e] = first ? out[e] * y.x - w * y.y : w * y.y + out[e] * y.x;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (c + e >= rot) break;
            const bool first = c + e < hr;
            const float2 y = __ldg(reinterpret_cast<const float2*>(f) + (first ? c + e : c + e - hr));
            const float w = to_f32(x[first ? c + e + hr : c + e - hr]);
            out[e] = first ? out[e] * y.x - w * y.y : w * y.y + out[e] * y.x;
        }
    }
}

// Rows of bf16 heads, rotated, 16 bytes at a time and both halves of a pair together where the half layout allows:
// a unit u of a row is chunk u, or, where paired, chunks u and u + rot / 16.  put(chunk, values) takes each.
__device__ __forceinline__ bool paired(const DecArgs& a) { return a.rot > 0 && a.half && (a.rot / 2) % 8 == 0; }
__device__ __forceinline__ int units_of(const DecArgs& a, int chunks) { return paired(a) ? chunks - a.rot / 16 : chunks; }
template <typename Put>
__device__ __forceinline__ void turn_unit(const DecArgs& a, const __nv_bfloat16* x, int u, const float* f, Put put) {
    const int hc = a.rot / 16;                                   // chunks of half of the rotated channels
    if (!paired(a) || u >= hc) {
        float v[8];
        const int c = paired(a) ? u + hc : u;
        turned(x, c * 8, f, a.rot, a.half, v);
        put(c, v);
        return;
    }
    const uint4 l = __ldg(reinterpret_cast<const uint4*>(x + u * 8)), r = __ldg(reinterpret_cast<const uint4*>(x + (u + hc) * 8));
    float4 z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = __ldg(reinterpret_cast<const float4*>(f + u * 16) + e);
    const uint32_t lw[4] = {l.x, l.y, l.z, l.w}, rw[4] = {r.x, r.y, r.z, r.w};
    float lo[8], hi[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a0 = __uint_as_float(lw[e] << 16), a1 = __uint_as_float(lw[e] & 0xFFFF0000u);
        const float b0 = __uint_as_float(rw[e] << 16), b1 = __uint_as_float(rw[e] & 0xFFFF0000u);
        lo[2 * e] = a0 * z[e].x - b0 * z[e].y;
        hi[2 * e] = a0 * z[e].y + b0 * z[e].x;
        lo[2 * e + 1] = a1 * z[e].z - b1 * z[e].w;
        hi[2 * e + 1] = a1 * z[e].w + b1 * z[e].z;
    }
    put(u, lo);
    put(u + hc, hi);
}

// A bf16 cache as [batch * kv_heads][max_len][hd], boxes of `rows` rows x 64 channels of one head: rows from max_len
// on and channels from hd on read zero, and no coordinate passes 32 bits however long the caches are.
inline bool make_cache_map(CUtensorMap* map, const void* base, const DecodeProb& p, uint32_t rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)p.hd, (cuuint64_t)p.max_len, (cuuint64_t)(p.batch * p.kvh)};
    cuuint64_t strides[2] = {(cuuint64_t)p.hd * 2, (cuuint64_t)p.hd * 2 * p.max_len};
    cuuint32_t box[3] = {64, rows, 1};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a block works on.
struct Place {
    int64_t b;
    int kv, tile, split;           // row tile, run of the cache
    int64_t len;                   // cached tokens
    int64_t from, to;              // this run: cached rows from .. to - 1
    bool tail, idle;
};
template <int ROWS>
__device__ __forceinline__ Place place_of(const DecArgs& a, int tokens_per_tile) {
    Place p;
    const int tiles = (a.rows + ROWS - 1) / ROWS;
    int64_t x = blockIdx.x;
    p.split = (int)(x % a.n_split);
    x /= a.n_split;
    p.tile = (int)(x % tiles);
    x /= tiles;
    p.kv = (int)(x % a.kvh);
    p.b = x / a.kvh;
    p.len = __ldg(a.lens + p.b);
    p.idle = p.len < 0;
    if (p.len + a.M > a.max_len) {
        p.idle = true;
        if (threadIdx.x == 0) atomicOr(a.err, kErrCacheLen);
    }
    const int64_t n = p.idle ? 0 : p.len;
    const int64_t chunk = (n + (int64_t)a.n_split * tokens_per_tile - 1) / ((int64_t)a.n_split * tokens_per_tile) * tokens_per_tile;
    p.from = min(n, chunk * p.split);
    p.to = min(n, p.from + chunk);
    p.tail = p.split == a.n_split - 1;
    return p;
}
// A row of the last run that sees nothing at all takes a weight of 1 on a value of zero (its o is zero); a sum of
// zero is then that of a row without a finite score, which has no softmax (0 / 0).
__device__ __forceinline__ bool sees_nothing(const DecArgs& a, const Place& p, const uint64_t* seen, int row) {
    return p.tail && p.len == 0 && row < a.rows && seen[row / a.group] == 0;
}
// What each drafted token sees and the table row of its position; false where a position is outside the table.
__device__ __forceinline__ bool look_up(const DecArgs& a, const Place& p, uint64_t* seen, const float** turn) {
    bool ok = true;
    for (int m = threadIdx.x; m < a.M; m += kThreads) {
        const uint64_t s = seen_by(a, p.b, m);
        const int64_t pos = p.len + depth_of(s, m);
        ok = ok && (a.rot == 0 || pos < a.max_pos);
        seen[m] = s;
        turn[m] = a.rot ? a.cs + pos * a.rot : nullptr;
    }
    return __syncthreads_and(ok) != 0;
}

// Joins NP partial results of ROWS rows in shared memory (so [NP][ROWS][HD] not yet divided by the sum, smax and
// ssum [NP][ROWS]) and either writes o or leaves this run's part and, as the last block of its rows, joins the
// runs.  The loads of a join are independent of one another (weights first, then 16 values in flight per
// thread and more): a load and its use in turn, run by run, took longer than the attention itself.
// `weights`: shared memory for 2 x ROWS x n_split floats (n_split <= 64).
template <typename T, int HD, int ROWS, int NP>
__device__ __forceinline__ void finish(const DecArgs& a, const Place& p, const float* so, const float* smax,
                                       const float* ssum, float* weights, T* __restrict__ o) {
    __shared__ int last;
    __shared__ float inverse[ROWS];
    constexpr int kItems = ROWS * HD / 4 / kThreads;             // runs of four channels per thread
    static_assert(kItems >= 1, "a thread has work");
    const int tiles = (a.rows + ROWS - 1) / ROWS;
    const int64_t group = (p.b * a.kvh + p.kv) * tiles + p.tile;
    const int rows = min(ROWS, a.rows - p.tile * ROWS);
    float* parts = a.part + group * a.n_split * (int64_t)(ROWS * (HD + 2));
    float* stats = parts + (int64_t)a.n_split * ROWS * HD;       // [n_split][ROWS][2]: maximum, sum
    auto put = [&](int r, int c, float4 s, float inv) {
        const int row = p.tile * ROWS + r, m = row / a.group, g = row - m * a.group;
        T* to = o + (p.b * a.M + m) * a.os + ((int64_t)p.kv * a.group + g) * a.hd + c;
        if (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(to) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
        } else {
            *reinterpret_cast<uint2*>(to) = make_uint2(pack2(s.x * inv, s.y * inv), pack2(s.z * inv, s.w * inv));
        }
    };
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
        const int i = threadIdx.x + it * kThreads, r = i / (HD / 4), c = (i % (HD / 4)) * 4;
        if (r >= rows) break;
        float mx = -INFINITY, l = 0.f;
#pragma unroll
        for (int n = 0; n < NP; ++n) mx = fmaxf(mx, smax[n * ROWS + r]);
        const float use = mx == -INFINITY ? 0.f : mx;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const float w = exp2f(smax[n * ROWS + r] - use);
            const float4 x = *reinterpret_cast<const float4*>(so + (n * ROWS + r) * HD + c);
            s.x += w * x.x; s.y += w * x.y; s.z += w * x.z; s.w += w * x.w;
            l += w * ssum[n * ROWS + r];
        }
        if (a.n_split == 1) {
            if (c < a.hd) put(r, c, s, 1.f / l);
        } else {
            *reinterpret_cast<float4*>(parts + ((int64_t)p.split * ROWS + r) * HD + c) = s;
            if (c == 0) *reinterpret_cast<float2*>(stats + (p.split * ROWS + r) * 2) = make_float2(mx, l);
        }
    }
    if (a.n_split == 1) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t done = atomicAdd(a.count + group, 1u);
        last = done == (uint32_t)a.n_split - 1;
        if (last) a.count[group] = 0;            // ready for the next call
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    float* sums = weights + ROWS * a.n_split;
    for (int i = threadIdx.x; i < a.n_split * rows; i += kThreads) {
        const int n = i / rows, r = i - n * rows;
        const float2 x = __ldcg(reinterpret_cast<const float2*>(stats + (n * ROWS + r) * 2));
        weights[r * a.n_split + n] = x.x;
        sums[r * a.n_split + n] = x.y;
    }
    __syncthreads();
    if (threadIdx.x < rows) {
        float* w = weights + threadIdx.x * a.n_split;
        const float* l = sums + threadIdx.x * a.n_split;
        float mx = -INFINITY, sum = 0.f;
        for (int n = 0; n < a.n_split; ++n) mx = fmaxf(mx, w[n]);
        const float use = mx == -INFINITY ? 0.f : mx;
        for (int n = 0; n < a.n_split; ++n) {
            w[n] = exp2f(w[n] - use);
            sum += w[n] * l[n];
        }
        inverse[threadIdx.x] = 1.f / sum;
    }
    __syncthreads();
    float4 s[kItems];
#pragma unroll
    for (int it = 0; it < kItems; ++it) s[it] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll (kItems >= 8 ? 2 : 16 / kItems)
    for (int n = 0; n < a.n_split; ++n) {
        float4 x[kItems];
#pragma unroll
        for (int it = 0; it < kItems; ++it) {
            const int i = threadIdx.x + it * kThreads, r = i / (HD / 4), c = (i % (HD / 4)) * 4;
            x[it] = r < rows ? __ldcg(reinterpret_cast<const float4*>(parts + ((int64_t)n * ROWS + r) * HD + c))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int it = 0; it < kItems; ++it) {
            const int r = (threadIdx.x + it * kThreads) / (HD / 4);
            const float w = r < rows ? weights[r * a.n_split + n] : 0.f;
            s[it].x += w * x[it].x; s[it].y += w * x[it].y; s[it].z += w * x[it].z; s[it].w += w * x[it].w;
        }
    }
#pragma unroll
    for (int it = 0; it < kItems; ++it) {
        const int i = threadIdx.x + it * kThreads, r = i / (HD / 4), c = (i % (HD / 4)) * 4;
        if (r < rows && c < a.hd) put(r, c, s[it], inverse[r]);
    }
}

// The rows of an idle slot.
template <typename T, int ROWS>
__device__ __forceinline__ void zero_rows(const DecArgs& a, const Place& p, T* o) {
    if (!p.tail || threadIdx.x >= kThreads) return;
    const int rows = min(ROWS, a.rows - p.tile * ROWS);
    for (int i = threadIdx.x; i < rows * a.hd; i += kThreads) {
        const int row = p.tile * ROWS + i / a.hd, m = row / a.group, g = row - m * a.group;
        o[(p.b * a.M + m) * a.os + ((int64_t)p.kv * a.group + g) * a.hd + i % a.hd] = from_f32<T>(0.f);
    }
}


}  // namespace attn_dec

// The tcgen05 kernel of bf16 steps with many rows (attn_decode_tc.cu).
cudaError_t attn_decode_tc(const DecodeProb& p, const attn_dec::DecArgs& a, unsigned grid, const void* q, const void* k,
                           const void* v, void* k_cache, void* v_cache, void* o, cudaStream_t st);

}  // namespace dynconv
