// rope.cu -- rotary positions as an operator of its own: every head's first `rot` channels are
// turned pair by pair at the token's position,
//   (a, b) -> (a cos - b sin, a sin + b cos)     (inverse: sin negated),
// with the pairs consecutive (interleaved) or rot / 2 apart (half), the factors read from a
// caller's fp32 table, so that any context scaling is a matter of that table.  The products and
// their sum are in fp32, rounded once to the storage type.
//
// Memory-bound: x is read and y written once.  A block takes one token (its position and table
// row once, the row staying in L1 for every head), a thread one unit of 16 bytes of a head -- for
// the half layout the two 16-byte runs that pair up -- so loads and stores are 16 bytes wide
// where sizes and strides allow it; otherwise a unit is one pair (or one copied channel).
#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "prof.h"

namespace dynconv {
namespace {

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

struct RopeArgs {
    int64_t N, xs, ys, max_pos, n_docs, seqlen;
    int heads, hd, rot, inverse, copy;      // copy: the channels from rot on are written too
    const float* cs;
    const int32_t* cu;
    const int32_t* pos;
    uint32_t* err;
};

// V channels per access; HALF: units of V pairs (two accesses), else of V / 2 pairs (V >= 2) or one pair (V == 1).
template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(256) rope_heads_kernel(const T* x, T* y, RopeArgs a) {
    constexpr int kSpan = HALF ? V : (V == 1 ? 2 : V);       // channels of the rotated half / run per unit
    const int64_t n = blockIdx.x;
    int64_t p;
    if (a.pos != nullptr)
        p = __ldg(a.pos + n);
    else
        p = n - seg_start(n, a.cu, a.n_docs, a.seqlen);
    if (p < 0 || p >= a.max_pos) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrRopePos);
        p = p < 0 ? 0 : a.max_pos - 1;
    }
    const float* row = a.cs + p * a.rot;
    const int turned = HALF ? a.rot / 2 / kSpan : a.rot / kSpan;
    const int units = turned + (a.copy ? (a.hd - a.rot + V - 1) / V : 0);
    const int total = units * a.heads;
    const float sgn = a.inverse ? -1.f : 1.f;
    const T* xr = x + n * a.xs;
    T* yr = y + n * a.ys;
    for (int u = threadIdx.x; u < total; u += blockDim.x) {
        const int h = u / units, w = u - h * units;
        const T* xh = xr + (int64_t)h * a.hd;
        T* yh = yr + (int64_t)h * a.hd;
        if (w >= turned) {
            const int c = a.rot + (w - turned) * V;
            *reinterpret_cast<Vec<T, V>*>(yh + c) = *reinterpret_cast<const Vec<T, V>*>(xh + c);
        } else if (HALF) {
            const int c = w * V, o = a.rot / 2;
            const Vec<T, V> l = *reinterpret_cast<const Vec<T, V>*>(xh + c);
            const Vec<T, V> r = *reinterpret_cast<const Vec<T, V>*>(xh + c + o);
            Vec<T, V> lo, hi;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 f = __ldg(reinterpret_cast<const float2*>(row + 2 * (c + e)));
                const float p0 = to_f32(l.v[e]), p1 = to_f32(r.v[e]), s = sgn * f.y;
                lo.v[e] = from_f32<T>(p0 * f.x - p1 * s);
                hi.v[e] = from_f32<T>(p0 * s + p1 * f.x);
            }
            *reinterpret_cast<Vec<T, V>*>(yh + c) = lo;
            *reinterpret_cast<Vec<T, V>*>(yh + c + o) = hi;
        } else if (V == 1) {
            const int c = 2 * w;
            const float2 f = __ldg(reinterpret_cast<const float2*>(row + c));
            const float p0 = to_f32(xh[c]), p1 = to_f32(xh[c + 1]), s = sgn * f.y;
            yh[c] = from_f32<T>(p0 * f.x - p1 * s);
            yh[c + 1] = from_f32<T>(p0 * s + p1 * f.x);
        } else {
            const int c = w * V;
            Vec<T, V> z = *reinterpret_cast<const Vec<T, V>*>(xh + c);
#pragma unroll
            for (int e = 0; e + 1 < V; e += 2) {
                const float2 f = __ldg(reinterpret_cast<const float2*>(row + c + e));
                const float p0 = to_f32(z.v[e]), p1 = to_f32(z.v[e + 1]), s = sgn * f.y;
                z.v[e] = from_f32<T>(p0 * f.x - p1 * s);
                z.v[e + 1] = from_f32<T>(p0 * s + p1 * f.x);
            }
            *reinterpret_cast<Vec<T, V>*>(yh + c) = z;
        }
    }
}

template <typename T, int V, bool HALF>
cudaError_t launch_v(const RopeProb& p, const T* x, T* y, const RopeArgs& a, cudaStream_t st) {
    const int span = HALF ? V : (V == 1 ? 2 : V);
    const int units = (HALF ? p.rot / 2 / span : p.rot / span) + (a.copy ? (p.hd - p.rot + V - 1) / V : 0);
    const int total = units * p.heads;
    // a thread takes total / iters units: whole warps, no block above 256 threads, the last trip full
    const int iters = (total + 255) / 256;
    const int threads = std::min(256, ((total + iters - 1) / iters + 31) / 32 * 32);
    DC_LAUNCH(kRope, st, rope_heads_kernel<T, V, HALF><<<(unsigned)p.N, threads, 0, st>>>(x, y, a));
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const RopeProb& p, const void* xv, void* yv, uint32_t* err, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const T* x = static_cast<const T*>(xv);
    T* y = static_cast<T*>(yv);
    RopeArgs a{p.N, p.xs, p.ys, p.max_pos, p.n_docs, p.seqlen, p.heads, p.hd, p.rot, p.inverse,
               p.rot < p.hd && xv != yv ? 1 : 0, p.cs, p.cu, p.pos, err};
    // 16-byte units need every run to start on a 16-byte boundary (the base pointers do)
    const bool wide = p.hd % V == 0 && p.xs % V == 0 && p.ys % V == 0 && (p.half ? p.rot / 2 : p.rot) % V == 0;
    if (p.half) return wide ? launch_v<T, V, true>(p, x, y, a, st) : launch_v<T, 1, true>(p, x, y, a, st);
    return wide ? launch_v<T, V, false>(p, x, y, a, st) : launch_v<T, 1, false>(p, x, y, a, st);
}

}  // namespace

cudaError_t rope_launch(const RopeProb& p, const void* x, void* y, uint32_t* err, cudaStream_t st) {
    return p.dtype == 1 ? launch_t<__nv_bfloat16>(p, x, y, err, st) : launch_t<float>(p, x, y, err, st);
}

}  // namespace dynconv
