// rope.cu -- rotary positions as an operator of its own: every head's first `rot` channels are
// turned pair by pair at the token's position,
//   (a, b) -> (a cos - b sin, a sin + b cos)     (inverse: sin negated),
// with the pairs consecutive (interleaved) or rot / 2 apart (half), the factors read from a
// caller's fp32 table, so that any context scaling is a matter of that table.  The products and
// their sum are in fp32, rounded once to the storage type.
//
// Memory-bound: x is read and y written once.  Measured: 16384 tokens x 20 heads of 128, bf16, 32.0 us (5.2 TB/s, 0.80 of
// the copy rate); 15992 x 12 of 64, fp32, half of the channels rotated, 17.2 us (0.87); 64 tokens 2.1 us, a launch.  A
// block takes one token (its position and table row once, the row staying in L1 for every head), a thread one unit
// of 16 bytes of a head -- for the half layout the two 16-byte runs that pair up -- so loads and stores are 16 bytes
// wide where sizes and strides allow it; otherwise a unit is one pair (or one copied channel).
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
    constexpr int kPairs = HALF ? V : (V == 1 ? 1 : V / 2);  // pairs per unit
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
        const int at = h * a.hd + (w >= turned ? a.rot + (w - turned) * V : w * kSpan);
        Vec<T, V> l = *reinterpret_cast<const Vec<T, V>*>(xr + at), r;
        if (w < turned) {
            if (HALF) r = *reinterpret_cast<const Vec<T, V>*>(xr + at + a.rot / 2);
            else if (V == 1) r = *reinterpret_cast<const Vec<T, V>*>(xr + at + 1);
            // the factors: two pairs a load (a load's lanes are a run apart, so its width sets the L1 traffic)
            const float* z = row + (HALF ? 2 * w * V : w * kSpan);
            float f[2 * kPairs];
            if (kPairs >= 2) {
#pragma unroll
                for (int e = 0; e < kPairs / 2; ++e)
                    *reinterpret_cast<float4*>(&f[4 * e]) = __ldg(reinterpret_cast<const float4*>(z) + e);
            } else {
                *reinterpret_cast<float2*>(&f[0]) = __ldg(reinterpret_cast<const float2*>(z));
            }
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
                T& x = HALF || V == 1 ? l.v[HALF ? e : 0] : l.v[(2 * e) % V];
                T& y = HALF || V == 1 ? r.v[HALF ? e : 0] : l.v[(2 * e + 1) % V];
                const float p0 = to_f32(x), p1 = to_f32(y), c = f[2 * e], s = sgn * f[2 * e + 1];
                x = from_f32<T>(p0 * c - p1 * s);
                y = from_f32<T>(p0 * s + p1 * c);
            }
            if (HALF) *reinterpret_cast<Vec<T, V>*>(yr + at + a.rot / 2) = r;
            else if (V == 1) *reinterpret_cast<Vec<T, V>*>(yr + at + 1) = r;
        }
        *reinterpret_cast<Vec<T, V>*>(yr + at) = l;
    }
}

template <typename T, int V, bool HALF>
cudaError_t launch_v(const RopeProb& p, const T* x, T* y, const RopeArgs& a, cudaStream_t st) {
    const int span = HALF ? V : (V == 1 ? 2 : V);
    const int units = (HALF ? p.rot / 2 / span : p.rot / span) + (a.copy ? (p.hd - p.rot + V - 1) / V : 0);
    const int total = units * p.heads;
    // A thread takes total / trips units: whole warps, no block above 256 threads, the last trip full.  Small blocks of
    // three trips keep more tokens in flight (16384 tokens x 20 x 128 bf16: 32.0 us, 33.0 with one trip; 15992 x 12 x
    // 64 fp32, half of it rotated: 17.1 and 18.1); with fewer tokens than fill the GPU one trip is sooner done
    // (64 tokens x 20 x 128: 2.1 us, 3.1 with three).
    const int trips = std::max(p.N >= 8 * 148 ? 3 : 1, (total + 255) / 256);
    const int threads = std::min(256, ((total + trips - 1) / trips + 31) / 32 * 32);
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
