// layer.cuh -- device helpers shared by the norm, convolution and scan kernels:
// vectors of bf16 or f32 elements, the gates' functions and the search of a
// packed token's sequence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_common.cuh"

namespace kda {
namespace layer {

template <bool BF16>
struct ElemOf;
template <>
struct ElemOf<true> { using type = __nv_bfloat16; };
template <>
struct ElemOf<false> { using type = float; };
template <bool BF16>
using Elem = typename ElemOf<BF16>::type;

// V consecutive elements as loaded.  V > 1 takes one access of V elements (4,
// 8 or 16 bytes), which the address has to be a multiple of.
template <bool BF16, int V>
struct Vec {
    static constexpr int kBytes = V * (BF16 ? 2 : 4);
    static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const Elem<BF16> *p) {
        if constexpr (kBytes == 2) {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else if constexpr (kBytes == 8) {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            w[0] = x.x, w[1] = x.y;
        } else {
            const uint4 x = *reinterpret_cast<const uint4 *>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        }
    }
    __device__ __forceinline__ void store(Elem<BF16> *p) const {
        if constexpr (kBytes == 2) *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
        else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
        else if constexpr (kBytes == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (!BF16) return __uint_as_float(w[i]);
        else return (i & 1) ? __uint_as_float(w[i >> 1] & 0xffff0000u) : __uint_as_float(w[i >> 1] << 16);
    }
    // elements 2 i and 2 i + 1 (of one element: it and 0)
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (V == 1) return make_float2(get(0), 0.f);
        else return make_float2(get(2 * i), get(2 * i + 1));
    }
    __device__ __forceinline__ void set_pair(int i, float2 x) {
        if constexpr (!BF16) {
            w[V == 1 ? 0 : 2 * i] = __float_as_uint(x.x);
            if constexpr (V > 1) w[2 * i + 1] = __float_as_uint(x.y);
        } else {
            w[i] = pack_bf16(x.x, x.y);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[V]) {
        if constexpr (!BF16) {
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] = __float_as_uint(x[i]);
        } else if constexpr (V == 1) {
            w[0] = pack_bf16(x[0], 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) w[i >> 1] = pack_bf16(x[i], x[i + 1]);
        }
    }
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// What exp2_fast(x) is low by, added to x: over arguments from -1 to -2^-14 its
// results lie 0.1 to 0.4 of 2^-24 below 2^x on average.  A state multiplied by
// hundreds of them in a row shows that (dA of 2048 tokens: 1.8e-6 off against
// 1.0e-6), and the argument is a product that takes an addend for nothing.
constexpr float kExp2Low = 0.25f * 5.9604645e-8f * 1.4426950f;

// (of 2^126 and more: 0)
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-x): past e^-x = 2^126 it comes out 0 (where x sigmoid(x) is below 1.1e-36)
__device__ __forceinline__ float sigmoid(float x) { return rcp_fast(1.f + __expf(-x)); }
// x sigmoid(x); -inf gives NaN, as the product does
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// Pairs of the packed fp32 operations
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 sigmoid2(float2 x) {
    const float2 t = __fmul2_rn(x, both(-1.4426950408889634f));
    const float2 d = __fadd2_rn(make_float2(exp2_fast(t.x), exp2_fast(t.y)), both(1.f));
    return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}
__device__ __forceinline__ float2 silu2(float2 x) { return __fmul2_rn(x, sigmoid2(x)); }
// its derivative, from x and its sigmoid
__device__ __forceinline__ float2 dsilu2(float2 x, float2 s) {
    return __fmul2_rn(s, __ffma2_rn(x, __fadd2_rn(both(1.f), make_float2(-s.x, -s.y)), both(1.f)));
}

// ln(1 + e^v) = max(v, 0) + ln(1 + e), e = e^{-|v|} <= 1, and
// ln(1 + e) = 2 atanh(q), q = e / (2 + e) <= 1 / 3:
// no branch, and small values keep their relative precision, which the
// steps of a scan need: they add up what is off here over the tokens that a
// state remembers.  atanh(q) / q is a polynomial of degree four in q^2, through its
// values at the five Chebyshev points of [0, 1/9]: within 2^-26.9.  e is off by
// |v| 2^-24 and the exponential's own 2^-22.5 at most.
// sig: e^v / (1 + e^v), its derivative.
__device__ __forceinline__ float2 softplus2(float2 v, float2 &sig) {
    constexpr float c = -1.4426950408889634f;
    const float2 e = make_float2(exp2_fast(fabsf(v.x) * c), exp2_fast(fabsf(v.y) * c));
    const float2 below = __fadd2_rn(e, both(2.f)), one = __fadd2_rn(e, both(1.f));
    const float2 q = __fmul2_rn(e, make_float2(rcp_fast(below.x), rcp_fast(below.y))), w = __fmul2_rn(q, q);
    float2 s = __ffma2_rn(w, both(0.1407889f), both(0.13982579f));
    s = __ffma2_rn(w, s, both(0.20012298f));
    s = __ffma2_rn(w, s, both(0.33333161f));
    s = __ffma2_rn(w, s, both(1.f));
    sig = __fmul2_rn(make_float2(v.x >= 0.f ? 1.f : e.x, v.y >= 0.f ? 1.f : e.y), make_float2(rcp_fast(one.x), rcp_fast(one.y)));
    return __ffma2_rn(__fadd2_rn(q, q), s, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus(float v) {
    float2 sig;
    return softplus2(make_float2(v, 0.f), sig).x;
}

__device__ __forceinline__ void prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

// The first s in [0, N) for which past(s) holds (N if there is none), past
// being false up to some s and true from there on.  Each round asks for 32
// places, one per lane: a whole warp calls.
template <class F>
__device__ __forceinline__ int first_past(int N, F &&past) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = N;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, at >= lo + n || past(at));
        const int k = m ? __ffs(m) - 1 : 32;
        if (k == 0) break;
        const int next = lo + (k - 1) * step + 1;
        n = min(lo + k * step, lo + n) - next;
        lo = next;
    }
    return lo;
}

// the first sequence whose end is past token t
__device__ __forceinline__ int find_sequence(const int32_t *cu, int N, int t) {
    return first_past(N, [&](int s) { return cu[s + 1] > t; });
}

}  // namespace layer
}  // namespace kda
