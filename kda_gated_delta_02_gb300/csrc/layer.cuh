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

// 1 / (1 + e^-x): the quotient of a sum past 2^126 comes out 0, as it should
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
// x sigmoid(x); -inf gives NaN, as the product does
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// softplus, ln(1 + e^v), to a unit in the last place or two: the steps of a scan
// add up what is off here over the tokens that a state remembers
__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

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
