// cache4.cuh -- the paged 4-bit key/value cache: format arithmetic and the
// conversions shared by its kernels (page_plan.cu, cache4_rows.cu,
// cache4_attn.cu, cache4_attn_tc.cu).
//
// cache [pages][Hkv][page_size / 16 blocks][block bytes].  A block holds 16
// tokens of one head, in four parts one after the other:
//   key codes    [16 tokens][d / 2]        key scales   [16 tokens][d / 16]
//   value codes  [d / 16 groups][16][8]    value scales [d / 16 groups][16]
// A code is an e2m1 nibble (even channel low), a scale one e4m3 byte per group
// of 16 channels; the value held is code * scale, which f16 represents exactly
// (at most 2 + 4 significant bits, 2^-10 <= |x| <= 2688), so the tensor-core
// operands lose nothing over the cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace cache4 {

constexpr uint32_t kScaleNaN = 0x7F;  // e4m3 NaN: the key scales of a token whose key or value is not finite

__host__ __device__ constexpr int block_bytes(int d) { return 16 * (d + d / 8); }
__host__ __device__ constexpr int off_ks(int d) { return 16 * (d / 2); }
__host__ __device__ constexpr int off_vc(int d) { return 16 * (d / 2 + d / 16); }
__host__ __device__ constexpr int off_vs(int d) { return 16 * (d + d / 16); }

// log2 of a page size (a power of two from 16 to 256), or -1
inline int page_shift(int page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == (1 << s)) return s;
    return -1;
}

// eight codes of a 32-bit word as four f16 pairs (exact)
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&x)[4]) {
    asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(w));
}

// two e4m3 scales (low byte first) as an f16 pair (exact)
__device__ __forceinline__ uint32_t scales_to_f16(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"((unsigned short)two));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// f16 pairs times the low / high half of another pair
__device__ __forceinline__ uint32_t mul_low(uint32_t a, uint32_t s) {
    const __half2 r = __hmul2_rn(*reinterpret_cast<__half2 *>(&a), __low2half2(*reinterpret_cast<__half2 *>(&s)));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t mul_high(uint32_t a, uint32_t s) {
    const __half2 r = __hmul2_rn(*reinterpret_cast<__half2 *>(&a), __high2half2(*reinterpret_cast<__half2 *>(&s)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// f16 pair, lo in the low half
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
    return __half22float2(*reinterpret_cast<__half2 *>(&u));
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ float e4m3_to_float(uint32_t b) {
    return unpack_f16(scales_to_f16(b)).x;
}

}  // namespace cache4
}  // namespace kda
