// cache4_rows.cu -- key and value rows into the 4-bit pages, and back.
//
// Per group of 16 channels x (y = x / head scale where one is given):
//     s = e4m3(max|y| / 6),  code = e2m1(y / s)      (nearest, ties to even, saturating; s = 0 has codes 0)
//     x' = code * s * head scale.
// A thread takes one group of a token and head, of the key and of the value:
// 32 bytes in per row at bf16, 8 bytes of codes and one scale out.  Memory
// bounds it: 2 x (2 or 4) bytes read and 2 x 9/16 bytes written per channel.
//
// A token whose key or value is not finite in a head is marked there: its key
// scales are NaN and its value is zero, so every query that sees it comes out
// NaN and no other query does (a zero weight times NaN would spread it).
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache4.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

using namespace cache4;

template <bool BF16>
__device__ __forceinline__ void load16(const void *base, size_t elem, float (&x)[16]) {
    if constexpr (BF16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + elem);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 w = __ldg(p + h);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[h * 8 + 2 * j] = __uint_as_float(u[j] << 16);
                x[h * 8 + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + elem);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float4 w = __ldg(p + h);
            x[4 * h] = w.x, x[4 * h + 1] = w.y, x[4 * h + 2] = w.z, x[4 * h + 3] = w.w;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store16(void *base, size_t elem, const float (&x)[16]) {
    if constexpr (BF16) {
        uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + elem);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[h * 8 + 2 * j], x[h * 8 + 2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t *>(&v);
            }
            p[h] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + elem);
#pragma unroll
        for (int h = 0; h < 4; ++h) p[h] = make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
    }
}

// codes and scale byte of a group; returns whether it is finite
__device__ __forceinline__ bool quantise(float (&x)[16], float head_scale, uint2 &codes, uint32_t &scale) {
    float top = 0.f;
    bool finite = true;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (head_scale != 1.f) x[i] = x[i] / head_scale;
        finite = finite && fabsf(x[i]) <= 3.402823466e38f;
        top = fmaxf(top, fabsf(x[i]));
    }
    unsigned short b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(b) : "f"(0.f), "f"(top / 6.f));
    scale = b & 0xffu;
    const float s = e4m3_to_float(scale);
    uint32_t w[2] = {0, 0};
    if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            unsigned short c;
            asm("{\n.reg .b8 z;\ncvt.rn.satfinite.e2m1x2.f32 z, %1, %2;\ncvt.u16.u8 %0, z;\n}\n"
                : "=h"(c)
                : "f"(x[i + 1] / s), "f"(x[i] / s));
            w[i >> 3] |= (uint32_t)c << ((i & 7) * 4);
        }
    }
    codes = make_uint2(w[0], w[1]);
    return finite;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256)
cache4_append_kernel(Cache4RowsArgs a) {
    constexpr int GROUPS = D / 16;  // lanes of a token and head: 8 or 4 neighbours in a warp
    const long long items = (long long)a.T * a.Hkv * GROUPS;
    const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const bool live = item < items;
    const int grp = (int)(item % GROUPS);
    const long long th = live ? item / GROUPS : 0;
    const int h = (int)(th % a.Hkv), t = (int)(th / a.Hkv);
    const int slot = live ? a.slots[t] : -1;
    const bool in_range = slot < a.num_slots;
    if (live && !in_range && a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
    const bool write = live && slot >= 0 && in_range;
    uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
    uint32_t ks = 0, vs = 0;
    bool finite = true;
    if (write) {
        float x[16];
        load16<BF16>(a.k, (size_t)t * a.k_stride + (size_t)h * D + grp * 16, x);
        finite = quantise(x, a.k_scale ? a.k_scale[h] : 1.f, kc, ks);
        load16<BF16>(a.v, (size_t)t * a.v_stride + (size_t)h * D + grp * 16, x);
        finite = quantise(x, a.v_scale ? a.v_scale[h] : 1.f, vc, vs) && finite;
    }
#pragma unroll
    for (int o = 1; o < GROUPS; o <<= 1) finite = __shfl_xor_sync(0xffffffffu, (int)finite, o) && finite;
    if (!write) return;
    if (!finite) {
        kc = vc = make_uint2(0, 0);
        ks = kScaleNaN;
        vs = 0;
        if (grp == 0 && a.status) atomicOr(a.status, KDA_STATUS_NOT_FINITE);
    }
    const int page = slot >> a.page_shift, in_page = slot & ((1 << a.page_shift) - 1);
    const int blk = in_page >> 4, tok = in_page & 15;
    uint8_t *b = a.cache + (((size_t)page * a.Hkv + h) * ((size_t)1 << (a.page_shift - 4)) + blk) * block_bytes(D);
    *reinterpret_cast<uint2 *>(b + tok * (D / 2) + grp * 8) = kc;
    b[off_ks(D) + tok * GROUPS + grp] = (uint8_t)ks;
    *reinterpret_cast<uint2 *>(b + off_vc(D) + grp * 128 + tok * 8) = vc;
    b[off_vs(D) + grp * 16 + tok] = (uint8_t)vs;
}

__device__ __forceinline__ void values(uint2 codes, float s, float head_scale, float (&x)[16]) {
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t f[4];
        codes_to_f16(w[h], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = unpack_f16(f[j]);
            x[h * 8 + 2 * j] = v.x * s * head_scale;
            x[h * 8 + 2 * j + 1] = v.y * s * head_scale;
        }
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256)
cache4_read_kernel(Cache4RowsArgs a) {
    constexpr int GROUPS = D / 16;
    const long long item = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (item >= (long long)a.T * a.Hkv * GROUPS) return;
    const int grp = (int)(item % GROUPS);
    const long long th = item / GROUPS;
    const int h = (int)(th % a.Hkv), t = (int)(th / a.Hkv);
    const int slot = a.slots[t];
    if (slot >= a.num_slots && a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
    uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
    float ks = 0.f, vs = 0.f;
    if (slot >= 0 && slot < a.num_slots) {
        const int page = slot >> a.page_shift, in_page = slot & ((1 << a.page_shift) - 1);
        const int blk = in_page >> 4, tok = in_page & 15;
        const uint8_t *b =
            a.cache + (((size_t)page * a.Hkv + h) * ((size_t)1 << (a.page_shift - 4)) + blk) * block_bytes(D);
        kc = *reinterpret_cast<const uint2 *>(b + tok * (D / 2) + grp * 8);
        vc = *reinterpret_cast<const uint2 *>(b + off_vc(D) + grp * 128 + tok * 8);
        ks = e4m3_to_float(b[off_ks(D) + tok * GROUPS + grp]);
        vs = e4m3_to_float(b[off_vs(D) + grp * 16 + tok]);
        if (ks != ks) vs = ks;  // a marked token's value is not known either
    }
    float x[16];
    values(kc, ks, a.k_scale ? a.k_scale[h] : 1.f, x);
    store16<BF16>(a.k_out, ((size_t)t * a.Hkv + h) * D + grp * 16, x);
    values(vc, vs, a.v_scale ? a.v_scale[h] : 1.f, x);
    store16<BF16>(a.v_out, ((size_t)t * a.Hkv + h) * D + grp * 16, x);
}

template <bool READ>
cudaError_t launch(const Cache4RowsArgs &a, int d, bool bf16, cudaStream_t st) {
    const long long items = (long long)a.T * a.Hkv * (d / 16);
    const long long grid = (items + 255) / 256;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned g = (unsigned)grid;
#define KDA_ROWS(D, B)                                                     \
    if (READ) cache4_read_kernel<D, B><<<g, 256, 0, st>>>(a);              \
    else cache4_append_kernel<D, B><<<g, 256, 0, st>>>(a);
    if (d == 128 && bf16) { KDA_ROWS(128, true) }
    else if (d == 128) { KDA_ROWS(128, false) }
    else if (bf16) { KDA_ROWS(64, true) }
    else { KDA_ROWS(64, false) }
#undef KDA_ROWS
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache4_append(const Cache4RowsArgs &a, int d, bool bf16, cudaStream_t st) {
    return launch<false>(a, d, bf16, st);
}
cudaError_t launch_cache4_read(const Cache4RowsArgs &a, int d, bool bf16, cudaStream_t st) {
    return launch<true>(a, d, bf16, st);
}

}  // namespace kda
