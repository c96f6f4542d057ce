// cache4_rows.cu -- key and value rows into the 4-bit pages, and back.
//
// Per group of 16 channels x (y = x / head scale where one is given):
//     s = e4m3(max|y| / 6),  code = e2m1(y / s)      (nearest, ties to even, saturating; s = 0 has codes 0)
//     x' = code * s * head scale.
// A thread takes one group of a token and head, of the key and of the value:
// 32 bytes in per row at bf16, 8 bytes of codes and one scale out.  Memory
// bounds it: 2 x (2 or 4) bytes read and 2 x 9/16 bytes written per channel.
// Rows of 32K tokens x 12 heads x 128, 258 MB each way, other rows each time,
// by call.  Slots in random order: append 66 us (3.9 TB/s, 58 % of the measured
// copy bandwidth), read 54 us (71 %).  Slots in order: 49 and 43 us (78 and
// 88 %).  The difference is sectors of 32 bytes: a value of one token lies in
// 12 of them (its codes in 8, its scales in 4), of which it fills a quarter
// and a sixteenth; neighbouring tokens share them and scattered ones do not.
// (The same rows written again and again take 48 us at random slots: the L2
// cache holds some of them.)
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

// 32 bytes in one access where rows lie on 32-byte boundaries (a lane's share
// of a bf16 row is then one whole sector), in two otherwise
__device__ __forceinline__ void load32(const char *p, bool wide, uint32_t *w) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
}
__device__ __forceinline__ void store32(char *p, bool wide, const uint32_t *w) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// 16 channels as loaded: eight words of bf16 pairs, or sixteen floats
template <bool BF16>
struct Group {
    uint32_t w[BF16 ? 8 : 16];
    __device__ __forceinline__ void load(const void *base, size_t elem, bool wide) {
        const char *p = static_cast<const char *>(base) + elem * (BF16 ? 2 : 4);
        load32(p, wide, w);
        if constexpr (!BF16) load32(p + 32, wide, w + 8);
    }
    // channels 2 i and 2 i + 1
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (BF16) return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        else return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
};

// eight codes of four pairs, the first pair in the low byte
__device__ __forceinline__ uint32_t to_codes(const float2 (&y)[4]) {
    uint32_t r;
    asm("{\n.reg .b8 a, b, c, d;\n"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\ncvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        "mov.b32 %0, {a, b, c, d};\n}\n"
        : "=r"(r)
        : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
    return r;
}

// Codes and scale byte of a group; returns whether it is finite.
//
// The quotients decide ties, so they have to be exact where the true quotient
// is a midpoint of the codes.  bf16 channels without a head scale: x has 8
// significant bits, s has 4 and a midpoint m has 3, so x / s is m itself or at
// least 2^-8 m >= 2^-10 away from it.  x * (1 / s), off by 2^-22 of its value
// at most, is therefore brought to the nearest multiple of 2^-12 (adding and
// taking away 3 * 2^10, whose unit that is): midpoints become exact and no
// quotient changes sides.  This took the 12 instructions of a division per
// channel down to two for a pair.  Other inputs are divided.
template <bool BF16, bool SCALED>
__device__ __forceinline__ bool quantise(const Group<BF16> &g, float head_scale, uint2 &codes, uint32_t &scale) {
    float top;
    bool finite;
    float2 x[8];
    if constexpr (BF16 && !SCALED) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, g.w[i] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
        finite = m < 0x7f80u;
        top = __uint_as_float(m << 16);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = g.pair(i);
    } else {
        top = 0.f;
        finite = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = g.pair(i);
            finite = finite && fabsf(x[i].x) <= 3.402823466e38f && fabsf(x[i].y) <= 3.402823466e38f;
            if constexpr (SCALED) {
                // (a quotient past fp32 saturates as any other; 0 / 0 and a scale of NaN have none)
                x[i].x = x[i].x / head_scale, x[i].y = x[i].y / head_scale;
                finite = finite && x[i].x == x[i].x && x[i].y == x[i].y;
            }
            top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        }
    }
    unsigned short b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(b) : "f"(0.f), "f"(top / 6.f));
    scale = b & 0xffu;
    const float s = e4m3_to_float(scale);
    codes = make_uint2(0, 0);
    if (s > 0.f) {
        float2 y[2][4];
        if constexpr (BF16 && !SCALED) {
            const float r = 1.f / s;
            const float2 r2 = make_float2(r, r), unit = make_float2(3072.f, 3072.f), back = make_float2(-3072.f, -3072.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i >> 2][i & 3] = __fadd2_rn(__ffma2_rn(x[i], r2, unit), back);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i >> 2][i & 3] = make_float2(x[i].x / s, x[i].y / s);
        }
        codes = make_uint2(to_codes(y[0]), to_codes(y[1]));
    }
    return finite;
}

// the block of a slot and head
template <int D>
__device__ __forceinline__ uint8_t *block_of(const Cache4RowsArgs &a, int slot, int h) {
    const int page = slot >> a.page_shift, blk = (slot & ((1 << a.page_shift) - 1)) >> 4;
    return a.cache + ((((size_t)page * a.Hkv + h) << (a.page_shift - 4)) + blk) * block_bytes(D);
}

template <int D, bool BF16, bool SCALED>
__global__ void __launch_bounds__(256)
kda_cache4_append_kernel(Cache4RowsArgs a) {
    constexpr int GROUPS = D / 16;  // lanes of a token and head: 8 or 4 neighbours in a warp
    const uint32_t th = blockIdx.x * (256 / GROUPS) + threadIdx.x / GROUPS;  // below 2^32
    const int grp = threadIdx.x % GROUPS;
    const uint32_t t = th / (uint32_t)a.Hkv, h = th - t * (uint32_t)a.Hkv;
    const bool live = t < (uint32_t)a.T;
    // the rows are asked for beside their slot, not after it (a row without one is read in vain)
    Group<BF16> k, v;
    int slot = -1;
    if (live) {
        slot = __ldg(a.slots + t);
        k.load(a.k, (size_t)t * a.k_stride + h * D + grp * 16, a.wide);
        v.load(a.v, (size_t)t * a.v_stride + h * D + grp * 16, a.wide);
    }
    const bool in_range = slot < a.num_slots;
    if (live && !in_range && a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
    const bool write = slot >= 0 && in_range;
    uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
    uint32_t ks = 0, vs = 0;
    bool finite = true;
    if (write) {
        finite = quantise<BF16, SCALED>(k, SCALED && a.k_scale ? a.k_scale[h] : 1.f, kc, ks);
        finite = quantise<BF16, SCALED>(v, SCALED && a.v_scale ? a.v_scale[h] : 1.f, vc, vs) && finite;
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
    const int tok = slot & 15;
    uint8_t *b = block_of<D>(a, slot, h);
    *reinterpret_cast<uint2 *>(b + tok * (D / 2) + grp * 8) = kc;
    b[off_ks(D) + tok * GROUPS + grp] = (uint8_t)ks;
    *reinterpret_cast<uint2 *>(b + off_vc(D) + grp * 128 + tok * 8) = vc;
    b[off_vs(D) + grp * 16 + tok] = (uint8_t)vs;
}

// 16 channels that codes and a scale byte stand for, stored as bf16 or f32
template <bool BF16>
__device__ __forceinline__ void store_values(void *base, size_t elem, uint2 codes, uint32_t scale, float head_scale,
                                             bool wide) {
    const uint32_t f = scales_to_f16(scale), s = __byte_perm(f, f, 0x1010);
    uint32_t x[2][4], u[BF16 ? 8 : 16];
    codes_to_f16(codes.x, x[0]);
    codes_to_f16(codes.y, x[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 v = unpack_f16(mul_f16x2(x[j >> 2][j & 3], s)), y = make_float2(v.x * head_scale, v.y * head_scale);
        if constexpr (BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
            u[j] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
            u[2 * j] = __float_as_uint(y.x);
            u[2 * j + 1] = __float_as_uint(y.y);
        }
    }
    char *p = static_cast<char *>(base) + elem * (BF16 ? 2 : 4);
    store32(p, wide, u);
    if constexpr (!BF16) store32(p + 32, wide, u + 8);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256)
kda_cache4_read_kernel(Cache4RowsArgs a) {
    constexpr int GROUPS = D / 16;
    const uint32_t th = blockIdx.x * (256 / GROUPS) + threadIdx.x / GROUPS;
    const int grp = threadIdx.x % GROUPS;
    const uint32_t t = th / (uint32_t)a.Hkv, h = th - t * (uint32_t)a.Hkv;
    if (t >= (uint32_t)a.T) return;
    const int slot = __ldg(a.slots + t);
    if (slot >= a.num_slots && a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
    uint2 kc = make_uint2(0, 0), vc = make_uint2(0, 0);
    uint32_t ks = 0, vs = 0;
    if (slot >= 0 && slot < a.num_slots) {
        const int tok = slot & 15;
        const uint8_t *b = block_of<D>(a, slot, h);
        kc = *reinterpret_cast<const uint2 *>(b + tok * (D / 2) + grp * 8);
        vc = *reinterpret_cast<const uint2 *>(b + off_vc(D) + grp * 128 + tok * 8);
        ks = b[off_ks(D) + tok * GROUPS + grp];
        vs = b[off_vs(D) + grp * 16 + tok];
        if ((ks & 0x7fu) == kScaleNaN) vs = ks;  // a marked token's value is not known either
    }
    const size_t e = ((size_t)t * a.Hkv + h) * D + grp * 16;
    store_values<BF16>(a.k_out, e, kc, ks, a.k_scale ? a.k_scale[h] : 1.f, a.wide);
    store_values<BF16>(a.v_out, e, vc, vs, a.v_scale ? a.v_scale[h] : 1.f, a.wide);
}

template <bool READ, int D, bool BF16>
cudaError_t launch(const Cache4RowsArgs &a, cudaStream_t st) {
    const long long th = (long long)a.T * a.Hkv, per = 256 / (D / 16);  // th below 2^32 - 2^12 (checked by the caller)
    const unsigned grid = (unsigned)((th + per - 1) / per);
    if constexpr (READ) kda_cache4_read_kernel<D, BF16><<<grid, 256, 0, st>>>(a);
    else if (a.k_scale || a.v_scale) kda_cache4_append_kernel<D, BF16, true><<<grid, 256, 0, st>>>(a);
    else kda_cache4_append_kernel<D, BF16, false><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

template <bool READ>
cudaError_t launch(const Cache4RowsArgs &a, int d, bool bf16, cudaStream_t st) {
    if (d == 128) return bf16 ? launch<READ, 128, true>(a, st) : launch<READ, 128, false>(a, st);
    return bf16 ? launch<READ, 64, true>(a, st) : launch<READ, 64, false>(a, st);
}

}  // namespace

cudaError_t launch_cache4_append(const Cache4RowsArgs &a, int d, bool bf16, cudaStream_t st) {
    return launch<false>(a, d, bf16, st);
}
cudaError_t launch_cache4_read(const Cache4RowsArgs &a, int d, bool bf16, cudaStream_t st) {
    return launch<true>(a, d, bf16, st);
}

}  // namespace kda
