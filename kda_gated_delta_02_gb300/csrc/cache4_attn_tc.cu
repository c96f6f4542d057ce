// cache4_attn_tc.cu -- attention over the 4-bit pages for many rows per key
// head (verify windows of wide groups, prompt chunks): tcgen05 products.
//
// Same operator and division of the work as cache4_attn.cu, with row tiles of
// QT x 128 rows and key tiles of 128.  One persistent CTA per SM, warps by
// role:
//   producer   1 warp   bulk copies of 64 keys at a time into a raw ring
//   dequant    12 - 4 QT warps  codes and scales -> f16 (exact), into the swizzled
//                       shared-memory operands K (K-major) and V (N-major)
//   products   1 thread S = Q K^T into tensor memory, O += P V with P read
//                       from tensor memory (it takes the place of S)
//   softmax    4 QT warps, a thread per row: maximum, weights (f16, lifted by
//                       2^kLift), sum, and the accumulator's rescaling
// The running maximum that the weights refer to moves only when it would rise
// by more than 2^8, so the accumulator (in tensor memory) is rescaled a few
// times per row tile; f16 holds the weights of up to 2^15 that this allows.
// With QT = 2 the two row tiles take turns: one's products run while the
// other's softmax does.  With QT = 1 the next tile's S is formed in a second
// buffer meanwhile.
//
// What bounds it: at QT = 2 the products (1,024 cycles of the tensor pipe per
// 128 x 128 pair of tiles at d = 128) and, close by, shared memory, which
// carries the converted operands in (64 KB per key tile) and out.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache4.cuh"
#include "cache4_sched.cuh"
#include "kda_internal.h"
#include "kda_umma.cuh"

namespace kda {
namespace {

using namespace cache4;

constexpr int kTile = 128;    // keys per tile
constexpr float kLift = 7.f;  // weights are at most 2^(kLift + kSlack)
constexpr float kSlack = 8.f;

template <int D, int QT>
struct Cfg {
    // 14 warps: 128 registers per thread
    static constexpr int SOFT = 4 * QT, DEQ = 12 - SOFT, WARPS = SOFT + DEQ + 2, THREADS = WARPS * 32;
    static constexpr int ROWS = 128 * QT;
    static constexpr int OPERAND = 128 * D * 2;       // 128 rows of f16
    static constexpr int RAW = 4 * block_bytes(D);    // 64 keys
    static constexpr int RAWS = QT == 2 ? 3 : 6;      // raw stages
    static constexpr int off_q = 0, off_k = QT * OPERAND, off_v = off_k + 2 * OPERAND, off_raw = off_v + 2 * OPERAND;
    static constexpr int off_bar = off_raw + RAWS * RAW;
    // barriers: raw full / empty, K and V full / empty, S full, P full, O done, Q full, drain
    static constexpr int b_raw_full = 0, b_raw_empty = RAWS, b_k_full = 2 * RAWS, b_k_empty = b_k_full + 2,
                         b_v_full = b_k_full + 4, b_v_empty = b_k_full + 6, b_s_full = b_k_full + 8,
                         b_p_full = b_k_full + 10, b_o_done = b_k_full + 12, b_q_full = b_k_full + 14,
                         b_drain = b_k_full + 15, BARS = b_k_full + 16;
    static constexpr int off_misc = off_bar + BARS * 8;  // TMEM address, dead flag
    static constexpr int SMEM = off_misc + 16;
    // tensor memory columns: S (and P over it) 2 x 128, O QT x D
    static constexpr int t_o = 256;
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D += A B with A in tensor memory (f16, two consecutive K per column, the lower one in the low half)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred pp;\nsetp.ne.b32 pp, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pp;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 16 channels of one key: two words of codes times one scale into two 16-byte chunks
__device__ __forceinline__ void convert(uint2 w, uint32_t scale, uint32_t a0, uint32_t a1) {
    uint32_t x[4];
    codes_to_f16(w.x, x);
    sts128(a0, mul_f16x2(x[0], scale), mul_f16x2(x[1], scale), mul_f16x2(x[2], scale), mul_f16x2(x[3], scale));
    codes_to_f16(w.y, x);
    sts128(a1, mul_f16x2(x[0], scale), mul_f16x2(x[1], scale), mul_f16x2(x[2], scale), mul_f16x2(x[3], scale));
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t byte) {
    const uint32_t f = scales_to_f16(byte);
    return __byte_perm(f, f, 0x1010);
}

template <int D, int QT>
__global__ void __launch_bounds__((Cfg<D, QT>::THREADS), 1)
cache4_attn_tc_kernel(const Cache4AttnArgs a) {
    using C = Cfg<D, QT>;
    constexpr int BB = block_bytes(D), KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sb = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.Hq / a.Hkv;
    auto bar = [&](int i) { return sb + C::off_bar + i * 8; };
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + C::off_misc);

    if (tid == 0) {
        for (int i = 0; i < C::RAWS; ++i) {
            umma::mbar_init(bar(C::b_raw_full + i), 1);
            umma::mbar_init(bar(C::b_raw_empty + i), C::DEQ);
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar(C::b_k_full + i), C::DEQ);
            umma::mbar_init(bar(C::b_k_empty + i), 1);
            umma::mbar_init(bar(C::b_v_full + i), C::DEQ);
            umma::mbar_init(bar(C::b_v_empty + i), 1);
            umma::mbar_init(bar(C::b_s_full + i), 1);
            umma::mbar_init(bar(C::b_p_full + i), 128);
            umma::mbar_init(bar(C::b_o_done + i), 1);
        }
        umma::mbar_init(bar(C::b_q_full), C::ROWS);
        umma::mbar_init(bar(C::b_drain), 1);
        misc[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) umma::tmem_alloc(sb + C::off_misc, 512);
    Walk<C::ROWS, kTile> walk(a);
    const int me = blockIdx.x;
    walk.begin(a, reinterpret_cast<long long *>(smem), me, gridDim.x);
    umma::fence_before();
    __syncthreads();  // barriers, the tensor memory address, and the prefix (over the operands) has been read
    umma::fence_after();
    const uint32_t tmem = misc[0];

    // a bounded wait that gives up when any role has; `wait` for whole warps,
    // whose lanes then agree
    auto wait1 = [&](int i, uint32_t parity) {
        for (uint32_t n = 0; n < 64; ++n) {
            if (umma::mbar_wait(bar(i), parity & 1, kWaitLimit / 64)) return true;
            if (misc[1]) return false;
        }
        misc[1] = 1;
        if (a.status) atomicOr(a.status, KDA_STATUS_TIMEOUT);
        return false;
    };
    auto wait = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait1(i, parity)) != 0; };

    Item it;
    if (warp < C::SOFT) {
        // ------------------------------------------------------------ softmax: a thread per row
        const int t = warp >> 2, lane_base = (warp & 3) * 32;
        const int my = t * 128 + lane_base + lane;
        const uint32_t tq = tmem + ((uint32_t)lane_base << 16);
        uint32_t n = 0;  // key tiles so far
        int4 job = make_int4(-1, 0, 0, 0);
        auto work = [&]() {
            while (walk.next(a, it)) {
                const Req &q = it.q;
                const int rr = it.row0 + my;
                const bool valid = rr < q.rows;
                const int tok = min(rr, q.rows - 1) / G, x = valid ? rr % G : 0;
                const size_t head = (size_t)(q.q0 + tok) * a.Hq + it.h * G + x;
                float m = -INFINITY, l = 0.f, fac = 1.f;
                if (it.last > it.first) {
                    // the query row, scaled by a power of two to [2^8, 2^9) at its largest, as f16
                    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                                     (size_t)(q.q0 + tok) * a.q_stride +
                                                                     (size_t)(it.h * G + x) * D);
                    uint32_t top = 0;  // magnitudes, which order as integers
#pragma unroll 4
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 w = __ldg(p + i);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) top = max(top, max((u[j] << 16) & 0x7fffffffu, u[j] & 0x7fff0000u));
                    }
                    if (!valid) top = 0;
                    const int ex = min(max((int)(top >> 23), 9), 253);
                    const float base = a.scale * kLog2e * (a.k_scale ? a.k_scale[it.h] : 1.f);
                    // the sign (and a zero) of the scale goes into the query: the factor stays positive
                    const float up = (base < 0.f ? -1.f : base == 0.f || !valid ? 0.f : 1.f) *
                                     __uint_as_float((uint32_t)(262 - ex) << 23);
                    fac = fmaxf(fabsf(base) * __uint_as_float((uint32_t)(ex - 8) << 23), 1e-37f);
                    const uint32_t row = sb + C::off_q + t * C::OPERAND;
                    const int r = lane_base + lane;
#pragma unroll 4
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 w = __ldg(p + i);
                        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                        uint32_t f[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f[j] = pack_f16(__uint_as_float(u[j] << 16) * up, __uint_as_float(u[j] & 0xffff0000u) * up);
                        sts128(row + umma::kmaj(r, i * 8, 128), f[0], f[1], f[2], f[3]);
                    }
                    umma::fence_proxy_async();
                    arrive(bar(C::b_q_full));
                }
                // positions this row sees (a padding row sees what the last row does), and what the whole warp sees
                const int sees = q.len - q.n + tok;
                const int see_lo = __reduce_min_sync(0xffffffffu, sees), see_hi = __reduce_max_sync(0xffffffffu, sees);
                const uint32_t to = tq + C::t_o + t * D;
                for (int tile = it.first; tile < it.last; ++tile, ++n) {
                    const int b = QT == 2 ? t : (int)(n & 1);
                    const uint32_t parity = QT == 2 ? n : n >> 1;
                    const uint32_t ts = tq + b * 128;
                    if (!wait(C::b_s_full + b, parity)) return;
                    umma::fence_after();
                    const int key0 = tile * kTile;
                    const bool edge = key0 + kTile > see_lo + 1 || (a.window > 0 && key0 <= see_hi - a.window);
                    const int hi = sees - key0;                                             // last visible column
                    const int lo = a.window > 0 ? sees - a.window - key0 : -1;              // last hidden one before
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        umma::ld32(ts + c * 32, s);
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i > hi || c * 32 + i <= lo) s[i] = -INFINITY;
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2) top = fmaxf(top, fmaxf(s[i], s[i + 1]));
                    }
                    top *= fac;
                    if (tile == it.first) {
                        m = top;
                    } else {
                        const bool rise = top > m + kSlack || (m == -INFINITY && top > m);
                        if (__any_sync(0xffffffffu, rise)) {
                            // with one row tile the last product onto O may still run
                            if (QT == 1) {
                                if (!wait(C::b_o_done, n - 1)) return;
                                umma::fence_after();
                            }
                            const float f = rise ? exp2_fast(m - top) : 1.f;
                            l *= f;
                            if (rise) m = top;
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float o[32];
                                umma::ld32(to + c * 32, o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                umma::st32(to + c * 32, o);
                            }
                        }
                    }
                    const float off = kLift - (m == -INFINITY ? 0.f : m);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float s[32];
                        umma::ld32(ts + c * 32, s);
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (c * 32 + i > hi || c * 32 + i <= lo) s[i] = -INFINITY;
                        }
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float x0 = exp2_fast(fmaf(s[2 * i], fac, off)), x1 = exp2_fast(fmaf(s[2 * i + 1], fac, off));
                            l += x0 + x1;
                            p[i] = pack_f16(x0, x1);
                        }
                        // the weights take columns of S that this warp has read
                        st16(ts + c * 16, p);
                    }
                    wait_st();
                    umma::fence_before();
                    arrive(bar(C::b_p_full + b));
                }
                if (it.last > it.first) {
                    if (!wait(C::b_o_done + (QT == 2 ? t : 0), n - 1)) return;
                    umma::fence_after();
                }
                const bool none = it.last == it.first || (m == -INFINITY && l == 0.f);
                if (it.whole()) {
                    const float inv = none ? 0.f : (a.v_scale ? a.v_scale[it.h] : 1.f) / l;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        if (it.last > it.first) umma::ld32(to + c * 32, o);
                        if (valid) {
                            uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + head * D + c * 32);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t u[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const __nv_bfloat162 y = __floats2bfloat162_rn(none ? 0.f : o[8 * i + 2 * j] * inv,
                                                                                   none ? 0.f : o[8 * i + 2 * j + 1] * inv);
                                    u[j] = *reinterpret_cast<const uint32_t *>(&y);
                                }
                                p[i] = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        }
                    }
                    if (valid && a.lse) a.lse[head] = none ? -INFINITY : (m + log2f(l) - kLift) * kLn2;
                } else {
                    const int part = it.starts() ? 1 : 0;
                    float *w = a.parts + ((size_t)me * 2 + part) * ((size_t)C::ROWS * (D + 2));
                    if (valid) {
                        w[my] = none ? -INFINITY : m;
                        w[C::ROWS + my] = l;
                    }
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        if (it.last > it.first) umma::ld32(to + c * 32, o);
                        if (valid) {
                            float4 *p = reinterpret_cast<float4 *>(w + 2 * C::ROWS + (size_t)my * D + c * 32);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                p[i] = none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                            : make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                    }
                    if (part == 1) job = make_int4(it.r, it.h, it.rt, it.last_worker);
                }
                // the reads of O come before the next row tile's products (released by its first weights)
                umma::fence_before();
            }
        };
        work();
        if (tid == 0) a.jobs[me] = misc[1] ? make_int4(-1, 0, 0, 0) : job;
    } else if (warp < C::SOFT + C::DEQ) {
        // ------------------------------------------------------------ dequant
        const int d = tid - C::SOFT * 32;  // 0 .. 255
        uint32_t n = 0, raws = 0;
        auto work = [&]() {
            while (walk.next(a, it)) {
                for (int tile = it.first; tile < it.last; ++tile, ++n) {
                    const uint32_t ks = sb + C::off_k + (n & 1) * C::OPERAND, vs = sb + C::off_v + (n & 1) * C::OPERAND;
                    if (!wait(C::b_k_empty + (n & 1), (n >> 1) + 1)) return;
                    // keys: four lanes per key, lane g the channel groups g and (d = 128) g + 4
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t ri = (raws + half) % C::RAWS;
                        if (!wait(C::b_raw_full + ri, (raws + half) / C::RAWS)) return;
                        const uint32_t raw = sb + C::off_raw + ri * C::RAW;
#pragma unroll
                        for (int i = 0; i < D / 64 * (8 / C::DEQ); ++i) {
                            const int key = (d >> 2) + i / (D / 64) * (8 * C::DEQ), grp = (d & 3) + 4 * (i % (D / 64));
                            const int blk = key >> 4, tok = key & 15, kk = half * 64 + key;
                            const uint2 w = lds64(raw + blk * BB + tok * (D / 2) + grp * 8);
                            const uint32_t f = scale_pair(lds8(raw + blk * BB + off_ks(D) + tok * (D / 16) + grp));
                            convert(w, f, ks + umma::kmaj(kk, grp * 16, 128), ks + umma::kmaj(kk, grp * 16 + 8, 128));
                        }
                    }
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) arrive(bar(C::b_k_full + (n & 1)));
                    // values: sixteen lanes per block and group, one key each
                    if (!wait(C::b_v_empty + (n & 1), (n >> 1) + 1)) return;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t ri = (raws + half) % C::RAWS;
                        const uint32_t raw = sb + C::off_raw + ri * C::RAW;
#pragma unroll
                        for (int i = 0; i < D / 64 * (8 / C::DEQ); ++i) {
                            const int pair = (d >> 4) + 2 * C::DEQ * i, tok = d & 15;
                            const int blk = pair / (D / 16), grp = pair % (D / 16);
                            const int kk = half * 64 + blk * 16 + tok;
                            const uint2 w = lds64(raw + blk * BB + off_vc(D) + grp * 128 + tok * 8);
                            uint32_t f = scale_pair(lds8(raw + blk * BB + off_vs(D) + grp * 16 + tok));
                            // past the end the bytes are anything, NaN scales too: a zero weight does not undo that
                            if (tile * kTile + kk >= it.q.len) f = 0;
                            convert(w, f, vs + umma::mnmaj(grp * 16, kk, D / 64), vs + umma::mnmaj(grp * 16 + 8, kk, D / 64));
                        }
                        __syncwarp();
                        if (lane == 0) arrive(bar(C::b_raw_empty + ri));
                    }
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) arrive(bar(C::b_v_full + (n & 1)));
                    raws += 2;
                }
            }
        };
        work();
    } else if (warp == C::SOFT + C::DEQ) {
        // ------------------------------------------------------------ producer
        uint32_t raws = 0;
        const int chunk = a.page_shift < 6 ? 1 << (a.page_shift - 4) : 4;  // blocks per copy
        auto work = [&]() {
            while (walk.next(a, it)) {
                const int32_t *table = a.block_table + (size_t)it.r * a.max_pages;
                for (int tile = it.first; tile < it.last; ++tile)
                    for (int half = 0; half < 2; ++half, ++raws) {
                        const uint32_t ri = raws % C::RAWS;
                        const int key = tile * kTile + half * 64 + lane * chunk * 16;
                        // blocks of this lane's copy that hold keys
                        const int left = (it.q.len - key + 15) >> 4;
                        const int mine = lane * chunk < 4 ? min(max(left, 0), chunk) : 0;
                        int page = 0;
                        if (mine > 0) {
                            page = __ldg(table + (key >> a.page_shift));
                            if (page < 0 || page >= a.num_pages) {
                                page = 0;
                                if (a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
                            }
                        }
                        const int all = __reduce_add_sync(0xffffffffu, mine);
                        if (!wait(C::b_raw_empty + ri, raws / C::RAWS + 1)) return;
                        if (lane == 0) umma::mbar_expect_tx(bar(C::b_raw_full + ri), all * BB);
                        __syncwarp();
                        if (mine > 0) {
                            const int blk = (key & ((1 << a.page_shift) - 1)) >> 4;
                            const uint8_t *src = a.cache + ((((size_t)page * a.Hkv + it.h) << (a.page_shift - 4)) + blk) * BB;
                            umma::bulk_load(sb + C::off_raw + ri * C::RAW + lane * chunk * BB, src, mine * BB,
                                            bar(C::b_raw_full + ri));
                        }
                    }
            }
        };
        work();
        if (misc[1]) {
            // copies in flight end before the CTA leaves
            for (uint32_t i = raws > C::RAWS ? raws - C::RAWS : 0; i < raws; ++i)
                umma::mbar_wait(bar(C::b_raw_full + i % C::RAWS), (i / C::RAWS) & 1, kWaitLimit);
        }
    } else if (lane == 0) {
        // ------------------------------------------------------------ products
        constexpr uint32_t id_s = idesc_f16(128, 128, 0), id_o = idesc_f16(128, D, 1);
        const uint32_t sb4 = sb >> 4;
        uint32_t n = 0, items = 0;
        auto scores = [&](int t, uint32_t tile, int b) {
            const uint32_t q4 = sb4 + ((C::off_q + t * C::OPERAND) >> 4), k4 = sb4 + ((C::off_k + (tile & 1) * C::OPERAND) >> 4);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                umma::mma(tmem + b * 128, umma::sdesc4(q4 + o, 16, 1024), umma::sdesc4(k4 + o, 16, 1024), id_s, ks > 0);
            }
            umma::commit(bar(C::b_s_full + b));
        };
        auto values = [&](int t, uint32_t tile, int b, bool acc) {
            const uint32_t v4 = sb4 + ((C::off_v + (tile & 1) * C::OPERAND) >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_ts(tmem + C::t_o + t * D, tmem + b * 128 + ks * 8,
                       umma::sdesc4(v4 + ((ks * 16 * D * 2) >> 4), 1024, 16 * D), id_o, acc || ks > 0);
            umma::commit(bar(C::b_o_done + t));
        };
        auto work = [&]() {
            while (walk.next(a, it)) {
                const int tiles = it.last - it.first;
                if (tiles == 0) continue;
                if (!wait1(C::b_q_full, items++)) return;
                if (!wait1(C::b_k_full + (n & 1), n >> 1)) return;
                umma::fence_after();
                for (int t = 0; t < QT; ++t) scores(t, n, QT == 2 ? t : n & 1);
                umma::commit(bar(C::b_k_empty + (n & 1)));
                for (int j = 0; j < tiles; ++j, ++n) {
                    if (QT == 1 && j + 1 < tiles) {
                        if (!wait1(C::b_k_full + ((n + 1) & 1), (n + 1) >> 1)) return;
                        umma::fence_after();
                        scores(0, n + 1, (n + 1) & 1);
                        umma::commit(bar(C::b_k_empty + ((n + 1) & 1)));
                    }
                    for (int t = 0; t < QT; ++t) {
                        const int b = QT == 2 ? t : n & 1;
                        if (t == 0 && !wait1(C::b_v_full + (n & 1), n >> 1)) return;
                        if (!wait1(C::b_p_full + b, QT == 2 ? n : n >> 1)) return;
                        umma::fence_after();
                        values(t, n, b, j > 0);
                        if (QT == 2 && j + 1 < tiles) {
                            if (t == 0 && !wait1(C::b_k_full + ((n + 1) & 1), (n + 1) >> 1)) return;
                            umma::fence_after();
                            scores(t, n + 1, t);
                        }
                    }
                    umma::commit(bar(C::b_v_empty + (n & 1)));
                    if (QT == 2 && j + 1 < tiles) umma::commit(bar(C::b_k_empty + ((n + 1) & 1)));
                }
            }
        };
        work();
        // products in flight end before the CTA leaves
        umma::commit(bar(C::b_drain));
        umma::mbar_wait(bar(C::b_drain), 0, kWaitLimit);
    }
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
}

template <int D, int QT>
cudaError_t launch(const Cache4AttnArgs &a, int sms, cudaStream_t st) {
    auto kernel = cache4_attn_tc_kernel<D, QT>;
    constexpr int bytes = Cfg<D, QT>::SMEM;
    static_assert(bytes <= 232448, "shared memory of one CTA");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<sms, Cfg<D, QT>::THREADS, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t cache4_attn_tc_workspace(int sms, int d) {
    return (size_t)sms * (sizeof(int4) + 2 * 256 * (size_t)(d + 2) * sizeof(float));
}

// two row tiles at a time when a request may have more than 128 rows
cudaError_t launch_cache4_attn_tc(const Cache4AttnArgs &a, int d, long long rows, int sms, cudaStream_t st) {
    if (rows > 128) return d == 128 ? launch<128, 2>(a, sms, st) : launch<64, 2>(a, sms, st);
    return d == 128 ? launch<128, 1>(a, sms, st) : launch<64, 1>(a, sms, st);
}
cudaError_t launch_cache4_merge_tc(const Cache4AttnArgs &a, int d, long long rows, int sms, cudaStream_t st) {
    if (rows > 128)
        return d == 128 ? merge_shares<128, 256, kTile, false>(a, sms, kLift, st)
                        : merge_shares<64, 256, kTile, false>(a, sms, kLift, st);
    return d == 128 ? merge_shares<128, 128, kTile, false>(a, sms, kLift, st)
                    : merge_shares<64, 128, kTile, false>(a, sms, kLift, st);
}

}  // namespace kda
