// cache4_attn_tc.cu -- attention over the 4-bit pages for many rows per key
// head (verify windows of wide groups, prompt chunks): tcgen05 products.
//
// Same operator and division of the work as cache4_attn.cu, with row tiles of
// QT x 128 rows and key tiles of 128.  One persistent CTA per SM, warps by
// role:
//   softmax    8 warps  a thread per row of one of two score tiles: maximum,
//                       weights (f16, lifted by 2^kLift), sum, and the
//                       accumulator's rescaling; the epilogue
//   dequant    4 or 8   half for the keys and half for the values: codes and
//                       scales -> f16 (exact), into the swizzled shared-
//                       memory operands K (K-major) and V (N-major)
//   producer   1 warp   bulk copies of 64 (QT = 1: 128) keys at a time into a raw ring
//   products   1 warp   S = Q K^T into tensor memory, O += P V with P read
//                       from tensor memory (it takes the place of S)
//   queries    2 warps  QT = 1: the next item's query rows, scaled, as f16
//                       (QT = 2: the softmax threads, a row each)
// There are two score tiles S and two accumulators O in tensor memory (all
// 512 columns at d = 128).  With QT = 2 they belong to two row tiles, whose
// products and softmax take turns.  With QT = 1 (up to 128 rows) they belong
// to the even and the odd key tiles of the one row tile: two streams with
// maximum, sum and accumulator of their own, joined at the item's end.
//
// The running maximum that the weights refer to moves only when it would rise
// by more than 2^8, so the accumulator is rescaled a few times per item; f16
// holds the weights of up to 2^15 that this allows.
//
// What bounds it.  The products take 1,028 cycles of the tensor pipe per 128
// rows x 128 keys at d = 128.  QT = 2: a row tile's chain (its products, the
// scores' way to registers, weights, O, next scores) is longer than the other
// tile's products hide: about 2,800 cycles per 256 rows x 128 keys where the
// pipe wants 2,056.  632 GFLOP of prompt chunks (2 x 2,048 queries of 32
// heads over up to 16K keys), by call: 430 us with the join, 1.47 PFLOP/s,
// 76 % of the measured bf16 rate; 371 without the softmax, 391 without the
// conversion, 366 without both.  QT = 1: a key tile's conversion serves up to
// 128 rows only, and it and the two streams' softmax share the SM's issue
// slots beside products that the padded row tile makes as long as a full
// one's.  64 requests of up to 8 queries x 96 heads (752 MB, a third of it by
// the other kernel, 90 us alone): 277 us, 40 % of the measured copy bandwidth; 263
// without the softmax, 255 without the conversion, 230 without both, which is
// the pipe's time.  Memory bounds neither: copies taken out gain nothing.
//
// Measured on the way (us, the two calls above): one thread issuing the
// products from a divergent branch, operands moved to uniform registers for
// each, 591 / 451, the whole warp with an elected lane 483 / 420; one stream
// for QT = 1 420, two 352; the roles' loops unrolled, with instruction
// fetch the first cause of stalls, 997 / 817, rolled up 597 / 463; the maximum formed by the
// tensor-memory load instead of by the threads 480 / 306 to 466 / 302; QT =
// 2's registers shared out 176 / 96 / 64 (144 bytes spilled) 466, 192 / 72 /
// 56 437, 200 / 64 / 48 (4 bytes) 428, 208 / 48 / 48 435; raw stages of 128
// keys for QT = 1, with half of the waits of those of 64, 295 to 279.  Slower and left
// out: copies of keys and values apart (1,152 bytes each) 406 for QT = 1;
// half of a row's scores kept from maximum to weights for QT = 1, 312; the
// accumulator rescaled after the first weights instead of before them 441 for
// QT = 2; one arrival per warp instead of per thread 437 for QT = 2.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache4.cuh"
#include "cache4_sched.cuh"
#include "kda_internal.h"
#include "kda_umma.cuh"

namespace kda {
namespace {

using namespace cache4;

constexpr int kTile = ManyRows::TILE;    // keys per tile
constexpr int kLead = ManyRows::LEAD;    // an item's start and end, in tiles
// The first wait for scores: a test build (KDA_TEST_SHORT_FIRST_WAIT) gives up on it
// at once, to exercise the way out.
#ifdef KDA_TEST_SHORT_FIRST_WAIT
constexpr uint32_t kFirstWait = 0;
#else
constexpr uint32_t kFirstWait = kWaitLimit;
#endif
constexpr float kLift = ManyRows::LIFT;  // weights are at most 2^(kLift + kSlack)
constexpr float kSlack = 8.f;

template <int D, int QT>
struct Cfg {
    // Whole warpgroups by role, whose registers are shared out anew at the start:
    // a CTA of 16 warps is launched with 128 a thread, one of 20 with 96.  With
    // two row tiles a softmax thread holds its row's 128 scores; with one
    // there is half as much to weigh per key, and conversion gets two warpgroups.
    static constexpr int SOFT = 8, DEQ = QT == 2 ? 4 : 8, WARPS = SOFT + DEQ + 4, THREADS = WARPS * 32;
    static constexpr int R_LAUNCH = QT == 2 ? 128 : 96;
    static constexpr int R_SOFT = QT == 2 ? 200 : 128, R_DEQ = QT == 2 ? 64 : 72, R_MISC = QT == 2 ? 48 : 80;
    // the others give up what the softmax warpgroups take, and nobody waits for more than there is
    static_assert(R_SOFT >= R_LAUNCH && R_DEQ <= R_LAUNCH && R_MISC <= R_LAUNCH, "who takes and who gives registers");
    static_assert(SOFT / 4 * R_SOFT + DEQ / 4 * R_DEQ + R_MISC <= WARPS / 4 * R_LAUNCH, "registers of the CTA");
    static constexpr int ROWS = 128 * QT;
    static constexpr int OPERAND = 128 * D * 2;       // 128 rows of f16
    static constexpr int KEYS = QT == 2 ? 64 : 128;   // keys of a raw stage
    static constexpr int RAW = KEYS / 16 * block_bytes(D), RAWS = 3;
    static constexpr int off_q = 0, off_k = QT * OPERAND, off_v = off_k + 2 * OPERAND, off_raw = off_v + 2 * OPERAND;
    static constexpr int off_bar = off_raw + RAWS * RAW;
    // barriers: raw full / empty, K and V full / empty, S full, P full (two halves), O done, Q full /
    // empty, O free, the two streams' exchange, drain
    static constexpr int b_raw_full = 0, b_raw_empty = RAWS, b_k_full = 2 * RAWS, b_k_empty = b_k_full + 2,
                         b_v_full = b_k_full + 4, b_v_empty = b_k_full + 6, b_s_full = b_k_full + 8,
                         b_p_full = b_k_full + 10, b_o_done = b_k_full + 14, b_q_full = b_k_full + 16,
                         b_q_empty = b_k_full + 17, b_o_free = b_k_full + 18, b_pair = b_k_full + 19,
                         b_drain = b_k_full + 20, BARS = b_k_full + 21;
    static constexpr int off_misc = off_bar + BARS * 8;  // TMEM address, dead flag
    // QT = 1: maxima and sums of the two streams, in two places that items take in turn: a stream without a tile
    // of the next item waits for nothing before it writes that item's, and the other may still be reading
    static constexpr int PAIR_PLACES = 2;
    static constexpr int off_ml = off_misc + 16;
    static constexpr int off_fac = off_ml + (QT == 1 ? PAIR_PLACES * 2 * 128 * 8 : 0);  // factors of the rows' scores, two items
    static constexpr int off_item = (off_fac + (QT == 1 ? 2 * ROWS * 4 : 0) + 15) & ~15;  // the softmax warps' place in the work
    static constexpr int SMEM = off_item + SOFT * 176;
    // tensor memory columns: S (and P over it) 2 x 128, O 2 x D
    static constexpr int t_o = 256;
};

__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Products and commits are written for a whole warp that runs convergent, with
// one lane (elect.sync) issuing: operands that the compiler knows to be
// uniform sit in uniform registers, which the instruction takes, instead of
// being moved there for every product (about 100 cycles each from a branch of
// one thread).
__device__ __forceinline__ uint32_t elect() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n.reg .pred pp, e;\nsetp.ne.b32 e, %5, 0;\nsetp.ne.b32 pp, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, pp;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead));
}
// A in tensor memory (f16, two consecutive K per column, the lower one in the low half)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t lead) {
    asm volatile(
        "{\n.reg .pred pp, e;\nsetp.ne.b32 e, %5, 0;\nsetp.ne.b32 pp, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pp;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead));
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
    asm volatile(
        "{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"(lead)
        : "memory");
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// 32 consecutive columns of this thread's tensor memory lane, without the wait:
// several loads go out together, then umma::wait_ld() and hold() on each array
__device__ __forceinline__ void ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ld16_async(uint32_t taddr, float (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void hold16(float (&r)[16]) {
    asm volatile(""
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]),
                   "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void hold(uint32_t (&r)[32]) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
          "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
          "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
          "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) : : "memory");
}

// the same, and their largest (NaN where all are, as fmaxf): the load forms it on its way
__device__ __forceinline__ void ld32_max_async(uint32_t taddr, uint32_t (&r)[32], float &top) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=f"(top)
        : "r"(taddr)
        : "memory");
}

// 32 N scores of this thread's row; returns their largest
template <int N>
__device__ __forceinline__ float load_scores(uint32_t taddr, uint32_t (&s)[N][32]) {
    float top[N];
#pragma unroll
    for (int c = 0; c < N; ++c) ld32_max_async(taddr + c * 32, s[c], top[c]);
    umma::wait_ld();
#pragma unroll
    for (int c = 0; c < N; ++c) {
        hold(s[c]);
        asm volatile("" : "+f"(top[c]) : : "memory");
    }
#pragma unroll
    for (int c = 1; c < N; ++c) top[0] = fmaxf(top[0], top[c]);
    return top[0];
}
__device__ __forceinline__ void st32b(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void st16_async(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
    st16_async(taddr, r);
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
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

// A query row goes in scaled by a power of two that brings its largest element
// to [2^8, 2^9), as f16; its scores get the inverse and the softmax scale as a
// factor.  The sign of the scale (a zero and NaN as well) goes into the row, so
// that the factor is positive and may follow the maximum.
__device__ __forceinline__ uint32_t magnitude(const uint4 &w) {  // of eight bf16, which orders as an integer
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max((u[j] << 16) & 0x7fffffffu, u[j] & 0x7fff0000u));
    return top;
}
__device__ __forceinline__ int exponent(uint32_t top) { return min(max((int)(top >> 23), 9), 253); }
__device__ __forceinline__ float scale_up(float base, int ex) {
    return (base < 0.f ? -1.f : base > 0.f ? 1.f : base) * __uint_as_float((uint32_t)(262 - ex) << 23);
}
__device__ __forceinline__ float factor(float base, int ex) {
    return fmaxf(fabsf(base) * __uint_as_float((uint32_t)(ex - 8) << 23), 1e-37f);
}
__device__ __forceinline__ void store_query(uint32_t addr, const uint4 &w, float up) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pack_f16(__uint_as_float(u[j] << 16) * up, __uint_as_float(u[j] & 0xffff0000u) * up);
    sts128(addr, f[0], f[1], f[2], f[3]);
}

template <int D, int QT>
__global__ void __launch_bounds__((Cfg<D, QT>::THREADS), 1)
kda_cache4_attn_tc_kernel(const Cache4AttnArgs a) {
    using C = Cfg<D, QT>;
    constexpr int BB = block_bytes(D), KS = D / 16;
    extern __shared__ __align__(1024) unsigned char smem[];
    const uint32_t sb = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = a.Hq / a.Hkv;
    auto bar = [&](int i) { return sb + C::off_bar + i * 8; };
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + C::off_misc);

    allow_dependents();
    if (tid == 0) {
        for (int i = 0; i < C::RAWS; ++i) {
            umma::mbar_init(bar(C::b_raw_full + i), 1);
            umma::mbar_init(bar(C::b_raw_empty + i), C::DEQ);
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(bar(C::b_k_full + i), C::DEQ / 2);
            umma::mbar_init(bar(C::b_k_empty + i), 1);
            umma::mbar_init(bar(C::b_v_full + i), C::DEQ / 2);
            umma::mbar_init(bar(C::b_v_empty + i), 1);
            umma::mbar_init(bar(C::b_s_full + i), 1);
            umma::mbar_init(bar(C::b_p_full + 2 * i), 128);
            umma::mbar_init(bar(C::b_p_full + 2 * i + 1), 128);
            umma::mbar_init(bar(C::b_o_done + i), 1);
        }
        umma::mbar_init(bar(C::b_q_full), QT == 2 ? 256 : 64);
        umma::mbar_init(bar(C::b_q_empty), 1);
        umma::mbar_init(bar(C::b_o_free), 256);
        umma::mbar_init(bar(C::b_drain), 1);
        umma::mbar_init(bar(C::b_pair), 256);
        misc[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) umma::tmem_alloc(sb + C::off_misc, 512);
    Walk<C::ROWS, kTile, kLead> walk(a);
    const int me = blockIdx.x;
    walk.begin(a, reinterpret_cast<long long *>(smem), me, gridDim.x);
    umma::fence_before();
    __syncthreads();  // barriers, the tensor memory address, and the prefix (over the operands) has been read
    umma::fence_after();
    const uint32_t tmem = misc[0];

    // a bounded wait that gives up when any role has; `wait` for whole warps,
    // whose lanes then agree
    auto wait1 = [&](int i, uint32_t parity, uint32_t limit = kWaitLimit) {
#pragma unroll 1
        for (uint32_t n = 0; n < limit; n += 4096) {
            if (poll(bar(i), parity & 1, 4096)) return true;
            if (misc[1]) return false;
        }
        misc[1] = 1;
        return false;
    };
    auto wait = [&](int i, uint32_t parity, uint32_t limit = kWaitLimit) {
        return __all_sync(0xffffffffu, wait1(i, parity, limit)) != 0;
    };

    Item it;
    if (warp < C::SOFT) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::R_SOFT));
        // ------------------------------------------------------------ softmax: a thread per row of a score tile
        // scores per load: a load from tensor memory takes about 200 cycles beside the products, however wide
        constexpr int CHUNK = QT == 2 ? 128 : 64;
        const int t = warp >> 2, lane_base = (warp & 3) * 32, r = lane_base + lane, my = (QT == 2 ? t * 128 : 0) + r;
        const uint32_t tq = tmem + ((uint32_t)lane_base << 16), ts = tq + t * 128, to = tq + C::t_o + t * D;
        uint32_t n = 0, mine = 0, items = 0;  // key tiles so far, those of this stream, items with key tiles
        // The place in the work lives in shared memory, a copy per warp: its
        // twenty-odd registers are needed between items only.
        struct Place {
            Walk<C::ROWS, kTile, kLead> walk;
            Item it;
            int4 job;
            int more;
        };
        static_assert(sizeof(Place) <= 176, "room of a warp's place");
        Place &at = *reinterpret_cast<Place *>(smem + C::off_item + warp * 176);
        if (lane == 0) {
            at.walk = walk;
            at.job = make_int4(-1, 0, 0, 0);
        }
        auto work = [&]() {
            while (true) {
                __syncwarp();
                if (lane == 0) {
                    Walk<C::ROWS, kTile, kLead> w = at.walk;
                    Item next;
                    at.more = w.next(a, next);
                    at.it = next;
                    if (at.more && next.starts && !next.ends) at.job = make_int4(next.r, next.h, next.rt, w.last_worker());
                    at.walk = w;
                }
                __syncwarp();
                if (!at.more) break;
                const int tile0 = at.it.first, tile1 = at.it.last;
                const bool some = tile1 > tile0;
                const int rows = at.walk.q.rows, rr = at.it.row0 + my, tok = min(rr, rows - 1) / G;
                const bool valid = rr < rows, idle = rr - lane >= rows;
                float m = -INFINITY, l = 0.f, fac = 1.f;
                if (QT == 2 && some) {
                    // this thread's query row (its score tile's last products have read the row before)
                    const float base = a.scale * kLog2e * (a.k_scale ? a.k_scale[at.it.h] : 1.f);
                    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                                     (size_t)(at.walk.q.q0 + tok) * a.q_stride +
                                                                     (size_t)(at.it.h * G + (valid ? rr % G : 0)) * D);
                    uint4 w[D / 8];
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) w[i] = __ldg(p + i);
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) top = max(top, magnitude(w[i]));
                    const int ex = exponent(top);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        store_query(sb + C::off_q + t * C::OPERAND + umma::kmaj(r, i * 8, 128), w[i],
                                    valid ? scale_up(base, ex) : 0.f);
                    fac = factor(base, ex);
                    umma::fence_proxy_async();
                    arrive(bar(C::b_q_full));
                }
                // positions this row sees (a padding row sees what the last row does), and what the whole warp sees
                const int sees = at.walk.q.len - at.walk.q.n + tok;
                const int see_lo = __reduce_min_sync(0xffffffffu, sees), see_hi = __reduce_max_sync(0xffffffffu, sees);
                bool begun = false;
#pragma unroll 1
                for (int tile = tile0; tile < tile1; ++tile, ++n) {
                    if (QT == 1 && (int)(n & 1) != t) continue;
                    if (!wait(C::b_s_full + t, mine++, n == 0 ? kFirstWait : kWaitLimit)) return;
                    umma::fence_after();
                    if (idle) {
                        // no row of this warp is there: its weights may be anything (rows do not mix)
                        umma::fence_before();
                        arrive(bar(C::b_p_full + 2 * t));
                        arrive(bar(C::b_p_full + 2 * t + 1));
                        continue;
                    }
                    const int key0 = tile * kTile;
                    if (key0 > see_lo + 1 - kTile || (a.window > 0 && key0 <= see_hi - a.window)) {
                        // hidden columns become -inf where they are; few tiles have any
                        const int hi = sees - key0, lo = a.window > 0 ? hi - a.window : -1;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t s[32];
                            ld32_async(ts + c * 32, s);
                            umma::wait_ld();
                            hold(s);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i > hi - c * 32 || i <= lo - c * 32) s[i] = 0xff800000u;
                            st32b(ts + c * 32, s);
                        }
                        wait_st();
                    }
                    uint32_t s[CHUNK / 32][32];
                    float off;
                    // where the maximum is far from zero it is taken from the scores in tensor memory, and they are loaded again
#pragma unroll 1
                    for (bool lowered = false;; lowered = true) {
                        float top = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 128 / CHUNK; ++c) top = fmaxf(top, load_scores(ts + c * CHUNK, s));
                        if (lowered) break;
                        // (the scores that have arrived came after the queries and their factors)
                        if (QT == 1 && !begun)
                            fac = reinterpret_cast<volatile float *>(smem + C::off_fac)[(items & 1) * C::ROWS + my];
                        if (!begun) m = top;
                        begun = true;
                        const bool rise = (top - m) * fac > kSlack;  // (false where both are -inf)
                        const float low = scaled(m == -INFINITY ? 0.f : m, fac);
                        off = kLift - low;
                        if (!__any_sync(0xffffffffu, rise || fabsf(low) >= kFar)) break;
                        // (this stream's last product onto O came before the scores that have arrived)
                        if (__any_sync(0xffffffffu, rise)) {
                            const float f = rise ? exp2_fast(scaled(m, fac) - scaled(top, fac)) : 1.f;
                            l *= f;
                            if (rise) m = top;
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                float o[16];
                                umma::ld16(to + c * 16, o);
                                uint32_t u[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * f);
                                st16(to + c * 16, u);
                            }
                        }
                        const float ref = m == -INFINITY ? 0.f : m;
                        const bool big = fabsf(scaled(ref, fac)) >= kFar;
                        off = kLift - (big ? 0.f : scaled(ref, fac));
                        if (!__any_sync(0xffffffffu, big)) break;
                        const float sub = big ? ref : 0.f;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t v[32];
                            ld32_async(ts + c * 32, v);
                            umma::wait_ld();
                            hold(v);
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) - sub);
                            st32b(ts + c * 32, v);
                        }
                        wait_st();
                        if (QT == 1) break;
                    }
                    const float2 fac2 = make_float2(fac, fac), off2 = make_float2(off, off);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    // the weights take the place of columns of S that have been read; the products may start on the
                    // first half
                    auto weights = [&](int column, const uint32_t(&v)[32]) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 y =
                                __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), fac2, off2);
                            const float2 e = make_float2(exp2_fast(y.x), exp2_fast(y.y));
                            sum[i & 1] = __fadd2_rn(sum[i & 1], e);
                            p[i] = pack_f16(e.x, e.y);
                        }
                        st16_async(ts + column, p);
                    };
                    auto release = [&](int half) {
                        wait_st();
                        umma::fence_before();
                        arrive(bar(C::b_p_full + 2 * t + half));
                    };
                    if constexpr (QT == 2) {
                        weights(0, s[0]);
                        weights(16, s[1]);
                        release(0);
                        weights(32, s[CHUNK / 32 - 2]);
                        weights(48, s[CHUNK / 32 - 1]);
                        release(1);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            load_scores(ts + c * 64, s);
                                weights(c * 32, s[0]);
                            weights(c * 32 + 16, s[1]);
                            release(c);
                        }
                    }
                    sum[0] = __fadd2_rn(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                }
                m = scaled(m, fac);
                if (some) {
                    if (mine > 0 && !wait(C::b_o_done + t, mine - 1)) return;
                    umma::fence_after();
                }
                // with one row tile the streams' results are joined: each takes half the channels
                float fo[2] = {1.f, 1.f};
                if (QT == 1 && some) {
                    volatile float2 *ml =
                        reinterpret_cast<volatile float2 *>(smem + C::off_ml) + items % C::PAIR_PLACES * (2 * 128);
                    ml[t * 128 + r].x = m;
                    ml[t * 128 + r].y = l;
                    umma::fence_before();
                    arrive(bar(C::b_pair));
                    if (!wait(C::b_pair, items)) return;
                    umma::fence_after();
                    const float m0 = ml[r].x, m1 = ml[128 + r].x, l0 = ml[r].y, l1 = ml[128 + r].y;
                    // (a stream writes here again two items on, which takes the other's arrival for the item between)
                    m = fmaxf(m0, m1);
                    const float ref = m == -INFINITY ? 0.f : m;
                    fo[0] = exp2_fast(m0 - ref), fo[1] = exp2_fast(m1 - ref);
                    l = fo[0] * l0 + fo[1] * l1;
                    // a stream without a tile has no sum in tensor memory
                    if (tile1 - tile0 == 1) fo[((n - 1) & 1) ^ 1] = -1.f;
                }
                const bool none = !some || sees < 0;
                const bool whole = at.it.whole();
                const float f = none ? 0.f : whole ? (a.v_scale ? a.v_scale[at.it.h] : 1.f) / l : 1.f;
                const int row = at.it.row0 + my, token = row / G;
                const size_t head = (size_t)(at.walk.q.q0 + token) * a.Hq + at.it.h * G + (row - token * G);
                float *part = a.parts + ((size_t)me * 2 + (at.it.starts ? 1 : 0)) * ((size_t)C::ROWS * (D + 2));
                if (valid && whole && a.lse) a.lse[head] = none ? -INFINITY : (m + log2f(l) - kLift) * kLn2;
                if (valid && !whole) {
                    part[my] = none ? -INFINITY : m;
                    part[C::ROWS + my] = l;
                }
                char *dst = whole ? reinterpret_cast<char *>(static_cast<__nv_bfloat16 *>(a.o) + head * D)
                                  : reinterpret_cast<char *>(part + 2 * C::ROWS + (size_t)my * D);
#pragma unroll 1
                for (int c = QT == 2 ? 0 : t * (D / 32); c < (QT == 2 ? D / 16 : (t + 1) * (D / 32)); ++c) {
                    float o[16];
                    if (QT == 2) {
                        if (some) umma::ld16(to + c * 16, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = none ? 0.f : o[i] * f;
                    } else {
                        float y[16];
                        if (some) {
                            ld16_async(tq + C::t_o + c * 16, o);
                            ld16_async(tq + C::t_o + D + c * 16, y);
                            umma::wait_ld();
                            hold16(o);
                            hold16(y);
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y0 = fo[0] == -1.f ? 0.f : o[i] * fo[0], y1 = fo[1] == -1.f ? 0.f : y[i] * fo[1];
                            o[i] = none ? 0.f : (y0 + y1) * f;
                        }
                    }
                    if (valid && whole) {
                        uint4 *p = reinterpret_cast<uint4 *>(dst) + c * 2;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * i + 2 * j], o[8 * i + 2 * j + 1]);
                                u[j] = *reinterpret_cast<const uint32_t *>(&y);
                            }
                            p[i] = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    } else if (valid) {
                        float4 *p = reinterpret_cast<float4 *>(dst) + c * 4;
#pragma unroll
                        for (int i = 0; i < 4; ++i) p[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                // the reads of O come before the next item's products: those of a row tile of two follow the
                // weights of its own warps, those of two streams wait until both streams have read
                umma::fence_before();
                if (some) {
                    if (QT == 1) arrive(bar(C::b_o_free));
                    ++items;
                }
            }
        };
        work();
        if (tid == 0) a.jobs[me] = misc[1] ? make_int4(-1, 0, 0, 0) : at.job;
    } else if (warp < C::SOFT + C::DEQ) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::R_DEQ));
        // ------------------------------------------------------------ dequant
        const int d = tid - C::SOFT * 32;
        constexpr int NK = D / 64, NG = D / 16, BATCH = 4;
        constexpr int THR = C::DEQ * 16;                   // threads for the keys, and as many for the values
        const bool for_keys = d < THR;
        const int e = for_keys ? d : d - THR;
        // Keys: four lanes per key; lane g takes the channel groups g and (d =
        // 128) g + 4, so the eight lanes of a 128-byte store row write eight
        // different chunks.
        constexpr int K_ROWS = THR / 4, K_STEPS = C::KEYS / K_ROWS * NK;       // keys per pass; conversions per stage
        // Values: sixteen lanes per block and group, a key each.
        constexpr int PAIRS = THR / 16, V_STEPS = C::KEYS / 16 * NG / PAIRS;         // (block, group) pairs per pass
        constexpr int SPLIT = NG > PAIRS ? NG / PAIRS : 1;                // passes over the groups of a block
        constexpr int V_BLKS = PAIRS > NG ? PAIRS / NG : 1;               // blocks per pass
        uint32_t codes, scale, out0, out1;
        int blk_key;  // key of the first conversion in its stage
        if (for_keys) {
            const int key = e >> 2, g = e & 3;
            codes = (key >> 4) * BB + (key & 15) * (D / 2) + g * 8;
            scale = (key >> 4) * BB + off_ks(D) + (key & 15) * NG + g;
            out0 = umma::kmaj(key, g * 16, 128), out1 = umma::kmaj(key, g * 16 + 8, 128);
            blk_key = key;
        } else {
            const int tok = e & 15, grp = (e >> 4) % NG, blk = (e >> 4) / NG;
            codes = blk * BB + off_vc(D) + grp * 128 + tok * 8;
            scale = blk * BB + off_vs(D) + grp * 16 + tok;
            out0 = umma::mnmaj(grp * 16, blk * 16 + tok, NK), out1 = umma::mnmaj(grp * 16 + 8, blk * 16 + tok, NK);
            blk_key = blk * 16 + tok;
        }
        const int b_empty = for_keys ? C::b_k_empty : C::b_v_empty, b_full = for_keys ? C::b_k_full : C::b_v_full;
        uint32_t n = 0, raws = 0;
        auto work = [&]() {
            while (walk.next(a, it)) {
#pragma unroll 1
                for (int tile = it.first; tile < it.last; ++tile, ++n) {
                    if (!wait(b_empty + (n & 1), (n >> 1) + 1)) return;
#pragma unroll 1
                    for (int half = 0; half < kTile / C::KEYS; ++half, ++raws) {
                        const uint32_t ri = raws % C::RAWS;
                        if (!wait(C::b_raw_full + ri, raws / C::RAWS)) return;
                        const uint32_t raw = sb + C::off_raw + ri * C::RAW;
                        uint2 w[BATCH];
                        uint32_t f[BATCH];
                        if (for_keys) {
                            const uint32_t out = sb + C::off_k + (n & 1) * C::OPERAND + half * 8192;
#pragma unroll
                            for (int p = 0; p < K_STEPS; p += BATCH) {
#pragma unroll
                                for (int j = 0; j < BATCH && p + j < K_STEPS; ++j) {
                                    const int row = (p + j) / NK * K_ROWS, c = (p + j) % NK;
                                    w[j] = lds64(raw + codes + row / 16 * BB + c * 32);
                                    f[j] = lds8(raw + scale + row / 16 * BB + c * 4);
                                }
#pragma unroll
                                for (int j = 0; j < BATCH && p + j < K_STEPS; ++j) {
                                    const uint32_t to = out + (p + j) / NK * K_ROWS * 128 + (p + j) % NK * 16384;
                                    convert(w[j], scale_pair(f[j]), to + out0, to + out1);
                                }
                            }
                        } else {
                            const uint32_t out = sb + C::off_v + (n & 1) * C::OPERAND + half * (8 * NK * 1024);
                            // past the end the bytes are anything, NaN scales too: a zero weight does not undo that
                            const int left = walk.q.len - (tile * kTile + half * C::KEYS + blk_key);
#pragma unroll
                            for (int p = 0; p < V_STEPS; p += BATCH) {
#pragma unroll
                                for (int j = 0; j < BATCH && p + j < V_STEPS; ++j) {
                                    const int blk = (p + j) / SPLIT * V_BLKS, c = (p + j) % SPLIT * PAIRS;
                                    w[j] = lds64(raw + codes + blk * BB + c * 128);
                                    f[j] = lds8(raw + scale + blk * BB + c * 16);
                                    if (blk * 16 >= left) f[j] = 0;
                                }
#pragma unroll
                                for (int j = 0; j < BATCH && p + j < V_STEPS; ++j) {
                                    const int blk = (p + j) / SPLIT * V_BLKS, c = (p + j) % SPLIT * PAIRS;
                                    // c is a multiple of 64 channels where it is not 0
                                    const uint32_t to = out + blk * 2 * NK * 1024 + c / 4 * 1024;
                                    convert(w[j], scale_pair(f[j]), to + out0, to + out1);
                                }
                            }
                        }
                        __syncwarp();
                        if (lane == 0) arrive(bar(C::b_raw_empty + ri));
                    }
                    umma::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) arrive(bar(b_full + (n & 1)));
                }
            }
        };
        work();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::R_MISC));
    if (warp == C::SOFT + C::DEQ) {
        // ------------------------------------------------------------ producer
        uint32_t raws = 0;
        constexpr int BLOCKS = C::KEYS / 16;
        const int chunk = min(1 << (a.page_shift - 4), BLOCKS);  // blocks per copy
        auto work = [&]() {
            while (walk.next(a, it)) {
                const int32_t *table = a.block_table + (size_t)it.r * a.max_pages;
                const int pages = (int)(((uint32_t)walk.q.len + (1u << a.page_shift) - 1) >> a.page_shift);
                int from = 0, entry = 0, held = 0;  // 32 table entries, one per lane, from page `from` on
#pragma unroll 1
                for (int tile = it.first; tile < it.last; ++tile)
#pragma unroll 1
                    for (int half = 0; half < kTile / C::KEYS; ++half, ++raws) {
                        const uint32_t ri = raws % C::RAWS;
                        const int key0 = tile * kTile + half * C::KEYS;
                        const uint32_t key = (uint32_t)key0 + lane * chunk * 16;  // (past the last one in lanes without a copy)
                        // blocks of this lane's copy that hold keys
                        const int left = (walk.q.len - key0 - lane * chunk * 16 + 15) >> 4;
                        const int mine = lane * chunk < BLOCKS ? min(max(left, 0), chunk) : 0;
                        const int page0 = key0 >> a.page_shift;
                        if (page0 + BLOCKS - 1 >= from + held) {
                            from = page0, held = 32;
                            entry = 0;
                            if (from + lane < pages) {
                                entry = __ldg(table + from + lane);
                                if (entry < 0 || entry >= a.num_pages) {
                                    entry = 0;  // the read stays in the pool
                                    if (a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
                                }
                            }
                            __syncwarp();
                        }
                        const int page = __shfl_sync(0xffffffffu, entry, ((int)(key >> a.page_shift) - from) & 31);
                        const int all = __reduce_add_sync(0xffffffffu, mine);
                        if (!wait(C::b_raw_empty + ri, raws / C::RAWS + 1)) return;
                        if (lane == 0) umma::mbar_expect_tx(bar(C::b_raw_full + ri), all * BB);
                        __syncwarp();
                        if (mine > 0) {
                            const int blk = (key & ((1u << a.page_shift) - 1)) >> 4;
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
                poll(bar(C::b_raw_full + i % C::RAWS), (i / C::RAWS) & 1, kWaitLimit);
        }
    } else if (warp == C::SOFT + C::DEQ + 1) {
        // ------------------------------------------------------------ products
        constexpr uint32_t id_s = idesc_f16(128, 128, 0), id_o = idesc_f16(128, D, 1);
        const uint32_t lead = elect();
        const uint32_t sb4 = __shfl_sync(0xffffffffu, sb >> 4, 0), tm = __shfl_sync(0xffffffffu, tmem, 0);
        uint32_t n = 0, items = 0;
        auto scores = [&](int t, uint32_t tile, int b) {
            const uint32_t q4 = sb4 + ((C::off_q + t * C::OPERAND) >> 4), k4 = sb4 + ((C::off_k + (tile & 1) * C::OPERAND) >> 4);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const uint32_t o = ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4;
                mma_ss(tm + b * 128, umma::sdesc4(q4 + o, 16, 1024), umma::sdesc4(k4 + o, 16, 1024), id_s, ks > 0, lead);
            }
            commit(bar(C::b_s_full + b), lead);
        };
        auto values = [&](int t, uint32_t tile, bool acc, uint32_t parity) {
            const uint32_t v4 = sb4 + ((C::off_v + (tile & 1) * C::OPERAND) >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                if (ks % 4 == 0) {
                    if (!wait(C::b_p_full + 2 * t + ks / 4, parity)) return false;
                    umma::fence_after();
                }
                mma_ts(tm + C::t_o + t * D, tm + t * 128 + ks * 8, umma::sdesc4(v4 + ((ks * 16 * D * 2) >> 4), 1024, 16 * D),
                       id_o, acc || ks > 0, lead);
            }
            commit(bar(C::b_o_done + t), lead);
            return true;
        };
        auto work = [&]() {
            while (walk.next(a, it)) {
                const int tiles = __shfl_sync(0xffffffffu, it.last - it.first, 0);
                if (tiles == 0) continue;
                if (!wait(C::b_q_full, items++)) return;
                if (!wait(C::b_k_full + (n & 1), n >> 1)) return;
                umma::fence_after();
#pragma unroll
                for (int t = 0; t < QT; ++t) scores(t, n, QT == 2 ? t : n & 1);
                commit(bar(C::b_k_empty + (n & 1)), lead);
                if (QT == 1 && tiles == 1) commit(bar(C::b_q_empty), lead);
#pragma unroll 1
                for (int j = 0; j < tiles; ++j, ++n) {
                    if (QT == 1 && j + 1 < tiles) {
                        if (!wait(C::b_k_full + ((n + 1) & 1), (n + 1) >> 1)) return;
                        umma::fence_after();
                        scores(0, n + 1, (n + 1) & 1);
                        commit(bar(C::b_k_empty + ((n + 1) & 1)), lead);
                        if (j + 2 == tiles) commit(bar(C::b_q_empty), lead);
                    }
                    if (QT == 1 && j == 0 && !wait(C::b_o_free, items)) return;
                    if (!wait(C::b_v_full + (n & 1), n >> 1)) return;
                    if (QT == 1) {
                        if (!values(n & 1, n, j > 1, n >> 1)) return;
                    } else {
#pragma unroll
                        for (int t = 0; t < QT; ++t) {
                            if (!values(t, n, j > 0, n)) return;
                            if (j + 1 < tiles) {
                                if (t == 0 && !wait(C::b_k_full + ((n + 1) & 1), (n + 1) >> 1)) return;
                                umma::fence_after();
                                scores(t, n + 1, t);
                            }
                        }
                    }
                    commit(bar(C::b_v_empty + (n & 1)), lead);
                    if (QT == 2 && j + 1 < tiles) commit(bar(C::b_k_empty + ((n + 1) & 1)), lead);
                }
            }
        };
        work();
        // products in flight end before the CTA leaves
        commit(bar(C::b_drain), lead);
        poll(bar(C::b_drain), 0, kWaitLimit);
    } else if (QT == 1) {
        // ------------------------------------------------------------ queries: D / 8 lanes per row, ahead of the item
        constexpr int LANES = D / 8, STEP = 64 / LANES, BATCH = 8;
        const int e = tid - (C::SOFT + C::DEQ + 2) * 32, chunk = e % LANES, sub = e / LANES;
        uint32_t items = 0;
        auto work = [&]() {
            while (walk.next(a, it)) {
                if (it.last == it.first) continue;
                const Req &q = walk.q;
                const float base = a.scale * kLog2e * (a.k_scale ? a.k_scale[it.h] : 1.f);
                volatile float *facs = reinterpret_cast<volatile float *>(smem + C::off_fac) + (items & 1) * C::ROWS;
#pragma unroll 1
                for (int r0 = 0; r0 < C::ROWS; r0 += BATCH * STEP) {
                    uint4 w[BATCH];
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        const int rr = it.row0 + r0 + j * STEP + sub;
                        w[j] = make_uint4(0, 0, 0, 0);
                        if (rr < q.rows)
                            w[j] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                                         (size_t)(q.q0 + rr / G) * a.q_stride +
                                                                         (size_t)(it.h * G + rr % G) * D) + chunk);
                    }
                    // the last item's products have read Q
                    if (r0 == 0 && !wait(C::b_q_empty, items + 1)) return;
#pragma unroll
                    for (int j = 0; j < BATCH; ++j) {
                        const int row = r0 + j * STEP + sub;
                        uint32_t top = magnitude(w[j]);
#pragma unroll
                        for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        const int ex = exponent(top);
                        store_query(sb + C::off_q + umma::kmaj(row, chunk * 8, 128), w[j], scale_up(base, ex));
                        if (chunk == 0) facs[row] = factor(base, ex);
                    }
                }
                umma::fence_proxy_async();
                arrive(bar(C::b_q_full));
                ++items;
            }
        };
        work();
    }
    }
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    if (tid == 0 && misc[1] && a.status) atomicOr(a.status, KDA_STATUS_TIMEOUT);
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
    wait_for_primary();
}

template <int D, int QT>
cudaError_t launch(const Cache4AttnArgs &a, int sms, bool beside, cudaStream_t st) {
    auto kernel = kda_cache4_attn_tc_kernel<D, QT>;
    constexpr int bytes = Cfg<D, QT>::SMEM;
    static_assert(bytes <= 232448, "shared memory of one CTA");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sms);
    cfg.blockDim = dim3(Cfg<D, QT>::THREADS);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

size_t cache4_attn_tc_workspace(int sms, int d) {
    return (size_t)sms * (sizeof(int4) + 2 * 256 * (size_t)(d + 2) * sizeof(float));
}

// two row tiles at a time when a request may have more than 128 rows
int cache4_attn_tc_rows(long long rows) { return rows > 128 ? 256 : 128; }

cudaError_t launch_cache4_attn_tc(const Cache4AttnArgs &a, int d, long long rows, int sms, bool beside, cudaStream_t st) {
    if (cache4_attn_tc_rows(rows) == 256) return d == 128 ? launch<128, 2>(a, sms, beside, st) : launch<64, 2>(a, sms, beside, st);
    return d == 128 ? launch<128, 1>(a, sms, beside, st) : launch<64, 1>(a, sms, beside, st);
}

}  // namespace kda
