// cache4_attn.cu -- attention of packed, ragged queries over the 4-bit pages.
//
//   s_ij = scale q_i . k_j,   p_ij = e^{s_ij - max_j s_ij} over the visible j,
//   o_i = sum_j p_ij v_j / sum_j p_ij,   lse_i = log sum_j e^{s_ij}
//
// Query i of a request with n new tokens and L cached ones (the new among
// them) sits at position L - n + i and sees positions j <= its own (and
// j > its own - window).  The query heads of a group share a key head, so a
// row is a (token, head of the group) pair and rows of a request and key head
// are cut into row tiles.
//
// This file: few rows (single tokens, up to 16 rows; 32-bit queries of any
// number).  Memory bounds that, 9 d / 8 bytes per key and head against 4 d
// flops per row.  Every warp is a worker of its own: it takes an equal,
// contiguous share of all (request, key head, row tile, key tile) units in
// that order, keeps its own ring of key tiles filled by bulk copies and meets
// no barrier.  A key tile goes from shared memory to registers once, the
// codes become f16 pairs (exact) in the lanes that hold them as operand
// fragments, and the products run with keys on M and rows on N, so eight rows
// cost as much as one and no operand is padded.  The weights turn from the
// accumulator to an operand by an 8 x 8 transpose per register.  Running
// maximum, sum and the accumulator are fp32; the weights are rounded to f16
// (11 bits, scaled by 2^kLift so that small ones keep their bits), with a
// second f16 part for 32-bit queries, and so are the queries (scaled by a
// power of two per row), so that only that rounding separates the result from
// fp32.  A worker whose share cuts a row tile's keys leaves (max, sum, sum of
// weighted values), and kda_cache4_merge_kernel joins the shares in key order.
//
// Measured at d = 128, 96 query heads on 12 key heads (device time): 256
// single tokens over up to 8K keys (1.86 GB) 314 us, 5.9 TB/s, 88 % of the
// measured copy bandwidth; one token over 1M keys (1.81 GB) 301 us, 89 %; one
// over 1,003 keys 11.2 us.  After the copies comes instruction issue (57 %
// busy, the conversion's pipe 49 %): 534 warp instructions per 32 keys, of
// which the conversion of the codes is 290 and the products 32.
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache4.cuh"
#include "cache4_sched.cuh"
#include "kda_internal.h"
#include "kda_umma.cuh"

namespace kda {
namespace {

using namespace cache4;

// Work on a tile that does not grow with it (the wait, the copies, the maximum
// across lanes, the schedule) was a sixth of the instructions at 32 keys, and
// instruction issue is what comes after the copies here: 64 keys, in 12 warps
// of up to 168 registers.
constexpr int kTile = FewRows::TILE;     // keys per tile
constexpr int kBlocks = kTile / 16;      // blocks per tile
constexpr int kLead = FewRows::LEAD;     // an item's start and end, in tiles
constexpr int kWarps = 12;               // workers per CTA
constexpr int stages(int d) { return d == 128 ? 2 : 4; }  // tiles in flight per worker: 221 KB
// The first wait for a tile's copy: a test build (KDA_TEST_SHORT_FIRST_WAIT) gives up on it
// at once, to exercise the way out.
#ifdef KDA_TEST_SHORT_FIRST_WAIT
constexpr uint32_t kFirstWait = 0;
#else
constexpr uint32_t kFirstWait = kWaitLimit;
#endif
constexpr float kLift = FewRows::LIFT;  // weights are 2^(s - max + kLift), at most 2^15 of f16's 65504

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// transpose of an 8 x 8 matrix of 16-bit elements held one pair per lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kWarps * 32, 1)
kda_cache4_attn_kernel(const Cache4AttnArgs a) {
    constexpr int ROWS = 8 * NT, KS = D / 16, BB = block_bytes(D), STAGE = kBlocks * BB, kStages = stages(D);
    constexpr int PARTS = F32 ? 2 : 1;  // f16 parts of a query or weight
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ long long s_prefix[kWarps * 32 + 33];
    __shared__ __align__(8) uint64_t s_bar[kWarps * kStages];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int G = a.Hq / a.Hkv;

    allow_dependents();
    if (lane < kStages) umma::mbar_init(smem_addr(&s_bar[warp * kStages + lane]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    // neighbouring workers sit on different SMs, so that few units spread over all of them
    const int me = warp * gridDim.x + blockIdx.x;
    Walk<ROWS, kTile, kLead> walk(a);
    walk.begin(a, s_prefix, me, gridDim.x * kWarps);
    int4 job = make_int4(-1, 0, 0, 0);
    const uint32_t ring = smem_addr(smem) + warp * (kStages * STAGE);
    const uint32_t bars = smem_addr(&s_bar[warp * kStages]);
    uint32_t stage = 0, phase = 0;   // next stage to read and its parity
    bool dead = false;

    Item it;
    while (!dead && walk.next(a, it)) {
        const Req &q = walk.q;
        const int h = it.h, row0 = it.row0, pos0 = it.pos0, pos1 = it.pos1, first = it.first, last = it.last;

        // ---- query fragments: row g of every 8, channels (D / 4) t4 ...
        uint32_t qf[NT][PARTS][KS][2];
        float fac[NT][2];
        // the sign (and a zero) of the scale goes into the queries: the factor stays positive, so that it may
        // follow the maximum and a masked score stays -inf (a scale that is NaN makes the queries NaN)
        const float base = a.scale * kLog2e * (a.k_scale ? a.k_scale[h] : 1.f);
        const float sign = base < 0.f ? -1.f : base > 0.f ? 1.f : base;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rr = row0 + nt * 8 + g;
            float v[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; ++i) v[i] = 0.f;
            if (rr < q.rows) {
                const size_t e = (size_t)(q.q0 + rr / G) * a.q_stride + (size_t)(h * G + rr % G) * D + t4 * (D / 4);
                if constexpr (F32) {
                    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + e);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const float4 w = __ldg(p + i);
                        v[4 * i] = w.x, v[4 * i + 1] = w.y, v[4 * i + 2] = w.z, v[4 * i + 3] = w.w;
                    }
                } else {
                    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + e);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint4 w = __ldg(p + i);
                        const uint32_t s[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[8 * i + 2 * j] = __uint_as_float(s[j] << 16);
                            v[8 * i + 2 * j + 1] = __uint_as_float(s[j] & 0xffff0000u);
                        }
                    }
                }
            }
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(v[i]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // a power of two that brings the row's largest element to [2^8, 2^9)
            const int ex = min(max((int)(__float_as_uint(top) >> 23), 9), 253);
            const float up = sign * __uint_as_float((uint32_t)(262 - ex) << 23);
            const float down = __uint_as_float((uint32_t)(ex - 8) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float lo = v[4 * ks + 2 * b] * up, hi = v[4 * ks + 2 * b + 1] * up;
                    qf[nt][0][ks][b] = pack_f16(lo, hi);
                    if constexpr (F32) {
                        const float2 w = unpack_f16(qf[nt][0][ks][b]);
                        // (an infinity has no second part: it stays one)
                        qf[nt][PARTS - 1][ks][b] = pack_f16(lo == w.x ? 0.f : lo - w.x, hi == w.y ? 0.f : hi - w.y);
                    }
                }
            // this lane's accumulator columns are rows 2 t4 and 2 t4 + 1
#pragma unroll
            for (int j = 0; j < 2; ++j) fac[nt][j] = fmaxf(fabsf(base) * __shfl_sync(0xffffffffu, down, (2 * t4 + j) * 4), 1e-37f);
        }
        // last visible key of the columns' rows (-1: padding or nothing to see)
        int see[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int rr = row0 + nt * 8 + 2 * t4 + j;
                see[nt][j] = rr < q.rows ? q.len - q.n + rr / G : -1;
            }

        float m[NT][2], l[NT][2], acc[NT][KS][4];  // (m: the largest score, without its factor)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.f;
        }

        // ---- ring: block table entries, 32 at a time, one per lane; a copy is
        // what a page holds of the tile, issued by a lane of its own
        const int32_t *table = a.block_table + (size_t)it.r * a.max_pages;
        const int pages = (int)(((uint32_t)q.len + (1u << a.page_shift) - 1) >> a.page_shift);
        const int chunk = a.page_shift < 6 ? 1 << (a.page_shift - 4) : kBlocks;  // blocks per copy
        const uint8_t *base_h = a.cache + (((size_t)h << (a.page_shift - 4)) * BB);
        const size_t page_bytes = (((size_t)a.Hkv << (a.page_shift - 4)) * BB);
        int from = 0, held = 0, entry = 0;
        auto fill = [&](int tile, uint32_t st) {
            const int key0 = tile * kTile, page0 = key0 >> a.page_shift;
            const uint32_t key = (uint32_t)key0 + lane * chunk * 16;  // (past the last key in lanes without a copy)
            if (page0 + kBlocks > from + held) {
                from = page0, held = 32, entry = 0;
                if (from + lane < pages) {
                    entry = table[from + lane];
                    if (entry < 0 || entry >= a.num_pages) {
                        entry = 0;  // the read stays in the pool
                        if (a.status) atomicOr(a.status, KDA_STATUS_BAD_PAGE);
                    }
                }
                __syncwarp();
            }
            const int page = __shfl_sync(0xffffffffu, entry, ((int)(key >> a.page_shift) - from) & 31);
            const int all = min(kBlocks, (q.len - key0 + 15) >> 4);  // blocks with keys
            const uint32_t bar = bars + st * 8;
            if (lane == 0) umma::mbar_expect_tx(bar, all * BB);
            __syncwarp();
            const int mine = min(chunk, all - lane * chunk);
            if (mine > 0) {
                const int blk = (key & ((1u << a.page_shift) - 1)) >> 4;
                umma::bulk_load(ring + st * STAGE + lane * chunk * BB, base_h + page * page_bytes + blk * BB, mine * BB, bar);
            }
        };
        uint32_t put = stage;
        int filled = first;
#pragma unroll 1
        for (; filled < last && filled < first + kStages; ++filled) {
            fill(filled, put);
            put = put + 1 == kStages ? 0 : put + 1;
        }

#pragma unroll 1
        for (int tile = first; tile < last; ++tile) {
            if (!__all_sync(0xffffffffu, poll(bars + stage * 8, phase, tile == first ? kFirstWait : kWaitLimit))) {
                dead = true;
                if (lane == 0 && a.status) atomicOr(a.status, KDA_STATUS_TIMEOUT);
                // the copies in flight end before the warp leaves
                for (int i = tile; i < filled; ++i) {
                    poll(bars + stage * 8, phase, kWaitLimit);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
                break;
            }
            const uint32_t buf = ring + stage * STAGE;
            const int key0 = tile * kTile;
            const int blocks = (q.len - key0 + 15) >> 4;  // with keys in them, of this tile's
            // ---- S^T = K Q^T, 16 keys x 8 rows per product; row g of a
            // product is key 4 (g / 2) + (g & 1), row g + 8 two further, so
            // that lane t4 ends up with the weights of keys 4 t4 .. 4 t4 + 3
            float s[kBlocks][NT][4];
#pragma unroll
            for (int mt = 0; mt < kBlocks; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[mt][nt][j] = 0.f;
                if (mt >= blocks) continue;
                const uint32_t blk = buf + mt * BB;
                const int tok = 4 * (g >> 1) + (g & 1);
                uint32_t kw[2][D / 32], sc[2];
                if constexpr (D == 128) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 w = lds128(blk + (tok + 2 * i) * 64 + t4 * 16);
                        kw[i][0] = w.x, kw[i][1] = w.y, kw[i][2] = w.z, kw[i][3] = w.w;
                        sc[i] = scales_to_f16(lds16(blk + off_ks(D) + (tok + 2 * i) * 8 + t4 * 2));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint2 w = lds64(blk + (tok + 2 * i) * 32 + t4 * 8);
                        kw[i][0] = w.x, kw[i][1] = w.y;
                        sc[i] = scales_to_f16(lds8(blk + off_ks(D) + (tok + 2 * i) * 4 + t4));
                    }
                }
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t x0[4], x1[4];
                    codes_to_f16(kw[0][w], x0);
                    codes_to_f16(kw[1][w], x1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x0[j] = w < 2 ? mul_low(x0[j], sc[0]) : mul_high(x0[j], sc[0]);
                        x1[j] = w < 2 ? mul_low(x1[j], sc[1]) : mul_high(x1[j], sc[1]);
                    }
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int p = PARTS - 1; p >= 0; --p)
                                mma_f16(s[mt][nt], x0[2 * hh], x1[2 * hh], x0[2 * hh + 1], x1[2 * hh + 1],
                                        qf[nt][p][2 * w + hh][0], qf[nt][p][2 * w + hh][1]);
                }
            }
            // ---- masks: only tiles that some row of the tile does not see whole
            const bool edge = key0 > pos0 + 1 - kTile || (a.window > 0 && key0 <= pos1 - a.window);
            if (edge) {
                const int tok = key0 + 4 * (g >> 1) + (g & 1);
#pragma unroll
                for (int mt = 0; mt < kBlocks; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = tok + mt * 16 + (j >> 1) * 2, sees = see[nt][j & 1];
                            if (key > sees || (a.window > 0 && key <= sees - a.window)) s[mt][nt][j] = -INFINITY;
                        }
            }
            // ---- running maximum and weights
            uint32_t pf[NT][PARTS][kBlocks][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float top[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    top[j] = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
                    for (int mt = 1; mt < kBlocks; ++mt) top[j] = fmaxf(top[j], fmaxf(s[mt][nt][j], s[mt][nt][j + 2]));
                    top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 4));
                    top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
                    top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
                    top[j] = fmaxf(m[nt][j], top[j]);
                }
                if (__any_sync(0xffffffffu, top[0] > m[nt][0] || top[1] > m[nt][1])) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float shrink =
                            top[j] == -INFINITY ? 1.f : exp2_fast(scaled(m[nt][j], fac[nt][j]) - scaled(top[j], fac[nt][j]));
                        l[nt][j] *= shrink;
#pragma unroll
                        for (int i = 0; i < KS; ++i) {
                            acc[nt][i][j] *= shrink;
                            acc[nt][i][j + 2] *= shrink;
                        }
                        m[nt][j] = top[j];
                    }
                }
                float off[2], sub[2];
                bool far = false;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float ref = m[nt][j] == -INFINITY ? 0.f : m[nt][j], at = scaled(ref, fac[nt][j]);
                    const bool big = fabsf(at) >= kFar;
                    far = far || big;
                    sub[j] = big ? ref : 0.f;
                    off[j] = (F32 ? 0.f : kLift) - (big ? 0.f : at);
                }
                if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                    for (int mt = 0; mt < kBlocks; ++mt)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[mt][nt][j] -= sub[j & 1];
                }
#pragma unroll
                for (int mt = 0; mt < kBlocks; ++mt) {
                    float w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        w[j] = exp2_fast(fmaf(s[mt][nt][j], fac[nt][j & 1], off[j & 1]));
                        // 32-bit calls: an exponent near 15 would carry four bits less than one near 0
                        if constexpr (F32) w[j] *= 32768.f;
                        l[nt][j & 1] += w[j];
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t hi = pack_f16(w[2 * i], w[2 * i + 1]);
                        pf[nt][0][mt][i] = transpose8(hi);
                        if constexpr (F32) {
                            const float2 b = unpack_f16(hi);
                            pf[nt][PARTS - 1][mt][i] = transpose8(pack_f16(w[2 * i] - b.x, w[2 * i + 1] - b.y));
                        }
                    }
                }
            }
            // ---- O^T += V^T P^T: lane (g, t4) holds channels (D / 8) g ... of keys 4 t4 .. 4 t4 + 3
#pragma unroll
            for (int mt = 0; mt < kBlocks; ++mt) {
                if (mt >= blocks) continue;
                const uint32_t blk = buf + mt * BB;
                constexpr int W = D / 64;  // code words per key and lane
                uint32_t vw[4][W], sv;
                if constexpr (D == 128) {
                    const uint4 w0 = lds128(blk + off_vc(D) + g * 128 + t4 * 32);
                    const uint4 w1 = lds128(blk + off_vc(D) + g * 128 + t4 * 32 + 16);
                    vw[0][0] = w0.x, vw[0][W - 1] = w0.y, vw[1][0] = w0.z, vw[1][W - 1] = w0.w;
                    vw[2][0] = w1.x, vw[2][W - 1] = w1.y, vw[3][0] = w1.z, vw[3][W - 1] = w1.w;
                    sv = lds32(blk + off_vs(D) + g * 16 + t4 * 4);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vw[i][0] = lds32(blk + off_vc(D) + (g >> 1) * 128 + (t4 * 4 + i) * 8 + (g & 1) * 4);
                    sv = lds32(blk + off_vs(D) + (g >> 1) * 16 + t4 * 4);
                }
                if (key0 > q.len - kTile) {
                    // keys past the end hold anything, NaN scales too: a zero weight does not undo that
                    const int over = key0 - q.len + mt * 16 + t4 * 4 + 4;
                    if (over > 0) sv = over >= 4 ? 0u : sv & (0xffffffffu >> (8 * over));
                }
                const uint32_t s01 = scales_to_f16(sv & 0xffffu), s23 = scales_to_f16(sv >> 16);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd channels, keys (0, 1) and (2, 3)
                    constexpr uint32_t M = 0x0f0f0f0fu;
                    codes_to_f16((vw[0][w] & M) | ((vw[1][w] << 4) & ~M), e01);
                    codes_to_f16(((vw[0][w] >> 4) & M) | (vw[1][w] & ~M), o01);
                    codes_to_f16((vw[2][w] & M) | ((vw[3][w] << 4) & ~M), e23);
                    codes_to_f16(((vw[2][w] >> 4) & M) | (vw[3][w] & ~M), o23);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = mul_f16x2(e01[i], s01), a1 = mul_f16x2(o01[i], s01);
                        const uint32_t a2 = mul_f16x2(e23[i], s23), a3 = mul_f16x2(o23[i], s23);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int p = PARTS - 1; p >= 0; --p)
                                mma_f16(acc[nt][w * 4 + i], a0, a1, a2, a3, pf[nt][p][mt][0], pf[nt][p][mt][1]);
                    }
                }
            }
            __syncwarp();  // every lane has read the stage
            if (filled < last) {
                fill(filled, stage);
                ++filled;
            }
            if (++stage == kStages) stage = 0, phase ^= 1;
        }
        if (dead) break;

        // ---- the rows' sums over all lanes of a column
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
                l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
            }
        if (it.whole()) {
            const float vs = a.v_scale ? a.v_scale[h] : 1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int rr = row0 + nt * 8 + 2 * t4 + j;
                    if (rr >= q.rows) continue;
                    const size_t head = (size_t)(q.q0 + rr / G) * a.Hq + h * G + rr % G;
                    const bool none = see[nt][j] < 0;
                    const float inv = none ? 0.f : vs / l[nt][j];
                    float y[D / 8];
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        y[2 * i] = none ? 0.f : acc[nt][i][j] * inv;
                        y[2 * i + 1] = none ? 0.f : acc[nt][i][j + 2] * inv;
                    }
                    if constexpr (F32) {
                        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(a.o) + head * D + g * (D / 8));
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            p[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    } else {
                        uint4 *p = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + head * D + g * (D / 8));
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const __nv_bfloat162 b = __floats2bfloat162_rn(y[8 * i + 2 * c], y[8 * i + 2 * c + 1]);
                                w[c] = *reinterpret_cast<const uint32_t *>(&b);
                            }
                            p[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (a.lse && g == 0)
                        a.lse[head] = none ? -INFINITY : (scaled(m[nt][j], fac[nt][j]) + log2f(l[nt][j]) - kLift) * kLn2;
                }
        } else {
            // part 1 starts a row tile that goes on, part 0 continues one
            const int part = it.starts ? 1 : 0;
            float *w = a.parts + ((size_t)me * 2 + part) * (ROWS * (D + 2));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = nt * 8 + 2 * t4 + j;
                    if (g == 0) {
                        w[row] = scaled(m[nt][j], fac[nt][j]);
                        w[ROWS + row] = l[nt][j];
                    }
                    float4 *p = reinterpret_cast<float4 *>(w + 2 * ROWS + row * D + g * (D / 8));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        p[i] = make_float4(acc[nt][2 * i][j], acc[nt][2 * i][j + 2], acc[nt][2 * i + 1][j],
                                           acc[nt][2 * i + 1][j + 2]);
                }
            if (part == 1) job = make_int4(it.r, h, it.rt, walk.last_worker());
        }
    }
    if (lane == 0) a.jobs[me] = dead ? make_int4(-1, 0, 0, 0) : job;
}

constexpr int smem_bytes(int d) { return kWarps * stages(d) * kBlocks * block_bytes(d); }

template <int D, int NT, bool F32>
cudaError_t launch_attn(const Cache4AttnArgs &a, int sms, cudaStream_t st) {
    auto kernel = kda_cache4_attn_kernel<D, NT, F32>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(D));
    if (e != cudaSuccess) return e;
    kernel<<<sms, kWarps * 32, smem_bytes(D), st>>>(a);
    return cudaGetLastError();
}

}  // namespace

int cache4_attn_workers(int sms) { return sms * kWarps; }
size_t cache4_attn_workspace(int sms, int d) {
    return (size_t)cache4_attn_workers(sms) * (sizeof(int4) + 2 * 16 * (size_t)(d + 2) * sizeof(float));
}

// 16 rows a tile when a request may have more than 8 (the keys' conversion to
// f16 is then shared by two products: 131 MB of two-token requests at 8 heads
// a group 67 us, in tiles of 8 rows 71).  32-bit queries have two f16 parts and
// keep 8: with 16 a batch of 9 x up to 45 queries, d = 64, took 26.1 us instead
// of 23.8, having half the units.
int cache4_attn_rows(bool bf16, long long rows) { return bf16 && rows > 8 ? 16 : 8; }

cudaError_t launch_cache4_attn(const Cache4AttnArgs &a, int d, bool bf16, long long rows, int sms, cudaStream_t st) {
    const bool wide = cache4_attn_rows(bf16, rows) == 16;
    if (d == 128)
        return !bf16 ? launch_attn<128, 1, true>(a, sms, st)
               : wide ? launch_attn<128, 2, false>(a, sms, st)
                      : launch_attn<128, 1, false>(a, sms, st);
    return !bf16 ? launch_attn<64, 1, true>(a, sms, st)
           : wide ? launch_attn<64, 2, false>(a, sms, st)
                  : launch_attn<64, 1, false>(a, sms, st);
}

}  // namespace kda
