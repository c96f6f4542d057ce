// cache4_sched.cuh -- what the attention kernels over the 4-bit pages share:
// the division of the work among workers, the join of shares, small helpers.
//
// An item is a row tile (ROWS rows: pairs of a token and a head of the group)
// of one request and key head; a unit is one key tile (TILE keys) of an item.
// Units are numbered request by request, head by head, row tile by row tile,
// and every worker takes an equal, contiguous range of them, so one long
// request or many short ones load the SMs alike.  Row tiles of a request
// count as many units as its widest one; they are taken from both ends in
// turn (0, last, 1, last - 1, ...), so that under a causal mask neighbours
// share the load.  An item counts LEAD units more than it has key tiles: what
// its start and end cost, so that ranges of many short items are not the last
// to finish.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache4.cuh"
#include "kda_internal.h"

namespace kda {
namespace cache4 {

constexpr uint32_t kWaitLimit = 1u << 24;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A weight is 2^(score * factor + (lift - maximum * factor)), one multiply-add.
// The rounding of the maximum and of the offset lifts the largest weight by a
// step of fp32 at the maximum, 2^-3 at most below this, which f16 has room
// for.  From here on (where a score's own rounding is a factor of 2^(1/16) and
// more) the maximum is taken from the scores first, so that no weight is above
// 2^lift and the largest is never lost.
constexpr float kFar = 1048576.f;
// A maximum with its factor, rounded as it stands: two of the same value cancel
// (fused into a difference they would leave the product's rounding).
__device__ __forceinline__ float scaled(float top, float fac) { return __fmul_rn(top, fac); }

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    unsigned short r;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(r) : "r"(a));
    return r;
}

// Polls until the phase with this parity is over, at most `limit` times.
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, uint32_t limit) {
    if (limit == 0) return false;
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n.reg .u32 n;\nmov.u32 n, %3;\n"
        "AGAIN:\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n@p bra DONE;\n"
        "sub.u32 n, n, 1;\nsetp.ne.u32 p, n, 0;\n@p bra AGAIN;\nsetp.ne.u32 p, n, n;\n"
        "DONE:\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(limit)
        : "memory");
    return ok != 0;
}

// A request as the schedule sees it.
struct Req {
    int q0, n, len;  // first query row, new tokens, keys
    int rows, row_tiles;
    int units;       // key tiles of every row tile (the widest one's), and LEAD
    bool ok;
};

template <int ROWS, int TILE, int LEAD>
__device__ __forceinline__ Req request(const Cache4AttnArgs &a, int r, int G) {
    Req q;
    const int c0 = a.cu_seqlens[r], c1 = a.cu_seqlens[r + 1], len = a.seq_len[r];
    q.ok = c0 >= 0 && c1 >= c0 && c1 <= a.T && len >= 0 && len <= ((long long)a.max_pages << a.page_shift);
    q.q0 = c0;
    q.n = q.ok ? c1 - c0 : 0;
    q.len = q.ok ? len : 0;
    q.rows = q.n * G;
    // a call runs as one or two kernels; each takes the requests whose rows are in its range
    q.row_tiles = q.rows > a.rows_above && q.rows <= a.rows_to ? (q.rows + ROWS - 1) / ROWS : 0;
    int t = (int)(((uint32_t)q.len + TILE - 1) / TILE);  // (lengths go up to 2^31 - 16)
    if (a.window > 0) {
        // a row tile spans up to (ROWS - 1) / G + 2 tokens
        const long long span = ((long long)a.window + (ROWS - 1) / G + 1) / TILE + 2;
        if (span < t) t = (int)span;
    }
    q.units = (t > 0 ? t : 1) + LEAD;  // a row tile that sees nothing is still written
    return q;
}

struct Item {
    int r, h, rt, row0;     // request, key head, row tile and its first row
    int pos0, pos1;         // positions of the tile's first and last token
    int first, last;        // key tiles of this worker's share
    bool starts, ends;      // whether the share holds the item's first and last unit
    __device__ __forceinline__ bool whole() const { return starts && ends; }
};

template <int ROWS, int TILE, int LEAD>
struct Walk {
    int G;
    int r, h, i, unit;          // the next item and its unit
    long long u, u_end, share;  // the next unit's number, the end of the range, units per worker
    Req q;                      // request r

    __device__ __forceinline__ explicit Walk(const Cache4AttnArgs &a)
        : G(a.Hq / a.Hkv), r(0), h(0), i(0), unit(0), u(0), u_end(0), share(1) {}

    // All threads of the CTA; prefix has blockDim.x + 33 entries of shared
    // memory, free again after the CTA's next barrier.
    __device__ __forceinline__ void begin(const Cache4AttnArgs &a, long long *prefix, int worker, int workers) {
        const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5;
        long long *sums = prefix + nthr + 1;
        const int per = (a.R + nthr - 1) / nthr;
        const int r_lo = min(a.R, tid * per), r_hi = min(a.R, r_lo + per);
        long long x = 0;
        bool bad = false;
#pragma unroll 1
        for (int k = r_lo; k < r_hi; ++k) {
            const Req e = request<ROWS, TILE, LEAD>(a, k, G);
            bad |= !e.ok;
            x += (long long)e.row_tiles * a.Hkv * e.units;
        }
        if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, KDA_STATUS_BAD_SEQLENS);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < warp; ++w) x += sums[w];
        prefix[tid + 1] = x;
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
        const long long total = prefix[nthr];
        share = total > workers ? (total + workers - 1) / workers : 1;
        u = share * worker;
        u_end = min(total, u + share);
        if (u >= u_end) return;
        int lo = 0, hi = nthr;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= u) lo = mid;
            else hi = mid;
        }
        r = lo * per;
        long long off = u - prefix[lo];
#pragma unroll 1
        for (;; ++r) {
            q = request<ROWS, TILE, LEAD>(a, r, G);
            const long long units = (long long)q.row_tiles * a.Hkv * q.units;
            if (off < units) break;
            off -= units;
        }
        const long long item = off / q.units;
        unit = (int)(off - item * q.units);
        h = (int)(item / q.row_tiles);
        i = (int)(item - (long long)h * q.row_tiles);
    }

    __device__ __forceinline__ bool next(const Cache4AttnArgs &a, Item &it) {
        if (u >= u_end) return false;
        if (unit == q.units) {
            unit = 0;
            if (++i == q.row_tiles) {
                i = 0;
                if (++h == a.Hkv) {
                    h = 0;
#pragma unroll 1
                    do q = request<ROWS, TILE, LEAD>(a, ++r, G);
                    while (q.row_tiles == 0);
                }
            }
        }
        const int unit1 = (int)min((long long)q.units, unit + (u_end - u));
        it.r = r;
        it.h = h;
        it.rt = i & 1 ? q.row_tiles - 1 - (i >> 1) : i >> 1;
        it.row0 = it.rt * ROWS;
        const int row1 = min(q.rows, it.row0 + ROWS) - 1;
        it.pos0 = q.len - q.n + it.row0 / G;
        it.pos1 = q.len - q.n + row1 / G;
        const int key_lo = a.window > 0 ? max(0, it.pos0 - a.window + 1) : 0;
        const int tile_lo = key_lo / TILE;
        const int tiles = it.pos1 < 0 ? 0 : it.pos1 / TILE + 1 - tile_lo;
        it.first = tile_lo + min(max(unit - LEAD, 0), tiles);
        it.last = tile_lo + min(max(unit1 - LEAD, 0), tiles);
        it.starts = unit == 0;
        it.ends = unit1 == q.units;
        u += unit1 - unit;
        unit = unit1;
        return true;
    }

    // the worker whose range ends the current item
    __device__ __forceinline__ int last_worker() const { return (int)((u - unit + q.units - 1) / share); }
};

// What the two attention kernels' shares are made with: keys per tile, an
// item's start and end in tiles, and the power of two that lifts the weights.
// (Leads of 0 / 0, 2 / 2, 4 / 1 and 6 / 3 measured on ragged single tokens and
// verify windows at d = 128: 2 and 5 took 341 to 314 and 354 to 311 us.)
struct FewRows {
    static constexpr int TILE = 64, LEAD = 2;
    static constexpr float LIFT = 15.f;
};
struct ManyRows {
    static constexpr int TILE = 128, LEAD = 5;
    static constexpr float LIFT = 7.f;
};

// lets the next kernel's CTAs be placed as this kernel's leave
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
// until the kernel before is over and its writes are seen (at once where this one was launched in the ordinary way)
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

}  // namespace cache4
}  // namespace kda
