// scan.cu -- the selective state space recurrence over packed sequences, and
// single tokens.  Per channel c and state n, with v = dt + dt_bias, d = ln(1 + e^v):
//
//   h_t = e^{d_t A[c][n]} h_{t-1} + d_t x_t B_t[n],   y_t = (sum_n C_t[n] h_t + D[c] x_t) z_t sigmoid(z_t)
//
// What bounds it: issue slots.  A token and channel costs 8 bytes (bf16 x, dt,
// z, y) and, with 16 states, 20 special functions (0.6 cycles of an SM) and 32 packed
// pairs of operations, which take two slots each (0.5), beside the exponentials', the
// loads' and the token's own slots (0.55), where 8 bytes take 0.34.  16384 tokens x 4096 channels: 295 us in the
// walk (1.27 cycles) where blocks fill the SMs, 400 with 3.4 blocks an SM.
//
// A thread keeps 8 or 16 states of a channel, in pairs for the packed
// operations; the lanes that share a channel are neighbours.  Of eight tokens each of
// them forms the steps, and at the end the outputs, of its own share: the steps
// go round by shuffles, and the lanes' shares of the outputs are added on the
// way to their token's lane.  Eight tokens at a time give the long chains of a
// step (softplus: 13 operations) others to overlap with; with registers for four
// blocks an SM rather than seven the walk of 16384 tokens took 422 us and not 601.  A
// block of 128 threads walks its tokens 16 at a time: x, dt and z of the next
// 16 come by cp.async while these are worked on, and B and C (the same for all
// channels of a group) are widened to 32 bits once per block, so that a thread
// reads them as 16-byte broadcasts.
//
// The recurrence is serial along a sequence.  Where sequences times channels
// do not fill the GPU, or one sequence is far longer than the mean, they are
// cut into segments: a first kernel forms every segment's own end state from
// zero and its sum of d (the segment's decay is e^{A sum d}, exactly), a second
// chains these, and the walk then starts each segment from its true state.  The
// first kernel costs 0.75 of the walk (214 us beside 295), so the cut has to buy more.
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kda_internal.h"
#include "layer.cuh"
#include "scan.cuh"

namespace kda {
namespace {
using namespace layer;
using namespace scan;

constexpr int kTile = 16;  // tokens of a tile
constexpr int GROUP = kSaveEvery;

enum Mode : int {
    WALK = 0,     // outputs, final and saved states
    FORWARD = 1,  // a segment's end state from zero, and its sum of d
    REVERSE = 2,  // the same backwards: what reaches its start of the gradients dy C
};

template <bool BF16, int S, int M>
struct Layout {
    static constexpr int LN = S / M, CH = kThreads / LN;
    static constexpr int raw = kTile * CH * (BF16 ? 2 : 4);  // bytes of one tensor's tile
    static constexpr int bytes = 2 * 3 * raw + 2 * kTile * 2 * S * 4;
};

template <bool BF16, int S, int M, int MODE, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) kda_scan_kernel(ScanArgs a) {
    using E = Elem<BF16>;
    using L = Layout<BF16, S, M>;
    constexpr int LN = L::LN, CH = L::CH, OWN = GROUP / LN;  // tokens of a lane's own in a group
    extern __shared__ __align__(16) unsigned char smem[];
    E *raw = reinterpret_cast<E *>(smem);                            // [2][3][kTile][CH]
    float *bc = reinterpret_cast<float *>(smem + 2 * 3 * L::raw);    // [2][kTile][2 S]: B, then C
    const int tid = threadIdx.x, ch = tid / LN, ln = tid % LN;
    const Segment g = segment_of(a.cu_seqlens, a.N, a.T, a.seg, blockIdx.x);
    if (MODE == WALK && tid == 0 && blockIdx.y == 0) check_sequence(a, blockIdx.x);
    if (g.s < 0) return;
    if (MODE == FORWARD && g.last) return;
    if (MODE == REVERSE && g.first) return;
    const int per = a.D / a.G, tiles = (per + CH - 1) / CH;
    const int grp = blockIdx.y / tiles, c_in = (blockIdx.y - grp * tiles) * CH;  // first channel, in its group
    const int c0 = grp * per + c_in, left = per - c_in;                          // channels from c0 on in the group
    const bool live = ch < left;
    const int c = c0 + (live ? ch : 0);
    const bool third = MODE != FORWARD && a.z != nullptr;

    float2 A2[M / 2], h2[M / 2];
    {
        const float4 *p = reinterpret_cast<const float4 *>(a.A + (size_t)c * S + ln * M);
        const float *h0 = nullptr;
        if (MODE == WALK) h0 = g.first ? (a.initial_state ? a.initial_state + (size_t)g.s * a.D * S : nullptr)
                                       : a.seg_state + (size_t)blockIdx.x * a.D * S;
        const float4 *q = reinterpret_cast<const float4 *>(h0 + (h0 ? (size_t)c * S + ln * M : 0));
#pragma unroll
        for (int i = 0; i < M / 4; ++i) {
            const float4 v = p[i];
            A2[2 * i] = make_float2(v.x, v.y);
            A2[2 * i + 1] = make_float2(v.z, v.w);
            const float4 w = h0 ? q[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            h2[2 * i] = make_float2(w.x, w.y);
            h2[2 * i + 1] = make_float2(w.z, w.w);
        }
    }
    const float skip = MODE == WALK && a.Dskip ? a.Dskip[c] : 0.f, bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    float sum = 0.f;
    const int count = g.t1 - g.t0, steps = (count + kTile - 1) / kTile;
    // row r of the walk: forward from the first token, or backward from the last
    auto token = [&](int r) { return (long long)(MODE == REVERSE ? g.t1 - 1 - r : g.t0 + r); };

    // rows of tile i: copied to their place at once, or (rows off 16-byte boundaries) by way of registers, to be
    // stored after the tile before has been worked on
    constexpr int PART = VEC ? 1 : kTile * CH / kThreads;
    E held[3][PART];
    auto stage = [&](int i) {
        E *dst = raw + (i & 1) * 3 * kTile * CH;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k == 2 && !third) break;
            const E *src = static_cast<const E *>(k == 0 ? (MODE == REVERSE ? a.dy : a.x) : k == 1 ? a.dt : a.z) + c0;
            const long long stride = k == 0 ? (MODE == REVERSE ? a.dy_stride : a.x_stride) : k == 1 ? a.dt_stride : a.z_stride;
            if constexpr (VEC) {
                constexpr int EPC = BF16 ? 8 : 4, PER_ROW = CH / EPC;
#pragma unroll
                for (int e = tid; e < kTile * PER_ROW; e += kThreads) {
                    const int r = e / PER_ROW, o = (e % PER_ROW) * EPC, at = i * kTile + r;
                    const bool ok = at < count && o < left;
                    cp_async16(dst + (k * kTile + r) * CH + o, src + (ok ? token(at) * stride + o : 0), ok);
                }
            } else {
#pragma unroll
                for (int e = 0; e < PART; ++e) {
                    const int r = (tid + e * kThreads) / CH, o = (tid + e * kThreads) % CH, at = i * kTile + r;
                    held[k][e] = (E)0.f;
                    if (at < count && o < left) held[k][e] = src[token(at) * stride + o];
                }
            }
        }
        if constexpr (VEC) cp_async_commit();
    };
    auto put = [&](int i) {
        if constexpr (!VEC) {
            E *dst = raw + (i & 1) * 3 * kTile * CH;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (k == 2 && !third) break;
#pragma unroll
                for (int e = 0; e < PART; ++e) dst[k * kTile * CH + tid + e * kThreads] = held[k][e];
            }
        }
    };
    // four neighbouring values of B and C at a time (REVERSE wants C alone)
    constexpr int BCN = (kTile * 2 * S + 4 * kThreads - 1) / (4 * kThreads);
    Vec<BF16, 4> bcr[BCN];
    auto bc_load = [&](int i) {
#pragma unroll
        for (int k = 0; k < BCN; ++k) {
            const int e = 4 * (tid + k * kThreads), r = e / (2 * S), n = e % (2 * S), at = i * kTile + r;
            bcr[k].zero();
            if (at >= count || (MODE == FORWARD && n >= S) || (MODE == REVERSE && n < S)) continue;
            const E *p = static_cast<const E *>(n < S ? a.B : a.C) + token(at) * (n < S ? a.b_stride : a.c_stride) + grp * S + n % S;
            if (a.wide_bc) {
                bcr[k].load(p);
            } else {
                const float f[4] = {(float)p[0], (float)p[1], (float)p[2], (float)p[3]};
                bcr[k].set(f);
            }
        }
    };
    auto bc_store = [&](int i) {
#pragma unroll
        for (int k = 0; k < BCN; ++k)
            if (tid + k * kThreads < kTile * 2 * S / 4)
                reinterpret_cast<float4 *>(bc + (i & 1) * kTile * 2 * S)[tid + k * kThreads] =
                    make_float4(bcr[k].get(0), bcr[k].get(1), bcr[k].get(2), bcr[k].get(3));
    };

    if (steps > 0) {
        stage(0);
        bc_load(0);
        put(0);
        bc_store(0);
    }
#pragma unroll
    for (int i = 0; i < M / 2; ++i) A2[i] = make_float2(rate(A2[i].x), rate(A2[i].y));
    for (int i = 0; i < steps; ++i) {
        if constexpr (VEC) cp_async_wait_all();
        __syncthreads();
        const bool more = i + 1 < steps;
        if (more) {
            stage(i + 1);
            bc_load(i + 1);
        }
        const E *xs = raw + (i & 1) * 3 * kTile * CH + ch, *ds = xs + kTile * CH, *zs = ds + kTile * CH;
        const float *bt = bc + (i & 1) * kTile * 2 * S + ln * M + (MODE == REVERSE ? S : 0);
        const int rows = min(kTile, count - i * kTile);
        // eight tokens at a time.  Past the end the step is 0: decay 1 and nothing added.
        auto group = [&](auto all, int r0) {
            constexpr bool ALL = decltype(all)::value;  // no token past the end among the eight
            const int mine = r0 + ln * OWN;  // the lane's own tokens
            float d[OWN], in[OWN], y[GROUP];
#pragma unroll
            for (int j = 0; j < OWN; j += 2) {  // (two of them in packed operations)
                constexpr int NEXT = OWN > 1 ? 1 : 0;
                const int p = (mine + j) * CH, q = (mine + j + NEXT) * CH;
                float2 x = make_float2((float)xs[p], (float)xs[q]), sig;
                float2 v = __fadd2_rn(make_float2((float)ds[p], (float)ds[q]), both(bias));
                if (a.dt_softplus) v = softplus2(v, sig);
                if (!ALL && mine + j >= rows) v.x = 0.f;
                if (!ALL && mine + j + NEXT >= rows) v.y = 0.f;
                if (MODE == REVERSE && third) x = __fmul2_rn(x, silu2(make_float2((float)zs[p], (float)zs[q])));
                if (MODE != REVERSE) x = __fmul2_rn(v, x);
                d[j] = v.x, d[j + NEXT] = v.y;
                in[j] = ALL || mine + j < rows ? x.x : 0.f, in[j + NEXT] = ALL || mine + j + NEXT < rows ? x.y : 0.f;
                if (MODE != WALK) sum += NEXT ? v.x + v.y : v.x;
            }
            if constexpr (MODE == WALK) {
                if (a.saved && live) {
                    const long long slot = g.slot + (i * kTile + r0) / kSaveEvery;
                    float4 *p = reinterpret_cast<float4 *>(a.saved + ((size_t)slot * a.D + c) * S + ln * M);
#pragma unroll
                    for (int k = 0; k < M / 4; ++k) p[k] = make_float4(h2[2 * k].x, h2[2 * k].y, h2[2 * k + 1].x, h2[2 * k + 1].y);
                }
            }
#pragma unroll
            for (int r = 0; r < GROUP; ++r) {
                const int from = (tid & 31 & ~(LN - 1)) + r / OWN;
                const float dr = LN > 1 ? __shfl_sync(0xffffffffu, d[r % OWN], from) : d[r % OWN];
                const float ir = LN > 1 ? __shfl_sync(0xffffffffu, in[r % OWN], from) : in[r % OWN];
                const float2 dd = both(dr), ii = both(ir);
                float2 y2 = both(0.f);
                const float4 *b4 = reinterpret_cast<const float4 *>(bt + (r0 + r) * 2 * S), *c4 = b4 + S / 4;
#pragma unroll
                for (int k = 0; k < M / 4; ++k) {
                    const float4 B4 = b4[k];
                    float4 C4;
                    if constexpr (MODE == WALK) C4 = c4[k];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int n = 2 * k + e;
                        const float2 arg = __ffma2_rn(A2[n], dd, both(kExp2Low));
                        const float2 dec = make_float2(exp2_fast(arg.x), exp2_fast(arg.y));
                        const float2 b = e ? make_float2(B4.z, B4.w) : make_float2(B4.x, B4.y);
                        if constexpr (MODE == REVERSE) h2[n] = __fmul2_rn(dec, __ffma2_rn(b, ii, h2[n]));
                        else h2[n] = __ffma2_rn(dec, h2[n], __fmul2_rn(ii, b));
                        if constexpr (MODE == WALK)
                            y2 = __ffma2_rn(e ? make_float2(C4.z, C4.w) : make_float2(C4.x, C4.y), h2[n], y2);
                    }
                }
                if constexpr (MODE == WALK) y[r] = y2.x + y2.y;
            }
            if constexpr (MODE == WALK) {
                // the lanes' shares of eight outputs, each added up in its token's lane
#pragma unroll
                for (int o = LN / 2, n = GROUP / 2; o > 0; o /= 2, n /= 2) {
                    const bool up = ln & o;
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        const float send = up ? y[j] : y[j + n], keep = up ? y[j + n] : y[j];
                        y[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                }
                E *yp = static_cast<E *>(a.y) + token(i * kTile + mine) * a.y_stride + c;
#pragma unroll
                for (int j = 0; j < OWN; j += 2) {
                    constexpr int NEXT = OWN > 1 ? 1 : 0;
                    const int p = (mine + j) * CH, q = (mine + j + NEXT) * CH;
                    float2 out = __ffma2_rn(both(skip), make_float2((float)xs[p], (float)xs[q]), make_float2(y[j], y[j + NEXT]));
                    if (third) out = __fmul2_rn(out, silu2(make_float2((float)zs[p], (float)zs[q])));
                    if (live && (ALL || mine + j < rows)) yp[j * a.y_stride] = (E)out.x;
                    if (NEXT && live && (ALL || mine + j + NEXT < rows)) yp[(j + NEXT) * a.y_stride] = (E)out.y;
                }
            }
        };
#pragma unroll 1
        for (int r0 = 0; r0 < rows; r0 += GROUP) {
            if (r0 + GROUP <= rows) group(std::true_type(), r0);
            else group(std::false_type(), r0);
        }
        if (more) {
            put(i + 1);
            bc_store(i + 1);
        }
    }
    if constexpr (MODE != WALK) {
#pragma unroll
        for (int o = 1; o < LN; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (!live) return;
    float *out = nullptr;
    if (MODE == WALK) out = g.last && a.final_state ? a.final_state + (size_t)g.s * a.D * S : nullptr;
    else out = a.seg_state + (size_t)blockIdx.x * a.D * S;
    if (MODE != WALK && ln == 0) a.seg_sum[(size_t)blockIdx.x * a.D + c] = sum;
    if (!out) return;
    float4 *p = reinterpret_cast<float4 *>(out + (size_t)c * S + ln * M);
#pragma unroll
    for (int k = 0; k < M / 4; ++k) p[k] = make_float4(h2[2 * k].x, h2[2 * k].y, h2[2 * k + 1].x, h2[2 * k + 1].y);
}

// The segments' own states chained: seg_state[u] becomes the state at the
// start of segment u (reverse: the gradient at its end).  A thread per state.
// The decay e^{A sum d} is applied in two halves, so that a product in range
// is not lost to a factor out of it.  Eight segments' loads go out together: 38
// segments of 4096 channels 12 us (one by one, 11 of 2048 channels took 41).
__global__ void __launch_bounds__(256) kda_scan_chain_kernel(ScanArgs a, int S, bool reverse) {
    const int s = blockIdx.y;
    const long long e = (long long)blockIdx.x * 256 + threadIdx.x, size = (long long)a.D * S;
    const int b0 = a.cu_seqlens[s], b1 = a.cu_seqlens[s + 1];
    if (e >= size || b0 < 0 || b1 < b0 || b1 > a.T) return;
    const int count = (int)(((long long)b1 - b0 + a.seg - 1) / a.seg);
    if (count < 2) return;
    const int c = (int)(e / S);
    const long long u0 = b0 / a.seg + s;
    const float A = rate(a.A[e]);
    float *st = a.seg_state + u0 * size + e;
    const float *sum = a.seg_sum + u0 * a.D + c;
    const float *first = reverse ? a.dfinal : a.initial_state;
    float h = first ? first[s * size + e] : 0.f;
    // eight segments' loads at a time, then their chain
    constexpr int U = 8;
    for (int j0 = 0; j0 < count; j0 += U) {
        float own[U], k[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = min(j0 + i, count - 1), u = reverse ? count - 1 - j : j;
            own[i] = st[u * size];
            k[i] = exp2f(0.5f * (A * sum[(long long)u * a.D]));
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = j0 + i, u = reverse ? count - 1 - j : j;
            if (j >= count) break;
            st[u * size] = h;
            h = h == 0.f ? own[i] : fmaf(h * k[i], k[i], own[i]);
        }
    }
}

// One token per request, states in place.  Bytes bound it: 8 of state for a
// state, where 16 states share the channel's 8 (bf16) of x, dt, z and y.  A
// thread takes four neighbouring states (16 bytes) of four requests at a time,
// a channel S / 4 lanes, and a block walks `rows` requests with the rates A in
// registers.  The four requests' steps and outputs are dealt out to a
// channel's lanes.  256 x 8192 channels of 16 states: 51 us (5.6 TB/s); 82 with every lane
// forming all four, 58 with registers for two blocks an SM rather than four.  (32-bit rows
// spill under that cap: 66 us against 45 for their bytes, and 90 against 50 with 8 states.)
template <bool BF16, int S>
__global__ void __launch_bounds__(256, 4) kda_scan_step_kernel(ScanArgs a, int rows) {
    using E = Elem<BF16>;
    constexpr int LANES = S / 4, U = 4, OWN = LANES < U ? U / LANES : 1, DEAL = U / OWN;  // lanes that share the work
    const int lane = threadIdx.x & 31, ln = threadIdx.x % LANES, mine = ln % DEAL * OWN, per = a.D / a.G;
    const int blocks = (a.D + 256 / LANES - 1) / (256 / LANES), chunk = (int)blockIdx.x / blocks;
    const int at = ((int)blockIdx.x - chunk * blocks) * (256 / LANES) + threadIdx.x / LANES;
    const bool live = at < a.D;
    const int c = live ? at : a.D - 1, grp = c / per;
    float4 A4 = reinterpret_cast<const float4 *>(a.A + (size_t)c * S)[ln];
    const float2 A[2] = {make_float2(rate(A4.x), rate(A4.y)), make_float2(rate(A4.z), rate(A4.w))};
    const float skip = a.Dskip ? a.Dskip[c] : 0.f, bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    const E *x = static_cast<const E *>(a.x) + c, *dt = static_cast<const E *>(a.dt) + c, *z = static_cast<const E *>(a.z) + c;
    const E *B = static_cast<const E *>(a.B) + (size_t)grp * S + 4 * ln, *C = static_cast<const E *>(a.C) + (size_t)grp * S + 4 * ln;
    const int r0 = chunk * rows, r1 = min(r0 + rows, a.N);
    const size_t DS = (size_t)a.D * S;
    float *sp = a.state + r0 * DS + (size_t)c * S + 4 * ln;
    B += r0 * a.b_stride, C += r0 * a.c_stride;
    for (int r = r0; r < r1; r += U, sp += U * DS, B += U * a.b_stride, C += U * a.c_stride) {
        float4 h[U];
        Vec<BF16, 4> vb[U], vc[U];
        float xv[OWN], d[OWN], zv[OWN], in[OWN], y[U];
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const long long q = min(r + mine + j, r1 - 1);
            d[j] = (float)dt[q * a.dt_stride] + bias;
            xv[j] = (float)x[q * a.x_stride];
            zv[j] = a.z ? (float)z[q * a.z_stride] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + u >= r1) {
                h[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                vb[u].zero();
                vc[u].zero();
                continue;
            }
            h[u] = *reinterpret_cast<const float4 *>(sp + u * DS);
            const E *bp = B + u * a.b_stride, *cp = C + u * a.c_stride;
            if (a.wide_bc) {
                vb[u].load(bp);
                vc[u].load(cp);
            } else {
                const float f[4] = {(float)bp[0], (float)bp[1], (float)bp[2], (float)bp[3]};
                const float g[4] = {(float)cp[0], (float)cp[1], (float)cp[2], (float)cp[3]};
                vb[u].set(f);
                vc[u].set(g);
            }
        }
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            if (a.dt_softplus) d[j] = softplus(d[j]);
            in[j] = d[j] * xv[j];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int from = (lane & ~(LANES - 1)) + u / OWN;
            const float2 dd = both(__shfl_sync(0xffffffffu, d[u % OWN], from)), ii = both(__shfl_sync(0xffffffffu, in[u % OWN], from));
            float2 k[2] = {make_float2(h[u].x, h[u].y), make_float2(h[u].z, h[u].w)}, s = both(0.f);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 arg = __ffma2_rn(A[e], dd, both(kExp2Low));
                k[e] = __ffma2_rn(make_float2(exp2_fast(arg.x), exp2_fast(arg.y)), k[e], __fmul2_rn(ii, vb[u].pair(e)));
                s = __ffma2_rn(vc[u].pair(e), k[e], s);
            }
            y[u] = s.x + s.y;
            if (live && r + u < r1)
                *reinterpret_cast<float4 *>(sp + u * DS) = make_float4(k[0].x, k[0].y, k[1].x, k[1].y);
        }
        // a channel's lanes' shares added up, each request's in its lane
#pragma unroll
        for (int o = LANES / 2; o >= DEAL; o /= 2)
#pragma unroll
            for (int u = 0; u < U; ++u) y[u] += __shfl_xor_sync(0xffffffffu, y[u], o);
#pragma unroll
        for (int o = DEAL / 2, n = U / 2; o > 0; o /= 2, n /= 2) {
            const bool up = ln & o;
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const float send = up ? y[j] : y[j + n], keep = up ? y[j + n] : y[j];
                y[j] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            float out = fmaf(skip, xv[j], y[j]);
            if (a.z) out *= silu(zv[j]);
            if (live && ln < DEAL && r + mine + j < r1)
                static_cast<E *>(a.y)[(long long)(r + mine + j) * a.y_stride + c] = (E)out;
        }
    }
}

template <bool BF16, int S, int M, int MODE, bool VEC>
cudaError_t launch_scan_t(const ScanArgs &a, cudaStream_t st) {
    using L = Layout<BF16, S, M>;
    auto kern = kda_scan_kernel<BF16, S, M, MODE, VEC>;
    if (L::bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
        if (e != cudaSuccess) return e;
    }
    const int per = a.D / a.G, tiles = (per + L::CH - 1) / L::CH;
    kern<<<dim3(scan_units(a.N, a.T, a.seg), a.G * tiles), kThreads, L::bytes, st>>>(a);
    return cudaGetLastError();
}

template <bool BF16, int S>
cudaError_t launch_scan_s(const ScanArgs &a, int what, int sms, cudaStream_t st) {
    if (what == SCAN_STEP) {
        const int blocks = (a.D + 1024 / S - 1) / (1024 / S);
        // requests of a block: the rates are read once for them, while every SM has 16 blocks (four times what runs at once)
        int rows = 16;
        while (rows > 1 && (long long)blocks * ((a.N + rows - 1) / rows) < 16LL * sms) rows /= 2;
        kda_scan_step_kernel<BF16, S><<<blocks * ((a.N + rows - 1) / rows), 256, 0, st>>>(a, rows);
        return cudaGetLastError();
    }
    if (a.wide) {
        if (what == SCAN_FORWARD) return launch_scan_t<BF16, S, 8, FORWARD, true>(a, st);
        if (what == SCAN_REVERSE) return launch_scan_t<BF16, S, 8, REVERSE, true>(a, st);
        // 16 states a thread leave a fifth fewer instructions (no shuffles at 16 states a channel), but
        // half the warps: 16384 tokens x 4096 channels in many segments 306 us against 367, 8 sequences
        // of 2048, 1.7 blocks an SM, 566 against 404, 16 of them 733 against 688.  So where blocks fill the SMs.
        if constexpr (S >= 16) {
            using L = Layout<BF16, S, 16>;
            const int per = a.D / a.G, tiles = (per + L::CH - 1) / L::CH;
            const long long longest = a.seg ? (long long)a.T / a.seg : 0;  // segments there are at least
            if ((longest > a.N ? longest : a.N) * a.G * tiles >= 4LL * sms) return launch_scan_t<BF16, S, 16, WALK, true>(a, st);
        }
        return launch_scan_t<BF16, S, 8, WALK, true>(a, st);
    }
    if (what == SCAN_FORWARD) return launch_scan_t<BF16, S, 8, FORWARD, false>(a, st);
    if (what == SCAN_REVERSE) return launch_scan_t<BF16, S, 8, REVERSE, false>(a, st);
    return launch_scan_t<BF16, S, 8, WALK, false>(a, st);
}

}  // namespace

int scan_units(int N, int T, int seg) { return seg ? T / seg + N : N; }

int scan_channels(int S) { return kThreads * 8 / S; }

cudaError_t launch_scan(const ScanArgs &a, int S, int what, bool bf16, int sms, cudaStream_t st) {
    switch (S) {
        case 8: return bf16 ? launch_scan_s<true, 8>(a, what, sms, st) : launch_scan_s<false, 8>(a, what, sms, st);
        case 16: return bf16 ? launch_scan_s<true, 16>(a, what, sms, st) : launch_scan_s<false, 16>(a, what, sms, st);
        case 32: return bf16 ? launch_scan_s<true, 32>(a, what, sms, st) : launch_scan_s<false, 32>(a, what, sms, st);
        default: return bf16 ? launch_scan_s<true, 64>(a, what, sms, st) : launch_scan_s<false, 64>(a, what, sms, st);
    }
}

cudaError_t launch_scan_chain(const ScanArgs &a, int S, bool reverse, cudaStream_t st) {
    const long long size = (long long)a.D * S;
    kda_scan_chain_kernel<<<dim3((unsigned)((size + 255) / 256), a.N), 256, 0, st>>>(a, S, reverse);
    return cudaGetLastError();
}

}  // namespace kda
