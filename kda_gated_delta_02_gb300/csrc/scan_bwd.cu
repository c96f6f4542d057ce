// scan_bwd.cu -- gradients of the selective scan, from the states that the
// forward saved before every eighth token.  With e_t the gradient of the
// gated sum, e_t = dy_t z_t sigmoid(z_t), and l_t the gradient of h_t, last token first:
//
//   l_t = C_t e_t + a_{t+1} l_{t+1},  a_t = e^{d_t A}
//   dx_t = d_t sum_n l_t B_t + D e_t,   dd_t = x_t sum_n l_t B_t + sum_n l_t A a_t h_{t-1},   ddt = dd e^v / (1 + e^v)
//   dB_t = sum over channels of l_t d_t x_t,  dC_t = sum over channels of e_t h_t
//   dA = sum_t d_t l_t a_t h_{t-1},  dD = sum_t e_t x_t,  dz_t = dy_t (sum_n C_t h_t + D x_t) sigma'(z_t)
//
// What bounds it: instructions and shared memory.  A pair of states costs 15
// packed operations and four exponentials (two of them the recomputed states'), and the sums
// of dB and dC over channels go through shared memory: 8 sequences of 2048 tokens x
// 4096 channels in 16 x 152 blocks 1.25 ms, 5.3 cycles of an SM for a token and channel, issue slots
// three quarters (packed operations take two) and shared memory 69 % busy.  A thread keeps 2 channels of 8 states; S / 8 lanes
// share a pair of channels, and the tokens' own work (steps, gates, outputs) is dealt
// out to them.  The eight tokens from a saved state run forward with every
// second token's decayed state G = a h kept in shared memory, then backward: of the
// two tokens that share it, the earlier one has what it needs (G, G + b), the
// later one goes forward from it (a (G + b), and its own b more).  The state h = G + b kept in
// its place, and G taken back as h - b, took as long, and cost a state that
// forgets to e^-10 in a token all but three digits of dA.  The sums over channels
// add two in a thread's registers, then four floats at a time in shared
// memory: 4 stores, 4 loads and 20 additions and exchanges per token, where
// exchanges alone would take 62.  A block's four warps add theirs once per eight
// tokens, and a second kernel adds the blocks' in order.  Sums along the tokens (dA, dD,
// ddt_bias) are taken over eight tokens first.  The rows of the eight tokens
// before are in registers already, those of the eight before them on their way into L2
// (1.60 ms without).  Saved states cost 8 bytes a token and channel at 16
// states, written and read once; every sixteenth token would halve them for a sixth more operations.
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

constexpr int K = kSaveEvery;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int WARPS = kThreads / 32;

template <int S>
struct Layout {
    static constexpr int M = 8, LN = S / M, PAIRS = 32 / LN, CH = 2 * PAIRS * WARPS;
    static constexpr int V4 = 2 * M / 4;           // float4s of a thread's states, and of its dB and dC
    static constexpr int hist = K / 2 * V4 * 32;   // float4s of a warp
    static constexpr int red = 2 * V4 * 32;        // two tokens'
    static constexpr int vals = 5 * K * PAIRS;     // float2s of a warp
    static constexpr int out = (K + 1) * 2 * S;    // floats of a warp (the last row takes what is of no token)
    static constexpr int bytes = WARPS * (16 * (hist + red) + 8 * vals + 4 * out) + 4 * K * 2 * S;
};

// two neighbouring channels of a row, of which `one` and `two` say which are there
template <bool BF16, bool VEC>
struct Pair {
    Vec<BF16, 2> r;
    __device__ __forceinline__ void load(const Elem<BF16> *p, bool one, bool two) {
        if constexpr (VEC) {
            if (one) r.load(p);
            else r.zero();
        } else {
            const float f[2] = {one ? (float)p[0] : 0.f, two ? (float)p[1] : 0.f};
            r.set(f);
        }
    }
    __device__ __forceinline__ float2 get() const { return r.pair(0); }
    static __device__ __forceinline__ void store(Elem<BF16> *p, float2 v, bool one, bool two) {
        if constexpr (VEC) {
            Vec<BF16, 2> r;
            r.set_pair(0, v);
            if (one) r.store(p);
        } else {
            if (one) p[0] = (Elem<BF16>)v.x;
            if (two) p[1] = (Elem<BF16>)v.y;
        }
    }
};

template <bool BF16, int S, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) kda_scan_bwd_kernel(ScanArgs a) {
    using E = Elem<BF16>;
    using L = Layout<S>;
    constexpr int LN = L::LN, M = L::M, V4 = L::V4, PAIRS = L::PAIRS, OWN = K / LN;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ln = lane / PAIRS, pl = lane % PAIRS;
    float4 *hist = reinterpret_cast<float4 *>(smem) + warp * L::hist;                              // [K / 2][V4][32]
    float4 *red = reinterpret_cast<float4 *>(smem) + WARPS * L::hist + warp * L::red;              // [2][V4][32]
    float2 *vals = reinterpret_cast<float2 *>(smem + 16 * WARPS * (L::hist + L::red)) + warp * L::vals;  // [5][K][PAIRS]
    float *outs = reinterpret_cast<float *>(smem + WARPS * (16 * (L::hist + L::red) + 8 * L::vals));    // [WARPS][K + 1][2 S]
    float *bc = outs + WARPS * L::out;                                                             // [K][2 S]
    const Segment g = segment_of(a.cu_seqlens, a.N, a.T, a.seg, blockIdx.x);
    if (tid == 0 && blockIdx.y == 0) check_sequence(a, blockIdx.x);
    const int per = a.D / a.G, tiles = (per + L::CH - 1) / L::CH;
    const int grp = blockIdx.y / tiles, tile = blockIdx.y - grp * tiles;
    const int at = tile * L::CH + 2 * (warp * PAIRS + pl), c = grp * per + (at < per ? at : 0);  // the thread's first channel
    const bool one = at < per, two = at + 1 < per;
    const int c1 = two ? c + 1 : c;
    const size_t DS = (size_t)a.D * S;

    float2 A2[2][M / 2], carry[2][M / 2], dA[2][M / 2];
    const float *from = nullptr;
    if (g.s >= 0)
        from = g.first && g.last ? (a.dfinal ? a.dfinal + g.s * DS : nullptr) : a.seg_state + blockIdx.x * DS;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const size_t o = (size_t)(q ? c1 : c) * S + ln * M;
#pragma unroll
        for (int i = 0; i < M / 4; ++i) {
            const float4 v = reinterpret_cast<const float4 *>(a.A + o)[i];
            A2[q][2 * i] = make_float2(rate(v.x), rate(v.y)), A2[q][2 * i + 1] = make_float2(rate(v.z), rate(v.w));
            const float4 w = from && (q ? two : one) ? reinterpret_cast<const float4 *>(from + o)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
            carry[q][2 * i] = make_float2(w.x, w.y), carry[q][2 * i + 1] = make_float2(w.z, w.w);
            dA[q][2 * i] = dA[q][2 * i + 1] = both(0.f);
        }
    }
    const float2 skip = a.Dskip ? make_float2(a.Dskip[c], a.Dskip[c1]) : both(0.f);
    const float2 bias = a.dt_bias ? make_float2(a.dt_bias[c], a.dt_bias[c1]) : both(0.f);
    float2 dD = both(0.f), dbias = both(0.f);
    const E *Bp = static_cast<const E *>(a.B) + (size_t)grp * S, *Cp = static_cast<const E *>(a.C) + (size_t)grp * S;
    E *dxp = static_cast<E *>(a.dx) + c, *ddtp = static_cast<E *>(a.ddt) + c, *dzp = static_cast<E *>(a.dz) + c;
    const int count = g.s < 0 ? 0 : g.t1 - g.t0;

    // the eight tokens from t on are brought into L2, while later ones are worked on
    auto ahead = [&](long long t) {
        constexpr int LINE = 128 / (int)sizeof(E), LINES = (L::CH + LINE - 1) / LINE;
        const int c0 = tile * L::CH;
        for (int i = tid; i < 4 * K * LINES; i += kThreads) {
            const int what = i / (K * LINES), k = i / LINES % K, o = c0 + i % LINES * LINE;
            const void *base = what == 0 ? a.x : what == 1 ? a.dt : what == 2 ? a.dy : a.z;
            const long long stride = what == 0 ? a.x_stride : what == 1 ? a.dt_stride : what == 2 ? a.dy_stride : a.z_stride;
            if (base && o < per) prefetch(static_cast<const E *>(base) + (t + k) * stride + grp * per + o);
        }
        if (tid < 2 * K) prefetch(tid < K ? Bp + (t + tid) * a.b_stride : Cp + (t + tid - K) * a.c_stride);
        const float *st = a.saved + (size_t)(g.slot + (t - g.t0) / K) * DS + (size_t)(grp * per + c0) * S;
        for (int i = tid * 32; i < L::CH * S; i += 32 * kThreads)
            if (c0 + i / S < per) prefetch(st + i);
    };

    // a lane's own tokens of the eight from t0 on: dt, x, dy and z as they come, asked for eight tokens ahead
    Pair<BF16, VEC> raw[4][OWN];
    auto load = [&](int t0, int rows) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            if (w == 3 && !a.z) continue;
            const long long stride = w == 0 ? a.dt_stride : w == 1 ? a.x_stride : w == 2 ? a.dy_stride : a.z_stride;
            const E *p = static_cast<const E *>(w == 0 ? a.dt : w == 1 ? a.x : w == 2 ? a.dy : a.z) + c + (long long)(t0 + ln * OWN) * stride;
#pragma unroll
            for (int j = 0; j < OWN; ++j) raw[w][j].load(p + j * stride, one && ln * OWN + j < rows, two && ln * OWN + j < rows);
        }
    };
    const int last = (count + K - 1) / K - 1;
    if (last >= 0) load(g.t0 + last * K, count - last * K);
    for (int i = last; i >= 0; --i) {
        const int t0 = g.t0 + i * K, rows = min(K, g.t1 - t0);
        // the tokens' values, dealt out to the lanes of a pair: d, x, e, d's derivative, dy sigma'(z)
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            const float2 v = __fadd2_rn(raw[0][j].get(), bias), x = raw[1][j].get();
            float2 e = raw[2][j].get(), d = v, s = both(1.f), dz = both(0.f);
            if (a.dt_softplus) d = softplus2(v, s);
            if (a.z) {
                const float2 z = raw[3][j].get(), sg = sigmoid2(z);
                dz = __fmul2_rn(e, dsilu2(z, sg));
                e = __fmul2_rn(e, __fmul2_rn(z, sg));
            }
            float2 *p = vals + (ln * OWN + j) * PAIRS + pl;
            p[0] = d, p[K * PAIRS] = x, p[2 * K * PAIRS] = e, p[3 * K * PAIRS] = s, p[4 * K * PAIRS] = dz;
        }
        if (i > 0) load(t0 - K, K);
        for (int n = 4 * tid; n < K * 2 * S; n += 4 * kThreads) {
            const int k = n / (2 * S), m = n % (2 * S);
            const long long t = t0 + (k < rows ? k : 0);
            const E *p = m < S ? Bp + t * a.b_stride + m : Cp + t * a.c_stride + m - S;
            Vec<BF16, 4> v;
            if (a.wide_bc) {
                v.load(p);
            } else {
                const float f[4] = {(float)p[0], (float)p[1], (float)p[2], (float)p[3]};
                v.set(f);
            }
            *reinterpret_cast<float4 *>(bc + n) = make_float4(v.get(0), v.get(1), v.get(2), v.get(3));
        }
        float2 h[2][M / 2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float4 *p = reinterpret_cast<const float4 *>(a.saved + (size_t)(g.slot + i) * DS + (size_t)(q ? c1 : c) * S + ln * M);
#pragma unroll
            for (int n = 0; n < M / 4; ++n) {
                const float4 v = p[n];
                h[q][2 * n] = make_float2(v.x, v.y), h[q][2 * n + 1] = make_float2(v.z, v.w);
            }
        }
        if (i > 1) ahead(t0 - 2 * K);
        __syncthreads();
        // forward, the decayed states of tokens 0, 2, 4 and 6 kept
#pragma unroll 1
        for (int k = 0; k < min(rows, K - 1); ++k) {
            const float2 d = vals[k * PAIRS + pl], x = vals[(K + k) * PAIRS + pl];
            const float4 *b4 = reinterpret_cast<const float4 *>(bc + k * 2 * S + ln * M);
            const float2 dq[2] = {both(d.x), both(d.y)}, in[2] = {both(d.x * x.x), both(d.y * x.y)};
#pragma unroll
            for (int n = 0; n < M / 4; ++n) {
                const float4 B4 = b4[n];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float2 ah[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 arg = __ffma2_rn(A2[q][2 * n + e], dq[q], both(kExp2Low)), b = e ? make_float2(B4.z, B4.w) : make_float2(B4.x, B4.y);
                        ah[e] = __fmul2_rn(make_float2(exp2_fast(arg.x), exp2_fast(arg.y)), h[q][2 * n + e]);
                        h[q][2 * n + e] = __ffma2_rn(in[q], b, ah[e]);
                    }
                    if ((k & 1) == 0) hist[((k >> 1) * V4 + q * (M / 4) + n) * 32 + lane] = make_float4(ah[0].x, ah[0].y, ah[1].x, ah[1].y);
                }
            }
        }
        float2 dAt[2][M / 2], dDt = both(0.f), dbt = both(0.f);
#pragma unroll
        for (int n = 0; n < M / 2; ++n) dAt[0][n] = dAt[1][n] = both(0.f);
        // dB and dC of token k from `red`, place buf.  Row v there is four outputs of all lanes.  A lane adds up a row
        // over the PART lanes of its part (rotated, so that eight neighbours read eight places), and parts of one ln are joined.
        auto channels = [&](int k, int buf) {
            constexpr int PARTS = 32 / V4, PART = 32 / PARTS, JOIN = PARTS / LN;
            const int v = lane / PARTS, part = lane % PARTS;
            const float4 *p = red + (buf * V4 + v) * 32 + part * PART;
            float2 f0 = both(0.f), f1 = both(0.f);
#pragma unroll
            for (int j = 0; j < PART; ++j) {
                const float4 w = p[(j + (part >> 1)) % PART];
                f0 = __fadd2_rn(f0, make_float2(w.x, w.y)), f1 = __fadd2_rn(f1, make_float2(w.z, w.w));
            }
            // outputs of the lane's part: B for rows below M / 4, C above
            const int which = v >= M / 4, n0 = (part / JOIN) * M + (v - which * (M / 4)) * 4;
            float *out = outs + (warp * (K + 1) + k) * 2 * S + which * S + n0;
            if constexpr (JOIN >= 2) {  // two lanes: each keeps two of the four
                const bool up = part & 1;
                const float2 send = up ? f0 : f1;
                float2 mine = up ? f1 : f0;
                mine.x += __shfl_xor_sync(0xffffffffu, send.x, 1), mine.y += __shfl_xor_sync(0xffffffffu, send.y, 1);
                if constexpr (JOIN >= 4) {
                    const bool up2 = part & 2;
                    const float s2 = up2 ? mine.x : mine.y;
                    float m2 = up2 ? mine.y : mine.x;
                    m2 += __shfl_xor_sync(0xffffffffu, s2, 2);
                    if constexpr (JOIN >= 8) m2 += __shfl_xor_sync(0xffffffffu, m2, 4);
                    if (JOIN < 8 || (part & 4) == 0) out[(up ? 2 : 0) + (up2 ? 1 : 0)] = m2;
                } else {
                    out[up ? 2 : 0] = mine.x, out[up ? 3 : 1] = mine.y;
                }
            } else {
                *reinterpret_cast<float4 *>(out) = make_float4(f0.x, f0.y, f1.x, f1.y);
            }
        };
        // A token back: sums over the thread's states for (lB, lA, y) of both channels, and its share of dB and dC into
        // `red`.  Those of the token before it in the walk are added up meanwhile: later tokens of a pair use place 1,
        // earlier ones place 0.
        int before = K;
        auto back = [&](auto later, int k, float2 (&sums)[3]) {
            constexpr bool LATER = decltype(later)::value;
            channels(before, !LATER ? 1 : 0);  // (no wait for them: the operations below are others)
            before = k;
            const float2 d = vals[k * PAIRS + pl], x = vals[(K + k) * PAIRS + pl], ev = vals[(2 * K + k) * PAIRS + pl];
            const float4 *b4 = reinterpret_cast<const float4 *>(bc + k * 2 * S + ln * M), *c4 = b4 + S / 4;
            const float2 dq[2] = {both(d.x), both(d.y)}, in[2] = {both(d.x * x.x), both(d.y * x.y)}, eq[2] = {both(ev.x), both(ev.y)};
            float2 in0[2];  // of the earlier token
            if constexpr (LATER) {
                const float2 d0 = vals[(k - 1) * PAIRS + pl], x0 = vals[(K + k - 1) * PAIRS + pl];
                in0[0] = both(d0.x * x0.x), in0[1] = both(d0.y * x0.y);
            }
            float2 lB[2] = {both(0.f), both(0.f)}, lA[2] = {both(0.f), both(0.f)}, y[2] = {both(0.f), both(0.f)};
#pragma unroll
            for (int n = 0; n < M / 4; ++n) {
                const float4 B4 = b4[n], C4 = c4[n];
                float4 P4;  // B of the earlier token
                if constexpr (LATER) P4 = (b4 - 2 * S / 4)[n];
                float2 sB[2], sC[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 H4 = hist[((k >> 1) * V4 + q * (M / 4) + n) * 32 + lane];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 A = A2[q][2 * n + e], arg = __ffma2_rn(A, dq[q], both(kExp2Low)), dec = make_float2(exp2_fast(arg.x), exp2_fast(arg.y));
                        const float2 B = e ? make_float2(B4.z, B4.w) : make_float2(B4.x, B4.y);
                        const float2 C = e ? make_float2(C4.z, C4.w) : make_float2(C4.x, C4.y);
                        const float2 H = e ? make_float2(H4.z, H4.w) : make_float2(H4.x, H4.y);
                        float2 ah = H;  // of the earlier token, kept
                        if constexpr (LATER) ah = __fmul2_rn(dec, __ffma2_rn(in0[q], e ? make_float2(P4.z, P4.w) : make_float2(P4.x, P4.y), H));
                        const float2 hk = __ffma2_rn(in[q], B, ah);
                        const float2 l = __ffma2_rn(C, eq[q], carry[q][2 * n + e]);
                        const float2 u = __fmul2_rn(l, ah);
                        carry[q][2 * n + e] = __fmul2_rn(dec, l);
                        lB[q] = __ffma2_rn(l, B, lB[q]);
                        lA[q] = __ffma2_rn(u, A, lA[q]);
                        dAt[q][2 * n + e] = __ffma2_rn(dq[q], u, dAt[q][2 * n + e]);
                        y[q] = __ffma2_rn(C, hk, y[q]);
                        sB[e] = q ? __ffma2_rn(l, in[q], sB[e]) : __fmul2_rn(l, in[q]);
                        sC[e] = q ? __ffma2_rn(hk, eq[q], sC[e]) : __fmul2_rn(hk, eq[q]);
                    }
                }
                red[((LATER ? V4 : 0) + n) * 32 + lane] = make_float4(sB[0].x, sB[0].y, sB[1].x, sB[1].y);
                red[((LATER ? V4 : 0) + M / 4 + n) * 32 + lane] = make_float4(sC[0].x, sC[0].y, sC[1].x, sC[1].y);
            }
            sums[0] = make_float2(lB[0].x + lB[0].y, lB[1].x + lB[1].y);
            sums[1] = make_float2(lA[0].x + lA[0].y, lA[1].x + lA[1].y);
            sums[2] = make_float2(y[0].x + y[0].y, y[1].x + y[1].y);
            __syncwarp();
        };
        // a token's own gradients, from its sums over all states
        auto finish = [&](int k, const float2 (&sums)[3]) {
            const float2 *p = vals + k * PAIRS + pl;
            const float2 d = p[0], x = p[K * PAIRS], ev = p[2 * K * PAIRS], sg = p[3 * K * PAIRS], dz = p[4 * K * PAIRS];
            const float2 dx = __ffma2_rn(d, sums[0], __fmul2_rn(skip, ev));
            const float2 dd = __fmul2_rn(__ffma2_rn(x, sums[0], __fmul2_rn(both(kLn2), sums[1])), sg);
            dDt = __ffma2_rn(ev, x, dDt);
            dbt = __fadd2_rn(dbt, dd);
            const size_t at = (size_t)(t0 + k) * a.D + c;
            Pair<BF16, VEC>::store(static_cast<E *>(a.dx) + at, dx, one, two);
            Pair<BF16, VEC>::store(static_cast<E *>(a.ddt) + at, dd, one, two);
            if (a.z) Pair<BF16, VEC>::store(static_cast<E *>(a.dz) + at, __fmul2_rn(dz, __ffma2_rn(skip, x, sums[2])), one, two);
        };
#pragma unroll 1
        for (int k = (rows - 1) & ~1; k >= 0; k -= 2) {
            const bool pair = k + 1 < rows;
            float2 late[3], early[3];
            if (pair) {
                back(std::true_type(), k + 1, late);
                if constexpr (LN == 1) finish(k + 1, late);
            } else {
                late[0] = late[1] = late[2] = both(0.f);
            }
            back(std::false_type(), k, early);
            if constexpr (LN == 1) {
                finish(k, early);
            } else {
                // the upper half of a pair's lanes takes the later token, the lower half the earlier one
                const bool up = lane & 16;
#pragma unroll
                for (int j = 0; j < 3; ++j) {
                    const float2 send = up ? early[j] : late[j], keep = up ? late[j] : early[j];
                    late[j] = make_float2(keep.x + __shfl_xor_sync(0xffffffffu, send.x, 16), keep.y + __shfl_xor_sync(0xffffffffu, send.y, 16));
#pragma unroll
                    for (int o = 8; o >= PAIRS; o >>= 1)
                        late[j] = make_float2(late[j].x + __shfl_xor_sync(0xffffffffu, late[j].x, o),
                                              late[j].y + __shfl_xor_sync(0xffffffffu, late[j].y, o));
                }
                if (ln % (LN / 2) == 0 && (pair || !up)) finish(k + up, late);
            }
        }
        channels(before, 0);
#pragma unroll
        for (int n = 0; n < M / 2; ++n) dA[0][n] = __fadd2_rn(dA[0][n], dAt[0][n]), dA[1][n] = __fadd2_rn(dA[1][n], dAt[1][n]);
        dD = __fadd2_rn(dD, dDt), dbias = __fadd2_rn(dbias, dbt);
        __syncthreads();
        for (int n = tid; n < rows * 2 * S; n += kThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) s += outs[w * L::out + n];
            const int k = n / (2 * S), m = n % (2 * S);
            a.bc_parts[(((size_t)tile * a.T + t0 + k) * a.G + grp) * (2 * S) + m] = s;
        }
    }
    // the unit's sums, zero where it has no tokens
    if constexpr (LN > 1) {
#pragma unroll
        for (int o = 16; o >= PAIRS; o >>= 1) {
            dD.x += __shfl_xor_sync(0xffffffffu, dD.x, o), dD.y += __shfl_xor_sync(0xffffffffu, dD.y, o);
            dbias.x += __shfl_xor_sync(0xffffffffu, dbias.x, o), dbias.y += __shfl_xor_sync(0xffffffffu, dbias.y, o);
        }
    }
    float *parts = a.parts + blockIdx.x * scan_parts_width(a.D, S);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (!(q ? two : one)) continue;
        const size_t o = (size_t)(c + q) * S + ln * M;
#pragma unroll
        for (int n = 0; n < M / 4; ++n) {
            *reinterpret_cast<float4 *>(parts + o + 4 * n) = make_float4(dA[q][2 * n].x, dA[q][2 * n].y, dA[q][2 * n + 1].x, dA[q][2 * n + 1].y);
            if (g.first && a.dstate)
                *reinterpret_cast<float4 *>(a.dstate + g.s * DS + o + 4 * n) =
                    make_float4(carry[q][2 * n].x, carry[q][2 * n].y, carry[q][2 * n + 1].x, carry[q][2 * n + 1].y);
        }
        if (ln == 0) parts[DS + c + q] = q ? dD.y : dD.x, parts[DS + a.D + c + q] = q ? dbias.y : dbias.x;
    }
}

// dB and dC of a token and group: the channel tiles' partial rows in order.  A
// warp per token and group; rows of no sequence are left as they were.  Bytes bound it
// (128 per token, group and 128 channels at 16 states): 16384 tokens x 32 tiles 15 us.
template <bool BF16>
__global__ void __launch_bounds__(256) kda_scan_bc_kernel(ScanArgs a, int S, int tiles) {
    using E = Elem<BF16>;
    const long long tg = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, t = (int)(tg / a.G), grp = (int)(tg - (long long)t * a.G);
    if (t >= a.T) return;
    const int s = find_sequence(a.cu_seqlens, a.N, t);
    if (s >= a.N || a.cu_seqlens[s] > t || a.cu_seqlens[s] < 0 || a.cu_seqlens[s + 1] > a.T) return;
    const size_t step = (size_t)a.T * a.G * 2 * S, at = ((size_t)t * a.G + grp) * S;
    for (int n = lane; n < 2 * S; n += 32) {
        const float *p = a.bc_parts + 2 * at + n;
        float sum = 0.f;
        int i = 0;
        for (; i + 8 <= tiles; i += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = p[(i + k) * step];
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += v[k];
        }
        for (; i < tiles; ++i) sum += p[i * step];
        if (n < S) static_cast<E *>(a.dB)[at + n] = (E)sum;
        else static_cast<E *>(a.dC)[at + n - S] = (E)sum;
    }
}

template <bool BF16, int S>
cudaError_t launch_s(const ScanArgs &a, cudaStream_t st) {
    using L = Layout<S>;
    auto kern = a.wide ? kda_scan_bwd_kernel<BF16, S, true> : kda_scan_bwd_kernel<BF16, S, false>;
    const int per = a.D / a.G, tiles = (per + L::CH - 1) / L::CH;
    if (L::bytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
        if (e != cudaSuccess) return e;
    }
    kern<<<dim3(scan_units(a.N, a.T, a.seg), a.G * tiles), kThreads, L::bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

int scan_bwd_channels(int S) { return 2 * kThreads * 8 / S; }

cudaError_t launch_scan_bwd(const ScanArgs &a, int S, bool bf16, cudaStream_t st) {
    switch (S) {
        case 8: return bf16 ? launch_s<true, 8>(a, st) : launch_s<false, 8>(a, st);
        case 16: return bf16 ? launch_s<true, 16>(a, st) : launch_s<false, 16>(a, st);
        case 32: return bf16 ? launch_s<true, 32>(a, st) : launch_s<false, 32>(a, st);
        default: return bf16 ? launch_s<true, 64>(a, st) : launch_s<false, 64>(a, st);
    }
}

cudaError_t launch_scan_bc(const ScanArgs &a, int S, bool bf16, cudaStream_t st) {
    const int per = a.D / a.G, tiles = (per + scan_bwd_channels(S) - 1) / scan_bwd_channels(S);
    const unsigned grid = (unsigned)(((long long)a.T * a.G + 7) / 8);
    if (grid == 0) return cudaSuccess;
    if (bf16) kda_scan_bc_kernel<true><<<grid, 256, 0, st>>>(a, S, tiles);
    else kda_scan_bc_kernel<false><<<grid, 256, 0, st>>>(a, S, tiles);
    return cudaGetLastError();
}

}  // namespace kda
