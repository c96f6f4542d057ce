// conv.cu -- the short causal convolution over packed sequences, its gradients,
// and single tokens.
//
//   p_t = bias + sum_j w[c][j] x_{t - (W - 1) + j},   y_t = p_t sigmoid(p_t) or p_t
// rows before a sequence come from its tail (W - 1 rows, oldest first) or are
// zero; the tail after it is the last W - 1 rows of tail and sequence together.
//   q_t = dy_t y'(p_t),  dx_e = sum_k w[c][W - 1 - k] q_{e + k} (same sequence) + what the new tail passes back
//   dw[c][j] = sum_t q_t x_{t - (W - 1) + j},  dbias = sum_t q_t
//
// What bounds it: bytes (x in, y out; backward x and dy in, dx out), and nearly
// as much the instructions, which go in packed pairs of channels.  A thread owns four
// neighbouring channels and walks a run of tokens, with the W - 1 rows behind
// it in registers and the next four rows asked for; only W - 1 rows of a run of
// 8 to 128 are read twice, and the neighbouring run has them in L2.  Runs do
// not stop at sequence ends, so short sequences cost no threads: where one ends
// the window is filled from the next one's tail, token by token; four tokens of
// one sequence go without such checks.  The backward walks W - 1 tokens past
// its run, for the gradients that reach back into it.  Its sums for dw leave as
// one partial row per run and are added up in a fixed order.
// 16384 tokens x 8192 channels, bf16: forward 97 us (5.5 TB/s), backward 160 us
// (5.0 TB/s) and 10 for the sums; 16384 ragged tokens x 36864 channels 436 us (6.1
// TB/s).  Eight channels a thread with checks at every token took 149 us, 64
// registers (eight blocks an SM) rather than 71 gained 5 %; two channels a thread in
// the backward lost 16 %, its 123 registers forced to 102 spill and double it.  That
// backward is four blocks an SM that wait for rows asked for: latency.  All of this for
// bf16.  32-bit rows: forward 217 us (4.9 TB/s; 104 bytes of spills under the 64 registers), backward
// 277; 32-bit dy beside bf16 rows (144 registers, three blocks an SM) 218, where dy of bf16
// takes 174 measured the same way, after a flush of L2.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "layer.cuh"

namespace kda {
namespace {
using namespace layer;

constexpr int kThreads = 128;
constexpr int U = 4;          // rows asked for while as many are worked on
constexpr int kTailRows = 8;  // sequences of a block that writes tails

// the sequence a walk is in: tokens [a, b), b past the walk's end once there is none
struct Walk {
    int s, a, b;
};

// The first sequence from s on that has tokens at or after t and whose ends are
// in order and in [0, T]; a caller skips tokens before its start.
__device__ __forceinline__ Walk next_sequence(const int32_t *cu, int N, int T, int s, int t) {
    for (; s < N; ++s) {
        if (cu[s + 1] <= t) {  // empty ones, and as many as there are: by bisection
            int lo = s + 1, hi = N;
            while (lo < hi) {
                const int mid = lo + (hi - lo) / 2;
                if (cu[mid + 1] > t) hi = mid;
                else lo = mid + 1;
            }
            s = lo;
            if (s >= N) break;
        }
        const int a = cu[s], b = cu[s + 1];
        if (a >= 0 && a < b && b <= T && b > t) return {s, a, b};
    }
    return {N, 0x7fff0000, 0x7fff0000};  // past any T, with room for sums
}

// a row of pairs of channels, as loaded from p or zero
template <bool BF16, int V>
__device__ __forceinline__ void load_pairs(float2 (&x)[(V + 1) / 2], const Elem<BF16> *p, bool live) {
    Vec<BF16, V> r;
    if (live) r.load(p);
    else r.zero();
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) x[i] = r.pair(i);
}

// taps [pairs][W] and bias of channels c .. c + V - 1
template <int V, int W>
__device__ __forceinline__ void load_taps(float2 (&w)[(V + 1) / 2][W], float2 (&bias)[(V + 1) / 2], const float *wp,
                                          const float *bp, int c) {
    float t[(V + 1) / 2 * 2][W];
#pragma unroll
    for (int i = 0; i < (V + 1) / 2 * 2; ++i) {
        const float *p = wp + (long long)(c + (i < V ? i : 0)) * W;
        if constexpr (W == 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p);
            t[i][0] = q.x, t[i][1] = q.y, t[i][2] = q.z, t[i][3] = q.w;
        } else if constexpr (W == 2) {
            const float2 q = *reinterpret_cast<const float2 *>(p);
            t[i][0] = q.x, t[i][1] = q.y;
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) t[i][j] = p[j];
        }
    }
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[i][j] = make_float2(t[2 * i][j], t[2 * i + 1][j]);
        bias[i] = bp ? make_float2(bp[c + 2 * i], V > 1 ? bp[c + 2 * i + 1] : 0.f) : both(0.f);
    }
}

template <bool BF16, int V>
__device__ __forceinline__ void load_row(Vec<BF16, V> &r, const Elem<BF16> *p, bool live) {
    if (live) r.load(p);
    else r.zero();
}

template <bool BF16, int V, int W, bool ACT>
__global__ void __launch_bounds__(kThreads, 8) kda_conv_fwd_kernel(ConvArgs a) {
    using E = Elem<BF16>;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
    const bool live = c < a.C;
    const E *x = static_cast<const E *>(a.x) + c, *tail = static_cast<const E *>(a.tail) + c;
    if ((int)blockIdx.x >= a.runs) {
        // the tails after the sequences, and the check of their ends
        const int s0 = ((int)blockIdx.x - a.runs) * kTailRows;
        for (int s = s0; s < min(s0 + kTailRows, a.N); ++s) {
            const int b0 = a.cu_seqlens[s], b1 = a.cu_seqlens[s + 1];
            if (b0 < 0 || b1 < b0 || b1 > a.T) {
                if (threadIdx.x == 0 && blockIdx.y == 0) report_status(a.status, KDA_STATUS_BAD_SEQLENS);
                continue;
            }
            if (!a.tail_out || !live) continue;
            E *out = static_cast<E *>(a.tail_out) + c;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const int pos = b1 - b0 - (W - 1) + j;  // in the sequence; negative: in its old tail
                Vec<BF16, V> r;
                if (pos >= 0) r.load(x + (long long)(b0 + pos) * a.x_stride);
                else load_row(r, tail + ((long long)s * (W - 1) + pos + W - 1) * a.tail_stride, a.tail != nullptr);
                r.store(out + ((long long)s * (W - 1) + j) * a.tail_out_stride);
            }
        }
        return;
    }
    const int ta = (int)blockIdx.x * a.run, tb = min(ta + a.run, a.T);
    const int s_first = find_sequence(a.cu_seqlens, a.N, ta);
    if (!live) return;
    constexpr int P = (V + 1) / 2;
    float2 w[P][W], bias[P], win[W][P];  // taps; rows t - (W - 1) .. t
    load_taps<V, W>(w, bias, a.w, a.bias, c);
    E *y = static_cast<E *>(a.y) + c;
    Walk q = next_sequence(a.cu_seqlens, a.N, a.T, s_first, ta);
    // the rows before token t of sequence q
    auto fill = [&](int t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int pos = t - q.a - (W - 1) + j;
            if (pos >= 0) load_pairs<BF16, V>(win[j], x + (long long)(q.a + pos) * a.x_stride, true);
            else load_pairs<BF16, V>(win[j], tail + ((long long)q.s * (W - 1) + pos + W - 1) * a.tail_stride, a.tail != nullptr);
        }
    };
    if (q.a <= ta) fill(ta);
    // the output of the row that win[W - 1] holds, and the window moved on
    auto token = [&](E *to) {
        Vec<BF16, V> out;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 p = bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) p = __ffma2_rn(w[i][j], win[j][i], p);
            out.set_pair(i, ACT ? silu2(p) : p);
        }
        out.store(to);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i];
    };
    Vec<BF16, V> next[U];
    const E *ahead = x + (long long)ta * a.x_stride;  // of the rows asked for next
    auto ask = [&](int t0) {
#pragma unroll
        for (int u = 0; u < U; ++u, ahead += a.x_stride)
            if (t0 + u < tb) next[u].load(ahead);
    };
    ask(ta);
    E *yp = y + (long long)ta * a.y_stride;
#pragma unroll 1
    for (int t0 = ta; t0 < tb; t0 += U) {
        Vec<BF16, V> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
        ask(t0 + U);
        if (q.a <= t0 && t0 + U <= min(tb, q.b)) {  // all of one sequence
            if (t0 == q.a && t0 > ta) fill(t0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < P; ++i) win[W - 1][i] = now[u].pair(i);
                token(yp);
                yp += a.y_stride;
            }
        } else {
#pragma unroll 1
            for (int t = t0; t < min(t0 + U, tb); ++t) {
                if (t >= q.b) {
                    q = next_sequence(a.cu_seqlens, a.N, a.T, q.s + 1, t);
                    if (q.a < t) fill(t);
                }
                if (t < q.a) continue;  // rows of no sequence
                if (t == q.a && t > ta) fill(t);
                load_pairs<BF16, V>(win[W - 1], x + (long long)t * a.x_stride, true);
                token(y + (long long)t * a.y_stride);
            }
            yp += U * a.y_stride;
        }
    }
}

// dy of its own type (DYBF16): a following layer's gradients may be 32-bit
// beside bf16 activations.
template <bool BF16, bool DYBF16, int V, int W, bool ACT>
__global__ void __launch_bounds__(kThreads) kda_conv_bwd_kernel(ConvArgs a) {
    using E = Elem<BF16>;
    using G = Elem<DYBF16>;
    const int c = (blockIdx.y * kThreads + threadIdx.x) * V;
    const bool live = c < a.C;
    const E *x = static_cast<const E *>(a.x) + c, *tail = static_cast<const E *>(a.tail) + c;
    if ((int)blockIdx.x >= a.runs) {
        // sequences without tokens pass their tail's gradient on
        const int s0 = ((int)blockIdx.x - a.runs) * kTailRows;
        for (int s = s0; s < min(s0 + kTailRows, a.N); ++s) {
            const int b0 = a.cu_seqlens[s], b1 = a.cu_seqlens[s + 1];
            if (b0 < 0 || b1 < b0 || b1 > a.T) {
                if (threadIdx.x == 0 && blockIdx.y == 0) report_status(a.status, KDA_STATUS_BAD_SEQLENS);
                continue;
            }
            if (b1 > b0 || !a.dtail || !live) continue;
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const long long at = ((long long)s * (W - 1) + j) * a.C + c + i;
                    a.dtail[at] = a.dtail_out ? a.dtail_out[at] : 0.f;
                }
        }
        return;
    }
    const int ta = (int)blockIdx.x * a.run, tb = min(ta + a.run, a.T);
    const int s_first = find_sequence(a.cu_seqlens, a.N, ta);
    if (!live) return;
    const G *dy = static_cast<const G *>(a.dy) + c;
    E *dx = static_cast<E *>(a.dx) + c;
    constexpr int P = (V + 1) / 2;
    float2 w[P][W], bias[P], dw[P][W], db[P], win[W][P], g[W][P];  // g: gradients q of tokens t - (W - 1) .. t
    load_taps<V, W>(w, bias, a.w, a.bias, c);
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) dw[i][j] = both(0.f);
        db[i] = both(0.f);
    }
    Walk q = next_sequence(a.cu_seqlens, a.N, a.T, s_first, ta);
    auto fill = [&](int t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int pos = t - q.a - (W - 1) + j;
            if (pos >= 0) load_pairs<BF16, V>(win[j], x + (long long)(q.a + pos) * a.x_stride, true);
            else load_pairs<BF16, V>(win[j], tail + ((long long)q.s * (W - 1) + pos + W - 1) * a.tail_stride, a.tail != nullptr);
#pragma unroll
            for (int i = 0; i < P; ++i) g[j][i] = both(0.f);
        }
    };
    // the gradient of the row e = t - (W - 1), to which g[k] is the token k after
    // it: a row of the sequence, or of its tail where e is before its start.
    // last: e is one of the sequence's last W - 1 rows, row `last` of its new tail.
    auto emit = [&](int e, int last) {
        const bool in_tail = e < q.a;
        if (in_tail ? (!a.dtail || q.a < ta) : (e < ta || e >= tb)) return;
        float2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            o[i] = both(0.f);
#pragma unroll
            for (int k = 0; k < W; ++k) o[i] = __ffma2_rn(w[i][W - 1 - k], g[k][i], o[i]);
            if (last >= 0 && a.dtail_out) {
                const float *p = a.dtail_out + ((long long)q.s * (W - 1) + last) * a.C + c + 2 * i;
                o[i].x += p[0];
                if (V > 1) o[i].y += p[1];
            }
        }
        if (in_tail) {
            float *p = a.dtail + ((long long)q.s * (W - 1) + e - q.a + W - 1) * a.C + c;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                p[2 * i] = o[i].x;
                if (V > 1) p[2 * i + 1] = o[i].y;
            }
        } else {
            Vec<BF16, V> out;
#pragma unroll
            for (int i = 0; i < P; ++i) out.set_pair(i, o[i]);
            out.store(dx + (long long)e * a.dx_stride);
        }
    };
    auto shift = [&] {
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int i = 0; i < P; ++i) win[j][i] = win[j + 1][i], g[j][i] = g[j + 1][i];
    };
    if (q.a <= ta) fill(ta);
    // q of the token whose row win[W - 1] holds, from its dy in g[W - 1]
    auto token = [&](bool own) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 d = g[W - 1][i];
            if constexpr (ACT) {
                float2 p = bias[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = __ffma2_rn(w[i][j], win[j][i], p);
                d = __fmul2_rn(d, dsilu2(p, sigmoid2(p)));
            }
            g[W - 1][i] = d;
            if (own) {
#pragma unroll
                for (int j = 0; j < W; ++j) dw[i][j] = __ffma2_rn(d, win[j][i], dw[i][j]);
                db[i] = __fadd2_rn(db[i], d);
            }
        }
    };
    const int end = min(tb + W - 1, a.T);  // the walk's own tokens end at tb
    Vec<BF16, V> next[U];
    Vec<DYBF16, V> dnext[U];
    const E *ahead = x + (long long)ta * a.x_stride;
    const G *dahead = dy + (long long)ta * a.dy_stride;
    auto ask = [&](int t0) {
#pragma unroll
        for (int u = 0; u < U; ++u, ahead += a.x_stride, dahead += a.dy_stride)
            if (t0 + u < tb) {
                next[u].load(ahead);
                dnext[u].load(dahead);
            }
    };
    ask(ta);
    E *to = dx + ((long long)ta - (W - 1)) * a.dx_stride;  // of the row that token t0 completes
#pragma unroll 1
    for (int t0 = ta; t0 < end; t0 += U) {
        Vec<BF16, V> now[U];
        Vec<DYBF16, V> dnow[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u], dnow[u] = dnext[u];
        ask(t0 + U);
        if (max(ta, q.a) + W - 1 <= t0 && t0 + U <= tb && t0 + U < q.b) {  // all of one sequence and the run, and what they emit
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < P; ++i) win[W - 1][i] = now[u].pair(i), g[W - 1][i] = dnow[u].pair(i);
                token(true);
                Vec<BF16, V> out;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float2 o = both(0.f);
#pragma unroll
                    for (int k = 0; k < W; ++k) o = __ffma2_rn(w[i][W - 1 - k], g[k][i], o);
                    out.set_pair(i, o);
                }
                out.store(to);
                to += a.dx_stride;
                shift();
            }
        } else {
            to += U * a.dx_stride;
#pragma unroll 1
            for (int t = t0; t < min(t0 + U, end); ++t) {
                if (t >= q.b) {
                    q = next_sequence(a.cu_seqlens, a.N, a.T, q.s + 1, t);
                    if (q.a < t) fill(t);
                }
                if (t < q.a || (t >= tb && q.a >= tb)) continue;  // rows of no sequence, or of one after the run's
                if (t == q.a && t > ta) fill(t);
                load_pairs<BF16, V>(win[W - 1], x + (long long)t * a.x_stride, true);
                load_pairs<DYBF16, V>(g[W - 1], dy + (long long)t * a.dy_stride, true);
                token(t < tb);
                emit(t - (W - 1), -1);
                shift();
                if (t == q.b - 1) {  // nothing follows: the last W - 1 rows
#pragma unroll 1
                    for (int j = 0; j < W - 1; ++j) {
#pragma unroll
                        for (int i = 0; i < P; ++i) g[W - 1][i] = both(0.f);
                        emit(t - (W - 1) + 1 + j, j);
                        shift();
                    }
                }
            }
        }
    }
    if (!a.parts) return;
    float *out = a.parts + (long long)blockIdx.x * (W + 1) * a.C + c;  // [W + 1][C]
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 v = j < W ? dw[i][j < W ? j : 0] : db[i];
            out[(long long)j * a.C + 2 * i] = v.x;
            if (V > 1) out[(long long)j * a.C + 2 * i + 1] = v.y;
        }
}

// One token per request; tail [R][W - 1][C] moves on in place.  A block takes
// `run` requests, so that the taps (16 bytes a channel, as many as two bf16
// tails) are read once for them.  256 x 36864 channels, bf16: 31.4 us with other tails
// each time (4.8 TB/s), 26 with part of them in L2; 32-bit 54 (5.6 TB/s).  The tail is written in
// place, so a request's rows are asked for only after the one before has stored its
// own: loads in flight bound it, not bytes (17 stalls on them per instruction issued).
template <bool BF16, int V, int W>
__global__ void __launch_bounds__(kThreads) kda_conv_step_kernel(ConvArgs a) {
    using E = Elem<BF16>;
    constexpr int P = (V + 1) / 2;
    const int tiles = (a.C + kThreads * V - 1) / (kThreads * V), chunk = (int)blockIdx.x / tiles;
    const int c = (((int)blockIdx.x - chunk * tiles) * kThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    float2 w[P][W], bias[P];
    load_taps<V, W>(w, bias, a.w, a.bias, c);
    const int r1 = min((chunk + 1) * a.run, a.N);
#pragma unroll 2
    for (int r = chunk * a.run; r < r1; ++r) {
        E *tail = static_cast<E *>(a.tail_out) + (long long)r * (W - 1) * a.tail_out_stride + c;
        Vec<BF16, V> win[W], out;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j].load(tail + j * a.tail_out_stride);
        win[W - 1].load(static_cast<const E *>(a.x) + (long long)r * a.x_stride + c);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float2 p = bias[i];
#pragma unroll
            for (int j = 0; j < W; ++j) p = __ffma2_rn(w[i][j], win[j].pair(i), p);
            out.set_pair(i, a.act ? silu2(p) : p);
        }
        out.store(static_cast<E *>(a.y) + (long long)r * a.y_stride + c);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j + 1].store(tail + j * a.tail_out_stride);
    }
}

unsigned tiles(const ConvArgs &a, int v) { return (unsigned)((a.C + kThreads * v - 1) / (kThreads * v)); }

template <int W, bool ACT>
cudaError_t launch_walk(const ConvArgs &a, bool backward, bool bf16, bool dy_bf16, cudaStream_t st) {
    const int v = a.wide ? 4 : 1;
    const dim3 grid((unsigned)(a.runs + (a.N + kTailRows - 1) / kTailRows), tiles(a, v));
    auto go = [&](void (*kern)(ConvArgs)) {
        kern<<<grid, kThreads, 0, st>>>(a);
        return cudaGetLastError();
    };
    if (!backward) {
        if (bf16) return go(a.wide ? kda_conv_fwd_kernel<true, 4, W, ACT> : kda_conv_fwd_kernel<true, 1, W, ACT>);
        return go(a.wide ? kda_conv_fwd_kernel<false, 4, W, ACT> : kda_conv_fwd_kernel<false, 1, W, ACT>);
    }
    if (bf16 && dy_bf16) return go(a.wide ? kda_conv_bwd_kernel<true, true, 4, W, ACT> : kda_conv_bwd_kernel<true, true, 1, W, ACT>);
    if (bf16) return go(a.wide ? kda_conv_bwd_kernel<true, false, 4, W, ACT> : kda_conv_bwd_kernel<true, false, 1, W, ACT>);
    return go(a.wide ? kda_conv_bwd_kernel<false, false, 4, W, ACT> : kda_conv_bwd_kernel<false, false, 1, W, ACT>);
}

template <int W>
cudaError_t launch_w(const ConvArgs &a, int what, bool bf16, bool dy_bf16, cudaStream_t st) {
    if (what < 2) return a.act ? launch_walk<W, true>(a, what == 1, bf16, dy_bf16, st) : launch_walk<W, false>(a, what == 1, bf16, dy_bf16, st);
    const unsigned R = (unsigned)a.runs;
    if (bf16 && a.wide) kda_conv_step_kernel<true, 8, W><<<R * tiles(a, 8), kThreads, 0, st>>>(a);
    else if (bf16) kda_conv_step_kernel<true, 1, W><<<R * tiles(a, 1), kThreads, 0, st>>>(a);
    else if (a.wide) kda_conv_step_kernel<false, 4, W><<<R * tiles(a, 4), kThreads, 0, st>>>(a);
    else kda_conv_step_kernel<false, 1, W><<<R * tiles(a, 1), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Tokens of a run: long ones read fewer rows twice and (backward) leave fewer
// partial rows; short ones give every SM eight blocks or more.
int conv_run(int T, int C, int v, bool backward, int sms) {
    const long long tiles = (C + kThreads * v - 1) / (kThreads * v);
    int run = backward ? 128 : 64;
    while (run > 8 && tiles * ((T + run - 1) / run) < 8LL * sms) run /= 2;
    return run;
}

// Requests of a block of single tokens: up to 16, while every SM has 4 blocks
// (256 x 36864 channels, part of the tails in L2: 26.0 us, with 2 blocks 27.7, with 16 30.9)
int conv_step_run(int R, int C, int v, int sms) {
    const long long tiles = (C + kThreads * v - 1) / (kThreads * v);
    int run = 16;
    while (run > 1 && tiles * ((R + run - 1) / run) < 4LL * sms) run /= 2;
    return run;
}

cudaError_t launch_conv(const ConvArgs &a, int W, int what, bool bf16, bool dy_bf16, cudaStream_t st) {
    switch (W) {
        case 1: return launch_w<1>(a, what, bf16, dy_bf16, st);
        case 2: return launch_w<2>(a, what, bf16, dy_bf16, st);
        case 3: return launch_w<3>(a, what, bf16, dy_bf16, st);
        default: return launch_w<4>(a, what, bf16, dy_bf16, st);
    }
}

}  // namespace kda
