// conv.cu -- the short causal convolution over packed sequences, its gradients,
// and single tokens.
//
//   p_t = bias + sum_j w[c][j] x_{t - (W - 1) + j},   y_t = p_t sigmoid(p_t) or p_t
// rows before a sequence come from its tail (W - 1 rows, oldest first) or are
// zero; the tail after it is the last W - 1 rows of tail and sequence together.
//   q_t = dy_t y'(p_t),  dx_e = sum_k w[c][W - 1 - k] q_{e + k} (same sequence) + what the new tail passes back
//   dw[c][j] = sum_t q_t x_{t - (W - 1) + j},  dbias = sum_t q_t
//
// What bounds it: bytes (x in, y out; backward x and dy in, dx out).  A thread
// owns V neighbouring channels (16 bytes of the forward's row) and walks a run
// of tokens, with the W - 1 rows behind it in registers; only those are read
// twice, once per run (W - 1 rows in a run of 16 to 128, and the neighbouring
// run has them in L2).  Runs do not stop at sequence ends, so short sequences
// cost no threads: where one ends the window is filled from the next one's
// tail.  The backward walks W - 1 tokens past its run, for the gradients that
// reach back into it.  Its sums for dw leave as one partial row per run and are
// added up in a fixed order.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "layer.cuh"

namespace kda {
namespace {
using namespace layer;

constexpr int kThreads = 128;
constexpr int kTailRows = 8;  // sequences of a block that writes tails

// the sequence a walk is in: tokens [a, b), b past the walk's end once there is none
struct Walk {
    int s, a, b;
};

// The first sequence from s on that has tokens at or after t and whose ends are
// in order and in [0, T]; a caller skips tokens before its start.
__device__ __forceinline__ Walk next_sequence(const int32_t *cu, int N, int T, int s, int t) {
    for (; s < N; ++s) {
        const int a = cu[s], b = cu[s + 1];
        if (a >= 0 && a < b && b <= T && b > t) return {s, a, b};
    }
    return {N, 0x7fffffff, 0x7fffffff};
}

template <bool BF16, int V>
__device__ __forceinline__ void load_row(Vec<BF16, V> &r, const Elem<BF16> *p, bool live) {
    if (live) r.load(p);
    else r.zero();
}

template <bool BF16, int V, int W>
__global__ void __launch_bounds__(kThreads) kda_conv_fwd_kernel(ConvArgs a) {
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
    float w[V][W], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[i][j] = a.w[(long long)(c + i) * W + j];
        bias[i] = a.bias ? a.bias[c + i] : 0.f;
    }
    E *y = static_cast<E *>(a.y) + c;
    Walk q = next_sequence(a.cu_seqlens, a.N, a.T, s_first, ta);
    Vec<BF16, V> win[W];  // rows t - (W - 1) .. t
    // the rows before token t of sequence q into win[0 .. W - 2]
    auto fill = [&](int t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int pos = t - q.a - (W - 1) + j;
            if (pos >= 0) win[j].load(x + (long long)(q.a + pos) * a.x_stride);
            else load_row(win[j], tail + ((long long)q.s * (W - 1) + pos + W - 1) * a.tail_stride, a.tail != nullptr);
        }
    };
    if (q.a <= ta) fill(ta);
    constexpr int U = 4;  // rows in flight
    for (int t0 = ta; t0 < tb; t0 += U) {
        Vec<BF16, V> next[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t0 + u < tb) next[u].load(x + (long long)(t0 + u) * a.x_stride);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u;
            if (t >= tb) break;
            if (t >= q.b) {
                q = next_sequence(a.cu_seqlens, a.N, a.T, q.s + 1, t);
                if (q.a < t) fill(t);
            }
            if (t < q.a) continue;  // rows of no sequence
            if (t == q.a && t > ta) fill(t);
            win[W - 1] = next[u];
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float p = bias[i];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(w[i][j], win[j].get(i), p);
                o[i] = a.act ? silu(p) : p;
            }
            Vec<BF16, V> out;
            out.set(o);
            out.store(y + (long long)t * a.y_stride);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j] = win[j + 1];
        }
    }
}

// dy of its own type (DYBF16): a following layer's gradients may be 32-bit
// beside bf16 activations.
template <bool BF16, bool DYBF16, int V, int W>
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
    float w[V][W], bias[V], dw[V][W], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[i][j] = a.w[(long long)(c + i) * W + j], dw[i][j] = 0.f;
        bias[i] = a.bias ? a.bias[c + i] : 0.f;
        db[i] = 0.f;
    }
    Walk q = next_sequence(a.cu_seqlens, a.N, a.T, s_first, ta);
    Vec<BF16, V> win[W];
    float g[W][V];  // gradients q of tokens t - (W - 1) .. t of the sequence
    auto fill = [&](int t) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int pos = t - q.a - (W - 1) + j;
            if (pos >= 0) win[j].load(x + (long long)(q.a + pos) * a.x_stride);
            else load_row(win[j], tail + ((long long)q.s * (W - 1) + pos + W - 1) * a.tail_stride, a.tail != nullptr);
#pragma unroll
            for (int i = 0; i < V; ++i) g[j][i] = 0.f;
        }
    };
    // the gradient of the row e = t - (W - 1), to which g[k] is the token k after
    // it: a row of the sequence, or of its tail where e is before its start.
    // last: e is one of the sequence's last W - 1 rows, row `last` of its new tail.
    auto emit = [&](int e, int last) {
        const bool in_tail = e < q.a;
        if (in_tail ? (!a.dtail || q.a < ta) : (e < ta || e >= tb)) return;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            o[i] = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) o[i] = fmaf(w[i][W - 1 - k], g[k][i], o[i]);
            if (last >= 0 && a.dtail_out) o[i] += a.dtail_out[((long long)q.s * (W - 1) + last) * a.C + c + i];
        }
        if (in_tail) {
#pragma unroll
            for (int i = 0; i < V; ++i) a.dtail[((long long)q.s * (W - 1) + e - q.a + W - 1) * a.C + c + i] = o[i];
        } else {
            Vec<BF16, V> out;
            out.set(o);
            out.store(dx + (long long)e * a.dx_stride);
        }
    };
    auto shift = [&] {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            win[j] = win[j + 1];
#pragma unroll
            for (int i = 0; i < V; ++i) g[j][i] = g[j + 1][i];
        }
    };
    if (q.a <= ta) fill(ta);
    constexpr int U = 4;
    const int end = min(tb + W - 1, a.T);  // the walk's own tokens end at tb
    for (int t0 = ta; t0 < end; t0 += U) {
        Vec<BF16, V> next[U];
        Vec<DYBF16, V> dnext[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t0 + u < end) {
                next[u].load(x + (long long)(t0 + u) * a.x_stride);
                dnext[u].load(dy + (long long)(t0 + u) * a.dy_stride);
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u;
            if (t >= end) break;
            if (t >= q.b) {
                q = next_sequence(a.cu_seqlens, a.N, a.T, q.s + 1, t);
                if (q.a < t) fill(t);
            }
            if (t < q.a || (t >= tb && q.a >= tb)) continue;  // rows of no sequence, or of one after the run's
            if (t == q.a && t > ta) fill(t);
            win[W - 1] = next[u];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float d = dnext[u].get(i);
                if (a.act) {
                    float p = bias[i];
#pragma unroll
                    for (int j = 0; j < W; ++j) p = fmaf(w[i][j], win[j].get(i), p);
                    const float sg = sigmoid(p);
                    d *= sg * fmaf(p, 1.f - sg, 1.f);
                }
                g[W - 1][i] = d;
                if (t < tb) {
#pragma unroll
                    for (int j = 0; j < W; ++j) dw[i][j] = fmaf(d, win[j].get(i), dw[i][j]);
                    db[i] += d;
                }
            }
            emit(t - (W - 1), -1);
            shift();
            if (t == q.b - 1) {  // nothing follows: the last W - 1 rows
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[W - 1][i] = 0.f;
                    emit(t - (W - 1) + 1 + j, j);
                    shift();
                }
            }
        }
    }
    if (!a.parts) return;
    float *out = a.parts + (long long)blockIdx.x * (W + 1) * a.C + c;  // [W + 1][C]
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) out[(long long)j * a.C + i] = dw[i][j];
        out[(long long)W * a.C + i] = db[i];
    }
}

// One token per request; tail [R][W - 1][C] moves on in place.
template <bool BF16, int V, int W>
__global__ void __launch_bounds__(kThreads) kda_conv_step_kernel(ConvArgs a) {
    using E = Elem<BF16>;
    const int tiles = (a.C + kThreads * V - 1) / (kThreads * V), r = (int)blockIdx.x / tiles;
    const int c = (((int)blockIdx.x - r * tiles) * kThreads + threadIdx.x) * V;
    if (c >= a.C) return;
    E *tail = static_cast<E *>(a.tail_out) + (long long)r * (W - 1) * a.tail_out_stride + c;
    Vec<BF16, V> win[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j].load(tail + j * a.tail_out_stride);
    win[W - 1].load(static_cast<const E *>(a.x) + (long long)r * a.x_stride + c);
    float o[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float p = a.bias ? a.bias[c + i] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(a.w[(long long)(c + i) * W + j], win[j].get(i), p);
        o[i] = a.act ? silu(p) : p;
    }
    Vec<BF16, V> out;
    out.set(o);
    out.store(static_cast<E *>(a.y) + (long long)r * a.y_stride + c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j + 1].store(tail + j * a.tail_out_stride);
}

template <int W>
cudaError_t launch_w(const ConvArgs &a, int what, bool bf16, bool dy_bf16, cudaStream_t st) {
    auto tiles = [&](int v) { return (unsigned)((a.C + kThreads * v - 1) / (kThreads * v)); };
    const unsigned gx = (unsigned)(a.runs + (a.N + kTailRows - 1) / kTailRows);
    if (what == 0) {
        if (bf16 && a.wide) kda_conv_fwd_kernel<true, 8, W><<<dim3(gx, tiles(8)), kThreads, 0, st>>>(a);
        else if (bf16) kda_conv_fwd_kernel<true, 1, W><<<dim3(gx, tiles(1)), kThreads, 0, st>>>(a);
        else if (a.wide) kda_conv_fwd_kernel<false, 4, W><<<dim3(gx, tiles(4)), kThreads, 0, st>>>(a);
        else kda_conv_fwd_kernel<false, 1, W><<<dim3(gx, tiles(1)), kThreads, 0, st>>>(a);
    } else if (what == 1) {
        // (four channels a thread: eight would hold 136 registers of windows and sums)
        const dim3 g4(gx, tiles(4)), g1(gx, tiles(1));
        if (bf16 && dy_bf16 && a.wide) kda_conv_bwd_kernel<true, true, 4, W><<<g4, kThreads, 0, st>>>(a);
        else if (bf16 && dy_bf16) kda_conv_bwd_kernel<true, true, 1, W><<<g1, kThreads, 0, st>>>(a);
        else if (bf16 && a.wide) kda_conv_bwd_kernel<true, false, 4, W><<<g4, kThreads, 0, st>>>(a);
        else if (bf16) kda_conv_bwd_kernel<true, false, 1, W><<<g1, kThreads, 0, st>>>(a);
        else if (a.wide) kda_conv_bwd_kernel<false, false, 4, W><<<g4, kThreads, 0, st>>>(a);
        else kda_conv_bwd_kernel<false, false, 1, W><<<g1, kThreads, 0, st>>>(a);
    } else {
        const unsigned R = (unsigned)a.N;
        if (bf16 && a.wide) kda_conv_step_kernel<true, 8, W><<<R * tiles(8), kThreads, 0, st>>>(a);
        else if (bf16) kda_conv_step_kernel<true, 1, W><<<R * tiles(1), kThreads, 0, st>>>(a);
        else if (a.wide) kda_conv_step_kernel<false, 4, W><<<R * tiles(4), kThreads, 0, st>>>(a);
        else kda_conv_step_kernel<false, 1, W><<<R * tiles(1), kThreads, 0, st>>>(a);
    }
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

cudaError_t launch_conv(const ConvArgs &a, int W, int what, bool bf16, bool dy_bf16, cudaStream_t st) {
    switch (W) {
        case 1: return launch_w<1>(a, what, bf16, dy_bf16, st);
        case 2: return launch_w<2>(a, what, bf16, dy_bf16, st);
        case 3: return launch_w<3>(a, what, bf16, dy_bf16, st);
        default: return launch_w<4>(a, what, bf16, dy_bf16, st);
    }
}

}  // namespace kda
