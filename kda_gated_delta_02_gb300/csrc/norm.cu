// norm.cu -- RMS and layer norm of rows, and their gradients.
//
//   m = mean(x) (layer; 0 for rms),  r = 1 / sqrt(mean((x - m)^2) + eps),  n = (x - m) r,  y = n w + b
//   u = dy w,  dx = r (u - n mean(u n) - mean(u) [layer only])
//   dw = sum over rows of dy n,  db = sum over rows of dy
//
// What bounds it: bytes.  A row is read once and stays in registers through
// its sums (the variance from the differences, so that a large mean costs no
// digits); the backward reads x and dy and forms the row's statistics again
// from x, which costs no bytes and leaves nothing to keep between the passes.
// A row takes THREADS threads of a block (8 for the narrowest, so that a warp
// holds four; 512 for the widest) and a block walks several rows, each thread
// always at the same channels: weights stay in its registers, and so do the
// sums of the weights' gradients over its rows.  Those leave as one partial
// row per block and are added up in a fixed order by a second kernel: the same
// inputs give the same bits.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"
#include "layer.cuh"

namespace kda {
namespace {
using namespace layer;

// the sums of x[..] over the THREADS threads of a row; every one of them gets
// them.  Rows of more than a warp: one row per block at a time; buf holds a
// sum per warp, in two places by turns, so that one barrier is enough.
template <int THREADS, int N>
__device__ __forceinline__ void row_sums(float (&x)[N], float (*buf)[N][THREADS > 32 ? THREADS / 32 : 4], int &turn) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = (THREADS < 32 ? THREADS : 32) / 2; o > 0; o >>= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
    if constexpr (THREADS > 32) {
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) buf[turn][k][threadIdx.x >> 5] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float2 s = both(0.f);
#pragma unroll
            for (int i = 0; i < THREADS / 32; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&buf[turn][k][i]);
                s = __fadd2_rn(s, __fadd2_rn(make_float2(v.x, v.y), make_float2(v.z, v.w)));
            }
            x[k] = s.x + s.y;
        }
        turn ^= 1;
    }
}

// rows of a block at a time.  (A row of 32 threads or fewer shares a block
// with others; wider rows take whole blocks, of their own width.)
template <int THREADS>
__host__ __device__ constexpr int block_rows() { return THREADS > 32 ? 1 : 256 / THREADS; }
template <int THREADS>
__host__ __device__ constexpr int block_size() { return THREADS > 32 ? THREADS : 256; }

template <bool BF16, int V, int THREADS, int ITERS>
struct Row {
    using E = Elem<BF16>;
    Vec<BF16, V> raw[ITERS];
    __device__ __forceinline__ void load(const E *p, int lane, int d) {
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c < d) raw[i].load(p + c);
            else raw[i].zero();
        }
    }
};

// A thread's channels of a weight or bias: in registers where they are few,
// read again for every row (from L1) where a row takes many.
template <int V, int THREADS, int ITERS>
struct Channels {
    static constexpr bool HELD = V * ITERS <= 8;
    const float *p;
    float none;
    int lane, d;
    float held[HELD ? ITERS : 1][V];
    __device__ __forceinline__ Channels(const float *p, float none, int lane, int d) : p(p), none(none), lane(lane), d(d) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < ITERS; ++i) fetch(i, held[i]);
        }
    }
    __device__ __forceinline__ void fetch(int i, float (&x)[V]) const {
        const int c = (i * THREADS + lane) * V;
        if (!p || c >= d) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = none;
        } else if constexpr (V >= 4) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(p + c + j));
                x[j] = q.x, x[j + 1] = q.y, x[j + 2] = q.z, x[j + 3] = q.w;
            }
        } else {
            x[0] = __ldg(p + c);
        }
    }
    __device__ __forceinline__ void get(int i, float (&x)[V]) const {
        if constexpr (HELD) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = held[i][j];
        } else {
            fetch(i, x);
        }
    }
};

// rows asked for ahead: one, where two fit into the registers
template <int V, int ITERS>
__host__ __device__ constexpr bool ahead() { return V * ITERS <= 16; }

template <bool BF16, int V, int THREADS, int ITERS, bool LAYER>
__global__ void __launch_bounds__(block_size<THREADS>())
kda_norm_fwd_kernel(NormArgs a) {
    using E = Elem<BF16>;
    constexpr int ROWS = block_rows<THREADS>();
    constexpr bool AHEAD = ahead<V, ITERS>();
    __shared__ __align__(16) float buf[2][1][THREADS > 32 ? THREADS / 32 : 4];
    int turn = 0;
    const int lane = threadIdx.x % THREADS, d = a.d;
    const float inv_d = 1.f / (float)d;
    const E *x = static_cast<const E *>(a.x);
    E *y = static_cast<E *>(a.y);
    const Channels<V, THREADS, ITERS> weight(a.weight, 1.f, lane, d), bias(a.bias, 0.f, lane, d);
    // every thread of a warp makes the same number of turns: the sums are warp-wide
    const long long step = (long long)gridDim.x * ROWS;
    long long base = (long long)blockIdx.x * ROWS;
    auto row_of = [&](long long b) { return min(b + threadIdx.x / THREADS, a.rows - 1); };
    Row<BF16, V, THREADS, ITERS> r, next;
    if (AHEAD) next.load(x + row_of(base) * a.x_stride, lane, d);
    for (; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / THREADS;
        if constexpr (AHEAD) {
            r = next;
            if (base + step < a.rows) next.load(x + row_of(base + step) * a.x_stride, lane, d);
        } else {
            r.load(x + row_of(base) * a.x_stride, lane, d);
        }
        float m = 0.f, s[1];
        if constexpr (LAYER) {
            s[0] = 0.f;
#pragma unroll
            for (int i = 0; i < ITERS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] += r.raw[i].get(j);
            row_sums<THREADS>(s, buf, turn);
            m = s[0] * inv_d;
        }
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const bool in = (i * THREADS + lane) * V < d;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float c = in ? r.raw[i].get(j) - m : 0.f;
                s[0] = fmaf(c, c, s[0]);
            }
        }
        row_sums<THREADS>(s, buf, turn);
        const float rs = rsqrtf(s[0] * inv_d + a.eps);
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c >= d) continue;
            float o[V], w[V], b[V];
            weight.get(i, w);
            bias.get(i, b);
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = fmaf((r.raw[i].get(j) - m) * rs, w[j], b[j]);
            Vec<BF16, V> out;
            out.set(o);
            out.store(y + row * a.y_stride + c);
        }
    }
}

// ACC: the sums over rows live in shared memory, a place per thread and
// channel, where registers would not hold them beside two rows.
template <bool BF16, int V, int THREADS, int ITERS, bool LAYER>
__global__ void __launch_bounds__(block_size<THREADS>())
kda_norm_bwd_kernel(NormArgs a) {
    using E = Elem<BF16>;
    constexpr int ROWS = block_rows<THREADS>(), BLOCK = block_size<THREADS>();
    constexpr bool ACC = V * ITERS > 16, AHEAD = ahead<V, ITERS>();
    extern __shared__ float acc[];  // ACC: [2][ITERS * V][THREADS]; else [ROWS][2][d] when ROWS > 1
    __shared__ __align__(16) float buf1[2][1][THREADS > 32 ? THREADS / 32 : 4], buf3[2][3][THREADS > 32 ? THREADS / 32 : 4];
    int turn1 = 0, turn3 = 0;
    const int lane = threadIdx.x % THREADS, d = a.d;
    const float inv_d = 1.f / (float)d;
    const E *x = static_cast<const E *>(a.x), *dy = static_cast<const E *>(a.dy);
    E *dx = static_cast<E *>(a.dx);
    const Channels<V, THREADS, ITERS> weight(a.weight, 1.f, lane, d);
    float dw[ACC ? 1 : ITERS][V], db[ACC ? 1 : ITERS][V];
    if constexpr (ACC) {
        for (int i = threadIdx.x; i < 2 * ITERS * V * THREADS; i += BLOCK) acc[i] = 0.f;
        __syncthreads();
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) dw[i][j] = db[i][j] = 0.f;
    }
    const long long step = (long long)gridDim.x * ROWS;
    long long base = (long long)blockIdx.x * ROWS;
    auto row_of = [&](long long b) { return min(b + threadIdx.x / THREADS, a.rows - 1); };
    Row<BF16, V, THREADS, ITERS> r, g, next, gnext;
    auto load = [&](Row<BF16, V, THREADS, ITERS> &r, Row<BF16, V, THREADS, ITERS> &g, long long b) {
        r.load(x + row_of(b) * a.x_stride, lane, d);
        g.load(dy + row_of(b) * a.dy_stride, lane, d);
    };
    if (AHEAD) load(next, gnext, base);
    for (; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / THREADS;
        if constexpr (AHEAD) {
            r = next, g = gnext;
            if (base + step < a.rows) load(next, gnext, base + step);
        } else {
            load(r, g, base);
        }
        float m = 0.f;
        if constexpr (LAYER) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < ITERS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s[0] += r.raw[i].get(j);
            row_sums<THREADS>(s, buf1, turn1);
            m = s[0] * inv_d;
        }
        float s[3] = {0.f, 0.f, 0.f};  // of (x - m)^2, u (x - m) and u
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const bool in = (i * THREADS + lane) * V < d;
            float w[V];
            weight.get(i, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float c = in ? r.raw[i].get(j) - m : 0.f, u = g.raw[i].get(j) * w[j];
                s[0] = fmaf(c, c, s[0]);
                s[1] = fmaf(u, c, s[1]);
                s[2] += u;
            }
        }
        row_sums<THREADS>(s, buf3, turn3);
        const float rs = rsqrtf(s[0] * inv_d + a.eps), k = s[1] * inv_d * rs, us = LAYER ? s[2] * inv_d : 0.f;
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c >= d) continue;
            float o[V], w[V];
            weight.get(i, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = (r.raw[i].get(j) - m) * rs, e = g.raw[i].get(j);
                o[j] = rs * (fmaf(e, w[j], -us) - n * k);
                if constexpr (ACC) {
                    float *p = acc + (i * V + j) * THREADS + lane;
                    p[0] = fmaf(e, n, p[0]);
                    p[ITERS * V * THREADS] += e;
                } else {
                    dw[i][j] = fmaf(e, n, dw[i][j]);
                    db[i][j] += e;
                }
            }
            Vec<BF16, V> out;
            out.set(o);
            out.store(dx + row * a.dx_stride + c);
        }
    }
    if (!a.parts) return;
    // one partial row of dw and db per block: parts [blocks][2][d]
    float *out = a.parts + (size_t)blockIdx.x * 2 * d;
    if constexpr (ROWS > 1) {
        __syncthreads();
        float *mine = acc + (threadIdx.x / THREADS) * 2 * d;
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (i * THREADS + lane) * V + j;
                if (c < d) mine[c] = dw[i][j], mine[d + c] = db[i][j];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * d; c += BLOCK) {
            float s = 0.f;
            for (int k = 0; k < ROWS; ++k) s += acc[k * 2 * d + c];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (i * THREADS + lane) * V + j;
                if (c >= d) continue;
                if constexpr (ACC) {
                    const float *p = acc + (i * V + j) * THREADS + lane;
                    out[c] = p[0], out[d + c] = p[ITERS * V * THREADS];
                } else {
                    out[c] = dw[i][j], out[d + c] = db[i][j];
                }
            }
    }
}

}  // namespace

// Sums of partial rows, in the order of a fixed tree: 32 columns and 32 shares
// of the rows per block.
namespace {
__global__ void __launch_bounds__(1024) kda_sum_rows_kernel(SumRowsArgs a) {
    __shared__ float buf[32][33];
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.width) {
        const float *p = a.parts + c;
        int i = share;
        for (; i + 96 < a.rows; i += 128) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = p[(size_t)(i + 32 * k) * a.width];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += x[k];
        }
        for (; i < a.rows; i += 32) s[0] += p[(size_t)i * a.width];
    }
    buf[share][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    // column `share` of the block, its 32 sums over the lanes
    float t = buf[lane][share];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int col = blockIdx.x * 32 + share;
    if (lane != 0 || col >= a.width) return;
#pragma unroll
    for (int k = 0; k < SumRowsArgs::kOuts; ++k) {
        if (!a.out[k] || col < a.begin[k] || col >= a.begin[k + 1]) continue;
        // (the sums of a row are [cols][n], the output [n][cols])
        const int e = col - a.begin[k], cols = a.cols[k], n = (a.begin[k + 1] - a.begin[k]) / cols;
        a.out[k][cols == 1 ? (size_t)e : (size_t)(e % n) * cols + e / n] = t;
    }
}
}  // namespace

cudaError_t launch_sum_rows(const SumRowsArgs &a, cudaStream_t st) {
    kda_sum_rows_kernel<<<(a.width + 31) / 32, 1024, 0, st>>>(a);
    return cudaGetLastError();
}

namespace {

template <bool BF16, int V, int THREADS, int ITERS>
struct Shape {
    static constexpr int kRows = block_rows<THREADS>(), kBlock = block_size<THREADS>();
    // blocks of a walk over all rows: as many as run at once; a backward block
    // leaves a partial row, so fewer of the wide ones
    static long long blocks(const NormArgs &a, int sms, bool bwd) {
        const long long need = (a.rows + kRows - 1) / kRows;
        const long long most = (long long)sms * (bwd ? (kBlock > 256 ? 1 : 768 / kBlock) : (kBlock > 256 ? 1024 : 1536) / kBlock);
        return need < most ? need : most;
    }
    static cudaError_t fwd(const NormArgs &a, int sms, cudaStream_t st) {
        const unsigned grid = (unsigned)blocks(a, sms, false);
        if (a.layer) kda_norm_fwd_kernel<BF16, V, THREADS, ITERS, true><<<grid, kBlock, 0, st>>>(a);
        else kda_norm_fwd_kernel<BF16, V, THREADS, ITERS, false><<<grid, kBlock, 0, st>>>(a);
        return cudaGetLastError();
    }
    static cudaError_t bwd(const NormArgs &a, int sms, cudaStream_t st) {
        const unsigned grid = (unsigned)blocks(a, sms, true);
        const size_t smem = V * ITERS > 16 ? (size_t)2 * ITERS * V * THREADS * 4 : kRows > 1 ? (size_t)kRows * 2 * a.d * 4 : 0;
        auto kern = a.layer ? kda_norm_bwd_kernel<BF16, V, THREADS, ITERS, true> : kda_norm_bwd_kernel<BF16, V, THREADS, ITERS, false>;
        if (smem > 48 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        kern<<<grid, kBlock, smem, st>>>(a);
        return cudaGetLastError();
    }
    static long long run(int what, const NormArgs &a, int sms, cudaStream_t st) {
        if (what == 0) return blocks(a, sms, true);
        return (long long)(what == 1 ? fwd(a, sms, st) : bwd(a, sms, st));
    }
};

// what: 0 the backward's blocks, 1 forward, 2 backward.  The narrowest shape
// that holds a row: up to 16 channels a thread where a warp or less does.
template <bool BF16>
long long dispatch(int what, const NormArgs &a, int sms, cudaStream_t st) {
    constexpr int V = BF16 ? 8 : 4;
    const int d = a.d;
    if (a.wide) {
        if (d <= 8 * V) return Shape<BF16, V, 8, 1>::run(what, a, sms, st);
        if (d <= 16 * V) return Shape<BF16, V, 16, 1>::run(what, a, sms, st);
        if (d <= 32 * V) return Shape<BF16, V, 32, 1>::run(what, a, sms, st);
        if (d <= 64 * V) return Shape<BF16, V, 32, 2>::run(what, a, sms, st);
        if (d <= 128 * V) return Shape<BF16, V, 128, 1>::run(what, a, sms, st);
        if (d <= 256 * V) return Shape<BF16, V, 128, 2>::run(what, a, sms, st);
        if (d <= 512 * V) return Shape<BF16, V, 256, 2>::run(what, a, sms, st);
        if (d <= 1024 * V) return Shape<BF16, V, 512, 2>::run(what, a, sms, st);
        if (d <= 2048 * V) return Shape<BF16, V, 512, 4>::run(what, a, sms, st);
        if constexpr (!BF16) return Shape<BF16, V, 512, 8>::run(what, a, sms, st);
    }
    if (d <= 32) return Shape<BF16, 1, 32, 1>::run(what, a, sms, st);
    if (d <= 128) return Shape<BF16, 1, 32, 4>::run(what, a, sms, st);
    if (d <= 512) return Shape<BF16, 1, 32, 16>::run(what, a, sms, st);
    if (d <= 2048) return Shape<BF16, 1, 256, 8>::run(what, a, sms, st);
    if (d <= 8192) return Shape<BF16, 1, 512, 16>::run(what, a, sms, st);
    return Shape<BF16, 1, 512, 32>::run(what, a, sms, st);
}

}  // namespace

int norm_bwd_blocks(const NormArgs &a, bool bf16, int sms) {
    return (int)(bf16 ? dispatch<true>(0, a, sms, nullptr) : dispatch<false>(0, a, sms, nullptr));
}

cudaError_t launch_norm(const NormArgs &a, bool bf16, bool backward, int sms, cudaStream_t st) {
    return (cudaError_t)(bf16 ? dispatch<true>(backward ? 2 : 1, a, sms, st) : dispatch<false>(backward ? 2 : 1, a, sms, st));
}

}  // namespace kda
