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

// the sum of x over the THREADS threads of a row; every one of them gets it.
// Rows of more than a warp: one row per block at a time, buf holds a sum per warp.
template <int THREADS>
__device__ __forceinline__ float row_sum(float x, float *buf) {
#pragma unroll
    for (int o = (THREADS < 32 ? THREADS : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if constexpr (THREADS > 32) {
        const int warp = threadIdx.x >> 5;
        __syncthreads();  // the previous sum has been read
        if ((threadIdx.x & 31) == 0) buf[warp] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) x += buf[i];
    }
    return x;
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

template <bool BF16, int V, int THREADS, int ITERS, bool LAYER>
__global__ void __launch_bounds__(block_size<THREADS>())
kda_norm_fwd_kernel(NormArgs a) {
    using E = Elem<BF16>;
    constexpr int ROWS = block_rows<THREADS>();
    __shared__ float buf[THREADS > 32 ? THREADS / 32 : 1];
    const int lane = threadIdx.x % THREADS, d = a.d;
    const float inv_d = 1.f / (float)d;
    const E *x = static_cast<const E *>(a.x);
    E *y = static_cast<E *>(a.y);
    float w[ITERS][V], b[ITERS][V];
#pragma unroll
    for (int i = 0; i < ITERS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (i * THREADS + lane) * V + j;
            w[i][j] = a.weight && c < d ? a.weight[c] : 1.f;
            b[i][j] = a.bias && c < d ? a.bias[c] : 0.f;
        }
    // every thread of a warp makes the same number of turns: the sums are warp-wide
    const long long step = (long long)gridDim.x * ROWS;
    for (long long base = (long long)blockIdx.x * ROWS; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / THREADS;
        const bool live = row < a.rows;
        Row<BF16, V, THREADS, ITERS> r;
        r.load(x + (live ? row : base) * a.x_stride, lane, d);
        float m = 0.f;
        if constexpr (LAYER) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < ITERS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s += r.raw[i].get(j);
            m = row_sum<THREADS>(s, buf) * inv_d;
        }
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const bool in = (i * THREADS + lane) * V < d;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float c = in ? r.raw[i].get(j) - m : 0.f;
                q = fmaf(c, c, q);
            }
        }
        q = row_sum<THREADS>(q, buf) * inv_d;
        const float rs = rsqrtf(q + a.eps);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c >= d) continue;
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = fmaf((r.raw[i].get(j) - m) * rs, w[i][j], b[i][j]);
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
    constexpr bool ACC = V * ITERS > 16;
    extern __shared__ float acc[];  // ACC: [2][ITERS * V][THREADS]; else [ROWS][2][d] when ROWS > 1
    __shared__ float buf[THREADS > 32 ? THREADS / 32 : 1];
    const int lane = threadIdx.x % THREADS, d = a.d;
    const float inv_d = 1.f / (float)d;
    const E *x = static_cast<const E *>(a.x), *dy = static_cast<const E *>(a.dy);
    E *dx = static_cast<E *>(a.dx);
    float w[ACC ? 1 : ITERS][V], dw[ACC ? 1 : ITERS][V], db[ACC ? 1 : ITERS][V];
    if constexpr (ACC) {
        for (int i = threadIdx.x; i < 2 * ITERS * V * THREADS; i += BLOCK) acc[i] = 0.f;
        __syncthreads();
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (i * THREADS + lane) * V + j;
                w[i][j] = a.weight && c < d ? a.weight[c] : 1.f;
                dw[i][j] = db[i][j] = 0.f;
            }
    }
    auto weight = [&](int i, int j) -> float {
        if constexpr (ACC) {
            const int c = (i * THREADS + lane) * V + j;
            return a.weight && c < d ? __ldg(a.weight + c) : 1.f;
        } else {
            return w[i][j];
        }
    };
    const long long step = (long long)gridDim.x * ROWS;
    for (long long base = (long long)blockIdx.x * ROWS; base < a.rows; base += step) {
        const long long row = base + threadIdx.x / THREADS;
        const bool live = row < a.rows;
        Row<BF16, V, THREADS, ITERS> r, g;
        r.load(x + (live ? row : base) * a.x_stride, lane, d);
        g.load(dy + (live ? row : base) * a.dy_stride, lane, d);
        float m = 0.f;
        if constexpr (LAYER) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < ITERS; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) s += r.raw[i].get(j);
            m = row_sum<THREADS>(s, buf) * inv_d;
        }
        // sums of (x - m)^2, u (x - m) and u
        float q = 0.f, ux = 0.f, us = 0.f;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const bool in = (i * THREADS + lane) * V < d;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float c = in ? r.raw[i].get(j) - m : 0.f, u = g.raw[i].get(j) * weight(i, j);
                q = fmaf(c, c, q);
                ux = fmaf(u, c, ux);
                us += u;
            }
        }
        q = row_sum<THREADS>(q, buf) * inv_d;
        ux = row_sum<THREADS>(ux, buf) * inv_d;
        us = LAYER ? row_sum<THREADS>(us, buf) * inv_d : 0.f;
        const float rs = rsqrtf(q + a.eps), k = ux * rs;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c >= d) continue;
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = (r.raw[i].get(j) - m) * rs, e = g.raw[i].get(j);
                o[j] = rs * (fmaf(e, weight(i, j), -us) - n * k);
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
        const long long most = (long long)sms * (bwd ? (kBlock > 256 ? 1 : 4) : 2048 / kBlock);
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
