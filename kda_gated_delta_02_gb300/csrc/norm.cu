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
// holds four; 512 for the widest) and a block walks several rows, the next one
// asked for while one is worked on, each thread always at the same channels:
// few weights stay in its registers, and so do the sums of the weights'
// gradients over its rows.  Those leave as one partial row per block and are
// added up in a fixed order by a second kernel: the same inputs give the same
// bits.  786432 rows of 128, bf16: forward 67 us (6.0 TB/s), backward 107 (5.6) and 8
// for the sums; 4099 rows of 5120, f32: 31 us (5.5), 48 (5.3) and 9.  (Without the row
// ahead and with two barriers a sum the latter two took 54 and 73.)  A wide row's
// backward is one block of 512 threads of 128 registers an SM, so that nothing covers a
// row's barriers: 16384 channels of f32 200 us (4.0 TB/s), of 4099 rows.
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
    static constexpr int P = (V + 1) / 2;  // pairs of channels
    float2 held[HELD ? ITERS : 1][P];
    __device__ __forceinline__ Channels(const float *p, float none, int lane, int d) : p(p), none(none), lane(lane), d(d) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < ITERS; ++i) fetch(i, held[i]);
        }
    }
    __device__ __forceinline__ void fetch(int i, float2 (&x)[P]) const {
        const int c = (i * THREADS + lane) * V;
        if (!p || c >= d) {
#pragma unroll
            for (int j = 0; j < P; ++j) x[j] = both(none);
        } else if constexpr (V >= 4) {
#pragma unroll
            for (int j = 0; j < P; j += 2) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(p + c + 2 * j));
                x[j] = make_float2(q.x, q.y), x[j + 1] = make_float2(q.z, q.w);
            }
        } else {
            x[0] = make_float2(__ldg(p + c), none);
        }
    }
    __device__ __forceinline__ void get(int i, float2 (&x)[P]) const {
        if constexpr (HELD) {
#pragma unroll
            for (int j = 0; j < P; ++j) x[j] = held[i][j];
        } else {
            fetch(i, x);
        }
    }
};

// rows asked for ahead: one, where two fit into the registers
template <int V, int ITERS>
__host__ __device__ constexpr bool ahead() { return V > 1 ? V * ITERS <= 16 : ITERS <= 4; }  // (single channels fill half a pair)

template <bool BF16, int V, int THREADS, int ITERS, bool LAYER>
__global__ void __launch_bounds__(block_size<THREADS>())
kda_norm_fwd_kernel(NormArgs a) {
    using E = Elem<BF16>;
    constexpr int ROWS = block_rows<THREADS>(), P = (V + 1) / 2;
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
        float2 t = both(0.f);
        if constexpr (LAYER) {
#pragma unroll
            for (int i = 0; i < ITERS; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) t = __fadd2_rn(t, r.raw[i].pair(j));
            s[0] = t.x + t.y;
            row_sums<THREADS>(s, buf, turn);
            m = s[0] * inv_d;
        }
        t = both(0.f);
        const float2 mm = both(-m);
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            if (LAYER && (i * THREADS + lane) * V >= d) continue;  // (zeros, but for the mean)
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 c = LAYER ? __fadd2_rn(r.raw[i].pair(j), mm) : r.raw[i].pair(j);
                t = __ffma2_rn(c, c, t);
            }
        }
        s[0] = V > 1 ? t.x + t.y : t.x;
        row_sums<THREADS>(s, buf, turn);
        const float2 rs = both(rsqrtf(s[0] * inv_d + a.eps));
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c >= d) continue;
            float2 w[P], b[P];
            weight.get(i, w);
            bias.get(i, b);
            Vec<BF16, V> out;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 x = LAYER ? __fadd2_rn(r.raw[i].pair(j), mm) : r.raw[i].pair(j);
                out.set_pair(j, __ffma2_rn(__fmul2_rn(x, rs), w[j], b[j]));
            }
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
    constexpr int ROWS = block_rows<THREADS>(), BLOCK = block_size<THREADS>(), P = (V + 1) / 2;
    constexpr bool ACC = V * ITERS > 16, AHEAD = ahead<V, ITERS>();
    extern __shared__ __align__(16) float acc[];  // ACC: [2][ITERS * P][THREADS] pairs (or single ones); else [ROWS][2][d] when ROWS > 1
    __shared__ __align__(16) float buf1[2][1][THREADS > 32 ? THREADS / 32 : 4], buf3[2][LAYER ? 3 : 2][THREADS > 32 ? THREADS / 32 : 4];
    int turn1 = 0, turn3 = 0;
    const int lane = threadIdx.x % THREADS, d = a.d;
    const float inv_d = 1.f / (float)d;
    const E *x = static_cast<const E *>(a.x), *dy = static_cast<const E *>(a.dy);
    E *dx = static_cast<E *>(a.dx);
    const Channels<V, THREADS, ITERS> weight(a.weight, 1.f, lane, d);
    float2 dw[ACC ? 1 : ITERS][P], db[ACC ? 1 : ITERS][P];
    if constexpr (ACC) {
        for (int i = threadIdx.x; i < 2 * ITERS * V * THREADS; i += BLOCK) acc[i] = 0.f;
        __syncthreads();
    } else {
#pragma unroll
        for (int i = 0; i < ITERS; ++i)
#pragma unroll
            for (int j = 0; j < P; ++j) dw[i][j] = db[i][j] = both(0.f);
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
            float2 t = both(0.f);
#pragma unroll
            for (int i = 0; i < ITERS; ++i)
#pragma unroll
                for (int j = 0; j < P; ++j) t = __fadd2_rn(t, r.raw[i].pair(j));
            float s[1] = {t.x + t.y};
            row_sums<THREADS>(s, buf1, turn1);
            m = s[0] * inv_d;
        }
        const float2 mm = both(-m);
        float2 t[3] = {both(0.f), both(0.f), both(0.f)};  // sums of (x - m)^2, u (x - m) and u
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            if ((i * THREADS + lane) * V >= d) continue;
            float2 w[P];
            weight.get(i, w);
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 c = LAYER ? __fadd2_rn(r.raw[i].pair(j), mm) : r.raw[i].pair(j), e = g.raw[i].pair(j);
                const float2 u = make_float2(__fmul_rn(e.x, w[j].x), __fmul_rn(e.y, w[j].y));
                t[0] = __ffma2_rn(c, c, t[0]);
                t[1] = __ffma2_rn(u, c, t[1]);
                if (LAYER) t[2] = __fadd2_rn(t[2], u);
            }
        }
        float s[LAYER ? 3 : 2];
#pragma unroll
        for (int k = 0; k < (LAYER ? 3 : 2); ++k) s[k] = V > 1 ? t[k].x + t[k].y : t[k].x;
        row_sums<THREADS>(s, buf3, turn3);
        // dx = rs (u - n k - us) = rs u - (x - m) rs^2 k - rs us
        const float r1 = rsqrtf(s[0] * inv_d + a.eps), k1 = s[1] * inv_d * r1;
        const float2 rs = both(r1), kk = both(-k1), us = both(LAYER ? -s[LAYER ? 2 : 0] * inv_d : 0.f);
        if (row >= a.rows) continue;
#pragma unroll
        for (int i = 0; i < ITERS; ++i) {
            const int c = (i * THREADS + lane) * V;
            if (c >= d) continue;
            float2 w[P];
            weight.get(i, w);
            Vec<BF16, V> out;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const float2 x = LAYER ? __fadd2_rn(r.raw[i].pair(j), mm) : r.raw[i].pair(j), n = __fmul2_rn(x, rs), e = g.raw[i].pair(j);
                // (u rounded as it was when it was added up, so that a single channel's mean takes all of it away;
                // the packed product and sum would be contracted)
                const float2 u = make_float2(__fmul_rn(e.x, w[j].x), __fmul_rn(e.y, w[j].y));
                const float2 v = LAYER ? make_float2(__fadd_rn(u.x, us.x), __fadd_rn(u.y, us.y)) : u;
                out.set_pair(j, __fmul2_rn(rs, __ffma2_rn(n, kk, v)));
                if constexpr (ACC && V == 1) {
                    float *p = acc + i * THREADS + lane;
                    p[0] = fmaf(e.x, n.x, p[0]);
                    p[ITERS * THREADS] += e.x;
                } else if constexpr (ACC) {
                    float2 *p = reinterpret_cast<float2 *>(acc) + (i * P + j) * THREADS + lane;
                    p[0] = __ffma2_rn(e, n, p[0]);
                    p[ITERS * P * THREADS] = __fadd2_rn(p[ITERS * P * THREADS], e);
                } else {
                    dw[i][j] = __ffma2_rn(e, n, dw[i][j]);
                    db[i][j] = __fadd2_rn(db[i][j], e);
                }
            }
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
            for (int j = 0; j < P; ++j) {
                const int c = (i * THREADS + lane) * V + 2 * j;
                if (c < d) mine[c] = dw[i][j].x, mine[d + c] = db[i][j].x;
                if (V > 1 && c + 1 < d) mine[c + 1] = dw[i][j].y, mine[d + c + 1] = db[i][j].y;
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
            for (int j = 0; j < P; ++j) {
                const int c = (i * THREADS + lane) * V + 2 * j;
                if (c >= d) continue;
                float2 sw, sb;
                if constexpr (ACC && V == 1) {
                    sw.x = acc[i * THREADS + lane], sb.x = acc[(ITERS + i) * THREADS + lane];
                } else if constexpr (ACC) {
                    const float2 *p = reinterpret_cast<const float2 *>(acc) + (i * P + j) * THREADS + lane;
                    sw = p[0], sb = p[ITERS * P * THREADS];
                } else {
                    sw = dw[i][j], sb = db[i][j];
                }
                out[c] = sw.x, out[d + c] = sb.x;
                if (V > 1) out[c + 1] = sw.y, out[d + c + 1] = sb.y;
            }
    }
}

}  // namespace

// Sums of partial rows, in the order of a fixed tree: 32 columns and SHARES
// shares of the rows per block, 8 of them where columns are many, else 32.  128
// rows of 40960 columns: 10.1 us (16.2 with 32 shares); 608 of 256: 8, a launch and a
// chain of five loads.
namespace {
template <int SHARES>
__global__ void __launch_bounds__(32 * SHARES) kda_sum_rows_kernel(SumRowsArgs a) {
    __shared__ float buf[SHARES][32];
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.width) {
        const float *p = a.parts + (size_t)share * a.width + c;
        const size_t step = (size_t)SHARES * a.width;
        long long i = share;
        for (; i + 3 * SHARES < a.rows; i += 4 * SHARES, p += 4 * step) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = p[k * step];
#pragma unroll
            for (int k = 0; k < 4; ++k) s[k] += x[k];
        }
        for (; i < a.rows; i += SHARES, p += step) s[0] += *p;
    }
    buf[share][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (share > 0 || c >= a.width) return;
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < SHARES; ++k) t[k & 3] += buf[k][lane];
    const float sum = (t[0] + t[1]) + (t[2] + t[3]);
#pragma unroll
    for (int k = 0; k < SumRowsArgs::kOuts; ++k) {
        if (!a.out[k] || c < a.begin[k] || c >= a.begin[k + 1]) continue;
        // (the sums of a row are [cols][n], the output [n][cols])
        const int e = c - a.begin[k], cols = a.cols[k];
        if (cols == 1) {
            a.out[k][e] = sum;
        } else {
            const int n = (a.begin[k + 1] - a.begin[k]) / cols;
            a.out[k][(size_t)(e % n) * cols + e / n] = sum;
        }
    }
}
}  // namespace

cudaError_t launch_sum_rows(const SumRowsArgs &a, int sms, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.width + 31) / 32);
    if (grid >= 4u * sms) kda_sum_rows_kernel<8><<<grid, 256, 0, st>>>(a);
    else kda_sum_rows_kernel<32><<<grid, 1024, 0, st>>>(a);
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
        // (three turns of four f32 channels: up to 1 % less than four with the last ones idle, over all of 4,100 to 6,144
        // channels; 4099 rows of 5632, layer norm, 58.2 us back rather than 59.0)
        if constexpr (!BF16)
            if (d <= 1536 * V) return Shape<BF16, V, 512, 3>::run(what, a, sms, st);
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
