// cache4_merge.cu -- joins the shares of the attention kernels over the 4-bit pages.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache4_sched.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

using namespace cache4;

// The shares of a row tile's keys, in key order: o = sum_p 2^{m_p - M} O_p / sum_p 2^{m_p - M} l_p.
// A share is (m [ROWS], l [ROWS], O [ROWS][D]); worker w has two places, 1 for
// a row tile that starts in its range and 0 for one that it goes on with.
//
// A CTA joins one row of the row tiles that start in 16 workers' ranges (and
// end in later ones).  Up to 16 shares are one warp's work, different warps
// taking different row tiles; more are dealt out to the CTA's eight warps in
// contiguous runs, whose sums are added in that order.  What it costs is the
// chain of dependent loads (one thread walking 200 shares took 50 us) and the
// number of CTAs (one per worker and row, most with nothing to do, 15 us).
// The launch is a programmatic dependent of the attention kernel: its CTAs
// take their places as that kernel's leave.  Where a call ran both attention
// kernels, one launch joins the shares of both: 293 us instead of 302 with two
// (64 requests of 1 to 8 queries).  Four or eight rows per warp instead of one
// gained nothing (425 and 420 instead of 424 us for prompt chunks, whose
// shares are 40 MB, 18 us; 303 and 307 instead of 302 for the other).
constexpr int kMergeWorkers = 16;

template <int D>
struct Sum {
    static constexpr int C = D / 32;  // channels per lane
    float l, y[C];
    __device__ __forceinline__ void clear() {
        l = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) y[c] = 0.f;
    }
    __device__ __forceinline__ void add(float f, const float *share, int rows, int row, int lane) {
        l = fmaf(f, share[rows + row], l);
        const float *o = share + 2 * rows + (size_t)row * D + lane * C;
#pragma unroll
        for (int c = 0; c < C; c += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(o + c);
            y[c] = fmaf(f, v.x, y[c]);
            y[c + 1] = fmaf(f, v.y, y[c + 1]);
        }
    }
};

// one row of the row tiles that start in the ranges of workers w_first .. w_first + kMergeWorkers - 1
template <int D, int ROWS, typename KIND, bool F32>
__device__ __forceinline__ void join(const Cache4AttnArgs &a, int workers, int w_first, int row, float (&s_l)[8],
                                     float (&s_y)[8][D]) {
    constexpr int C = D / 32, W = kMergeWorkers;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.Hq / a.Hkv;
    const size_t step = (size_t)ROWS * (D + 2);
    int4 mine = make_int4(-1, 0, 0, 0);
    if (lane < W && w_first + lane < workers) mine = a.jobs[w_first + lane];
    uint32_t left = __ballot_sync(0xffffffffu, mine.x >= 0);
    for (int k = 0; left; ++k) {
        const int i = __ffs(left) - 1, w0 = w_first + i;
        left &= left - 1;
        const int4 job = make_int4(__shfl_sync(0xffffffffu, mine.x, i), __shfl_sync(0xffffffffu, mine.y, i),
                                   __shfl_sync(0xffffffffu, mine.z, i), __shfl_sync(0xffffffffu, mine.w, i));
        const int n = job.w - w0 + 1;
        const bool wide = n > 16;
        if (!wide && k % 8 != warp) continue;
        const Req q = request<ROWS, KIND::TILE, KIND::LEAD>(a, job.x, G);
        const int rr = job.z * ROWS + row;
        if (rr >= q.rows) continue;  // the same in every warp
        const float *first = a.parts + ((size_t)w0 * 2 + 1) * step, *later = a.parts + (size_t)w0 * 2 * step;
        auto share = [&](int j) { return j == 0 ? first : later + (size_t)j * 2 * step; };
        float m = -INFINITY;
        for (int j = lane; j < n; j += 32) m = fmaxf(m, share(j)[row]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -INFINITY ? 0.f : m;
        const int per = wide ? (n + 7) / 8 : n, lo = wide ? min(n, warp * per) : 0, hi = min(n, lo + per);
        Sum<D> sum;
        sum.clear();
#pragma unroll 8
        for (int j = lo; j < hi; ++j) sum.add(exp2_fast(share(j)[row] - ref), share(j), ROWS, row, lane);
        if (wide) {
            __syncthreads();  // the last row tile's sums have been read
            if (lane == 0) s_l[warp] = sum.l;
#pragma unroll
            for (int c = 0; c < C; ++c) s_y[warp][lane * C + c] = sum.y[c];
            __syncthreads();
            if (warp) continue;
            for (int w = 1; w < 8; ++w) {
                sum.l += s_l[w];
#pragma unroll
                for (int c = 0; c < C; ++c) sum.y[c] += s_y[w][lane * C + c];
            }
        }
        const size_t head = (size_t)(q.q0 + rr / G) * a.Hq + job.y * G + rr % G;
        const bool none = q.len - q.n + rr / G < 0;  // sees no key (scores of -inf alone are 0 / 0)
        const float inv = none ? 0.f : (a.v_scale ? a.v_scale[job.y] : 1.f) / sum.l;
#pragma unroll
        for (int c = 0; c < C; c += 2) {
            const float2 v = none ? make_float2(0.f, 0.f) : make_float2(sum.y[c] * inv, sum.y[c + 1] * inv);
            const size_t e = head * D + lane * C + c;
            if constexpr (F32) *reinterpret_cast<float2 *>(static_cast<float *>(a.o) + e) = v;
            else
                *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.o) + e) = __floats2bfloat162_rn(v.x, v.y);
        }
        if (a.lse && lane == 0) a.lse[head] = none ? -INFINITY : (m + log2f(sum.l) - KIND::LIFT) * kLn2;
    }
}

// FEW, MANY: rows per tile of the two kernels, 0 for one that the call did not run
template <int D, int FEW, int MANY, bool F32>
__global__ void __launch_bounds__(256)
kda_cache4_merge_kernel(const Cache4AttnArgs few, const Cache4AttnArgs many, int few_workers, int many_workers) {
    __shared__ float s_l[8], s_y[8][D];
    wait_for_primary();
    int block = blockIdx.x;
    if constexpr (FEW > 0) {
        const int groups = (few_workers + kMergeWorkers - 1) / kMergeWorkers;
        if (block < groups * FEW)
            return join<D, FEW, FewRows, F32>(few, few_workers, block % groups * kMergeWorkers, block / groups, s_l, s_y);
        block -= groups * FEW;
    }
    if constexpr (MANY > 0) {
        const int groups = (many_workers + kMergeWorkers - 1) / kMergeWorkers;
        join<D, MANY, ManyRows, F32>(many, many_workers, block % groups * kMergeWorkers, block / groups, s_l, s_y);
    }
}

template <int D, int FEW, int MANY, bool F32>
cudaError_t launch(const Cache4AttnArgs &few, const Cache4AttnArgs &many, int sms, cudaStream_t st) {
    const int few_workers = cache4_attn_workers(sms), many_workers = sms;
    auto groups = [](int workers) { return (unsigned)((workers + kMergeWorkers - 1) / kMergeWorkers); };
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(groups(few_workers) * FEW + groups(many_workers) * MANY);
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_cache4_merge_kernel<D, FEW, MANY, F32>, few, many, few_workers, many_workers);
}

template <int D>
cudaError_t launch_d(const Cache4AttnArgs &few, const Cache4AttnArgs &many, bool bf16, int few_rows, int many_rows, int sms,
                     cudaStream_t st) {
    if (!bf16) return launch<D, 8, 0, true>(few, many, sms, st);
    if (many_rows == 0)
        return few_rows == 8 ? launch<D, 8, 0, false>(few, many, sms, st) : launch<D, 16, 0, false>(few, many, sms, st);
    if (few_rows == 0)
        return many_rows == 128 ? launch<D, 0, 128, false>(few, many, sms, st) : launch<D, 0, 256, false>(few, many, sms, st);
    if (few_rows == 8)
        return many_rows == 128 ? launch<D, 8, 128, false>(few, many, sms, st) : launch<D, 8, 256, false>(few, many, sms, st);
    return many_rows == 128 ? launch<D, 16, 128, false>(few, many, sms, st) : launch<D, 16, 256, false>(few, many, sms, st);
}

}  // namespace

cudaError_t launch_cache4_merge(const Cache4AttnArgs &few, const Cache4AttnArgs &many, int d, bool bf16, int few_rows,
                                int many_rows, int sms, cudaStream_t st) {
    return d == 128 ? launch_d<128>(few, many, bf16, few_rows, many_rows, sms, st)
                    : launch_d<64>(few, many, bf16, few_rows, many_rows, sms, st);
}

}  // namespace kda
