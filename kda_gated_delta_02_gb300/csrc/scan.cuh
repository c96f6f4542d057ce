// scan.cuh -- what the kernels of the selective scan share (scan.cu,
// scan_bwd.cu): segments of packed sequences and the places of saved states.
#pragma once

#include "kda_internal.h"
#include "layer.cuh"

namespace kda {
namespace scan {

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSaveEvery = kScanSaveEvery;

// A in powers of two.  A rate of -infinity is held finite, so that a step of 0
// (past a sequence's end) leaves a state as it is.
__device__ __forceinline__ float rate(float A) {
    const float r = A * kLog2e;
    return r < -3.0e38f ? -3.0e38f : r;
}

// Segment j of sequence s (tokens [a, b), cut every `seg` tokens; 0: not cut)
// is unit floor(a / seg) + s + j: distinct, in order, below floor(T / seg) + N.
struct Segment {
    int s = -1, t0 = 0, t1 = 0;  // s < 0: no tokens here
    bool first = false, last = false;
    long long slot = 0;  // of the saved state at t0
};

__device__ __forceinline__ Segment segment_of(const int32_t *cu, int N, int T, int seg, int u) {
    Segment g;
    const int s = seg ? layer::first_past(N, [&](int k) { return (long long)cu[k + 1] / seg + k + 1 > u; }) : u;
    if (s >= N) return g;
    const int a = cu[s], b = cu[s + 1];
    if (a < 0 || b < a || b > T) return g;
    const long long j = seg ? u - ((long long)a / seg + s) : 0, at = a + j * (long long)seg;
    if (j < 0 || (j > 0 && at >= b)) return g;
    g.s = s;
    g.t0 = (int)at;
    g.t1 = seg && b - at > seg ? (int)(at + seg) : b;
    g.first = j == 0;
    g.last = g.t1 == b;
    g.slot = (long long)a / kSaveEvery + s + (at - a) / kSaveEvery;
    return g;
}

// The check of sequence u's ends; there are at least as many units as sequences.
__device__ __forceinline__ void check_sequence(const ScanArgs &a, int u) {
    if (u >= a.N) return;
    const int b0 = a.cu_seqlens[u], b1 = a.cu_seqlens[u + 1];
    if (b0 < 0 || b1 < b0 || b1 > a.T) report_status(a.status, KDA_STATUS_BAD_SEQLENS);
}

}  // namespace scan
}  // namespace kda
