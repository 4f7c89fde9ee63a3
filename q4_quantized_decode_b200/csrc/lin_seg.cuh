// Linear attention over prompts in parallel segments: where sequences and heads
// alone leave SMs idle, sequences are cut into equal segments; a first kernel
// takes what each segment adds to a state of zero, a second one runs through
// the segments of every head and leaves each its first state, the third
// computes all segments' outputs at once.
#pragma once

#include "linattn.cuh"

namespace q4 {

// The segments of a prompt: `segs` for every sequence, their states and decays.
struct LinSegArgs {
    LinArgs a;
    int segs, tokens;    // `tokens`: of a chunk, which segments are made of
    float* ws;           // [n_seqs][v_heads][segs][k_dim][v_dim], then [n_seqs][v_heads][segs] decays
};
__device__ __forceinline__ float* seg_state(const LinSegArgs& g, int s, int h, int i) {
    return g.ws + (((int64_t)s * g.a.v_heads + h) * g.segs + i) * g.a.k_dim * g.a.v_dim;
}
__device__ __forceinline__ float* seg_decay(const LinSegArgs& g, int s, int h, int i) {
    return g.ws + (int64_t)g.a.n_seqs * g.a.v_heads * g.segs * g.a.k_dim * g.a.v_dim +
           ((int64_t)s * g.a.v_heads + h) * g.segs + i;
}
// Tokens [t0, t1) of segment i of sequence s (whole chunks; later ones may be
// empty), and whether it is the last with tokens (or the first of none).
__device__ __forceinline__ void segment(const LinSegArgs& g, int s, int i, int64_t& t0, int64_t& t1, bool& last) {
    int64_t lo = g.a.start[s], hi = g.a.start[s + 1];
    if (lo < 0) lo = 0;
    if (hi > g.a.rows) hi = g.a.rows;
    if (hi < lo) hi = lo;
    const int64_t chunks = (hi - lo + g.tokens - 1) / g.tokens;
    const int64_t len = (chunks + g.segs - 1) / g.segs * g.tokens;
    t0 = lo + i * len < hi ? lo + i * len : hi;
    t1 = lo + (i + 1) * len < hi ? lo + (i + 1) * len : hi;
    last = t1 == hi && (t0 < t1 || i == 0);
}

__device__ __forceinline__ float exp2i(int e) {      // 2^e; 0 under and 2^127 over the range
    return e < -126 ? 0.f : __int_as_float((min(e, 127) + 127) << 23);
}
// The power that brings a magnitude x >= 0 to [2^14, 2^15), `cap` at most; 0
// for zero.
__device__ __forceinline__ int to_2_14(float x, int cap) {
    if (x == 0.f) return 0;
    return min(cap, 14 - ((__float_as_int(x) >> 23) - 127));
}

__device__ __forceinline__ uint32_t max_abs8(uint32_t m, uint4 v) {      // of 16-bit floats, in halves
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}

// The segments' first states: in each place of a segment's gain, the state
// that it starts from.
constexpr int kLinScanThreads = 128;
static __global__ void __launch_bounds__(kLinScanThreads) lin_scan_kernel(const LinSegArgs g) {
    pdl_wait();
    pdl_launch_dependents();
    const LinArgs& a = g.a;
    const int h = blockIdx.y, s = blockIdx.z;
    const int slot = a.slots ? a.slots[s] : s;
    if ((unsigned)slot >= (unsigned)a.n_slots) return;           // reported by the segments' kernel
    const int64_t e = ((int64_t)blockIdx.x * kLinScanThreads + threadIdx.x) * 4, size = (int64_t)a.k_dim * a.v_dim;
    if (e >= size) return;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.state_in) S = *reinterpret_cast<const float4*>(a.state_in + ((int64_t)slot * a.v_heads + h) * size + e);
    int n = g.segs;                                              // segments that have a gain
    for (int i = 0; i < g.segs; ++i) {
        int64_t t0, t1;
        bool last;
        segment(g, s, i, t0, t1, last);
        if (last) {
            n = i;
            break;
        }
    }
    float* p = seg_state(g, s, h, 0) + e;
    constexpr int kAhead = 4;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        float4 d[kAhead];
        float w[kAhead];
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
            if (i0 + y < n) {
                d[y] = *reinterpret_cast<const float4*>(p + (i0 + y) * size);
                w[y] = *seg_decay(g, s, h, i0 + y);
            }
#pragma unroll
        for (int y = 0; y < kAhead; ++y)
            if (i0 + y < n) {
                *reinterpret_cast<float4*>(p + (i0 + y) * size) = S;
                S.x = fmaf(S.x, w[y], d[y].x);
                S.y = fmaf(S.y, w[y], d[y].y);
                S.z = fmaf(S.z, w[y], d[y].z);
                S.w = fmaf(S.w, w[y], d[y].w);
            }
    }
    if (n < g.segs) *reinterpret_cast<float4*>(p + n * size) = S;
}

}  // namespace q4
