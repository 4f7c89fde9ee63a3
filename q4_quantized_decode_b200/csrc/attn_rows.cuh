// Attention of new tokens over a paged cache, one warp for one query row.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m),
// over the tokens j that the row sees, in one pass with the running maximum m
// and sum (32 bits).  A token that the row does not see is not read at all,
// so nothing in it (infinities, NaN, uninitialised pages) can reach the row.
#pragma once

#include "mix_common.cuh"

namespace q4 {

struct AttnArgs {
    RaggedArgs batch;
    KvArgs kv;
    const void* q;
    void* out;
    int64_t q_stride, o_stride;     // elements between rows
    int q_heads, group;             // query heads, query heads of a key head
    float scale_log2;               // scale * log2(e): the softmax runs on powers of two
    int causal, window;             // window 0: none
    int cap;                        // tokens that a row of the page table can hold
    int* err;
};

// Tokens [lo, hi) that new token t of a sequence (n new of len) sees.  Tokens
// past the page table's columns are left out and reported.
__device__ __forceinline__ void seen_range(const AttnArgs& a, int len, int n, int t, int& lo, int& hi) {
    const int64_t p = (int64_t)len - n + t;
    int64_t h = a.causal ? p + 1 : len;
    if (h > a.cap) {
        set_device_error(a.err, kDevIndex);
        h = a.cap;
    }
    int64_t l = a.window > 0 ? p - a.window + 1 : 0;
    if (h < 0) h = 0;
    if (l < 0) l = 0;
    if (l > h) l = h;
    lo = (int)l;
    hi = (int)h;
}

__device__ __forceinline__ float warp_xor_max(float v, int from) {
    for (int o = from; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_xor_sum(float v, int from) {
    for (int o = from; o < 32; o <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One row by a whole warp.  Lanes in groups of 8, 16 or 32 hold a 16-byte
// chunk of the head each; every group takes its own tokens and the groups'
// softmax sums are joined at the end.
template <typename T>
__device__ void attend_row(const AttnArgs& a, int s, int64_t r, int h, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    const int chunks = a.kv.head_dim / 8;
    const int lg = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    const int c = lane & (lg - 1), grp = lane / lg, groups = 32 / lg;
    const bool on = c < chunks;
    float q[8], o[8];
    const T* qp = static_cast<const T*>(a.q) + r * a.q_stride + (int64_t)h * a.kv.head_dim + 8 * c;
    if (on) unpack8<T>(*reinterpret_cast<const uint4*>(qp), q);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int64_t ho = (int64_t)(h / a.group) * a.kv.head_stride + 8 * c;
    for (int j0 = lo; j0 < hi; j0 += groups) {
        const int j = j0 + grp;
        int64_t off = -1;
        if (j < hi) off = token_offset(a.kv, s, j, a.err);
        float d = 0.f;
        if (off >= 0 && on) {
            float k[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.kv.k) + off + ho), k);
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fmaf(q[i], k[i], d);
        }
        for (int x = 1; x < lg; x <<= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
        if (off < 0) continue;
        d *= a.scale_log2;
        const float mn = fmaxf(m, d);
        const float mu = mn == -INFINITY ? 0.f : mn;     // all scores -inf so far: weights 0
        const float w = exp2f(m - mu), p = exp2f(d - mu);
        m = mn;
        l = l * w + p;
        if (on) {
            float v[8];
            unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.kv.v) + off + ho), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = o[i] * w + p * v[i];
        }
    }
    __syncwarp();
    // Join the groups.  A NaN score keeps its way: fmaxf drops it, the sum does not.
    const float mj = warp_xor_max(m, lg);
    const float w = exp2f(m - (mj == -INFINITY ? 0.f : mj));
    l = warp_xor_sum(l * w, lg);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = warp_xor_sum(o[i] * w, lg) * inv;
    if (on && grp == 0)
        *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + r * a.o_stride + (int64_t)h * a.kv.head_dim + 8 * c) =
            pack8<T>(y);
}

}  // namespace q4
