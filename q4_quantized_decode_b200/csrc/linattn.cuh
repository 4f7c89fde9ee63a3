// Linear attention with a decay for each head:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
// S a head's [k_dim][v_dim] state in 32 bits, g_t <= 0 the logarithm of the
// decay of the head at token t.
#pragma once

#include "mix_common.cuh"

namespace q4 {

struct LinArgs {
    const int32_t* start;        // [n_seqs + 1]
    const int32_t* slots;        // [n_seqs] the sequence's state, or null: its number
    const void* q;
    const void* k;
    const void* v;
    const float* g;              // [rows][v_heads], rows g_stride apart (0: fixed decays)
    const float* state_in;       // [n_slots][v_heads][k_dim][v_dim], or null: zeros
    float* state_out;            // may be state_in
    void* out;
    int64_t rows, q_stride, k_stride, v_stride, g_stride, o_stride;
    int n_seqs, n_slots, v_heads, each, k_dim, v_dim;   // each: value heads of a query and key head
    float scale;
    int* err;
};

// ---- token by token ---------------------------------------------------------
// A CTA keeps 32 columns of one head's state in registers and walks over the
// sequence's new tokens.  A single token is bound by the state's way in and
// out: each thread has all its rows' loads in flight at once, and a warp's
// load covers four rows of 128 contiguous bytes.  Measured (40 heads of 128 x
// 128): 96 sequences' tokens 82 us, 6.2 TB/s of states; one sequence's 3.0 us.
constexpr int kLinCols = 32;
constexpr int kLinThreads = 128;
constexpr int kLinRowGroups = kLinThreads / (kLinCols / 4);

template <typename T, int RPT>   // RPT: state rows of a thread, k_dim <= 16 * RPT
__global__ void __launch_bounds__(kLinThreads) lin_recur_kernel(const LinArgs a) {
    __shared__ float sq[16 * RPT], sk[16 * RPT];
    __shared__ float part[kLinThreads / 32][kLinCols];
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * kLinCols;
    const int slot = a.slots ? a.slots[s] : s;
    if ((unsigned)slot >= (unsigned)a.n_slots) {
        if (threadIdx.x == 0) set_device_error(a.err, kDevIndex);
        return;
    }
    int64_t t0 = a.start[s], t1 = a.start[s + 1];
    if (t0 < 0) t0 = 0;
    if (t1 > a.rows) t1 = a.rows;
    const int cl = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = c0 + 4 * cl;
    const bool con = col < a.v_dim;
    const int64_t so = ((int64_t)slot * a.v_heads + h) * a.k_dim * a.v_dim;
    float4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = i * kLinRowGroups + rg;
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a.state_in && con && row < a.k_dim)
            S[i] = *reinterpret_cast<const float4*>(a.state_in + so + (int64_t)row * a.v_dim + col);
    }
    const T* qb = static_cast<const T*>(a.q) + (int64_t)(h / a.each) * a.k_dim;
    const T* kb = static_cast<const T*>(a.k) + (int64_t)(h / a.each) * a.k_dim;
    for (int64_t t = t0; t < t1; ++t) {
        for (int i = threadIdx.x; i < 16 * RPT; i += kLinThreads) {
            sq[i] = i < a.k_dim ? Elem<T>::load(qb + t * a.q_stride + i) * a.scale : 0.f;
            sk[i] = i < a.k_dim ? Elem<T>::load(kb + t * a.k_stride + i) : 0.f;
        }
        const float decay = expf(a.g[t * a.g_stride + h]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (con) {
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const T*>(a.v) + t * a.v_stride +
                                                            (int64_t)h * a.v_dim + col);
            const float2 x = Elem<T>::unpack(w.x), y = Elem<T>::unpack(w.y);
            v = make_float4(x.x, x.y, y.x, y.y);
        }
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kk = sk[i * kLinRowGroups + rg], qq = sq[i * kLinRowGroups + rg];
            S[i].x = fmaf(S[i].x, decay, kk * v.x);
            S[i].y = fmaf(S[i].y, decay, kk * v.y);
            S[i].z = fmaf(S[i].z, decay, kk * v.z);
            S[i].w = fmaf(S[i].w, decay, kk * v.w);
            o.x = fmaf(qq, S[i].x, o.x);
            o.y = fmaf(qq, S[i].y, o.y);
            o.z = fmaf(qq, S[i].z, o.z);
            o.w = fmaf(qq, S[i].w, o.w);
        }
        // Sum over the row groups: four of a warp, then the warps in order.
#pragma unroll
        for (int x = 8; x < 32; x <<= 1) {
            o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, x);
            o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, x);
            o.z += __shfl_xor_sync(0xFFFFFFFFu, o.z, x);
            o.w += __shfl_xor_sync(0xFFFFFFFFu, o.w, x);
        }
        if (lane < 8) *reinterpret_cast<float4*>(&part[warp][4 * lane]) = o;
        __syncthreads();
        if (threadIdx.x < kLinCols / 2 && c0 + 2 * (int)threadIdx.x < a.v_dim) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < kLinThreads / 32; ++w) {
                x += part[w][2 * threadIdx.x];
                y += part[w][2 * threadIdx.x + 1];
            }
            *reinterpret_cast<uint32_t*>(static_cast<T*>(a.out) + t * a.o_stride + (int64_t)h * a.v_dim + c0 +
                                         2 * threadIdx.x) = Elem<T>::pack(x, y);
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int row = i * kLinRowGroups + rg;
        if (con && row < a.k_dim)
            *reinterpret_cast<float4*>(a.state_out + so + (int64_t)row * a.v_dim + col) = S[i];
    }
}

}  // namespace q4
