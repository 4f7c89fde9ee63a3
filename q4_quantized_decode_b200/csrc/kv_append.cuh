// New keys and values into a paged cache, keys and queries rotated by their
// positions on the way.
//
// A pair (a, b) of a head turns by the angle pos * w: (a cos - b sin,
// b cos + a sin), with cos and sin times an amplitude.  The angle is taken in
// turns in 64 bits, pos * (w / 2 pi) less its nearest whole number, because
// 32 bits of a position of a million leave no digits behind the point; the
// remainder, at most half a turn, goes through sincospi in 32 bits.  Products
// are in 32 bits and every output is rounded once.
//
// It moves each byte of q, k and v once in and once out and is bound by that.
// A thread keeps one place within the head (a pair of 16-byte chunks in the
// half layout, one chunk in the interleaved one), takes its eight angles once
// and walks over the heads with them, so nothing goes through shared memory;
// 64 threads a row keep 32 rows in flight on an SM.  Measured (40 query, 8 key
// heads of 128, f16): six prompts of up to 2048 tokens, 39 us, 5.2 TB/s; one
// token 3.0 us, 48 tokens far out (heads of 256, 64 of it rotated) 5.5.
#pragma once

#include "mix_common.cuh"

namespace q4 {

constexpr int kAppendThreads = 64;

enum : int { kRopeHalf = 0, kRopeInterleaved = 1, kRopeHalfScalar = 2 };

struct AppendArgs {
    RaggedArgs batch;
    KvArgs kv;
    const int32_t* pos;      // rotation positions of the rows, or null: the place in the cache
    const double* freqs;     // [rot / 2] radians per position
    const void* q;           // null: no queries
    const void* k;
    const void* v;
    void* q_out;
    int64_t q_stride, k_stride, v_stride, qo_stride;   // elements between rows
    int q_heads, rot;
    float amp;
    int* err;
};

__device__ __forceinline__ void rope_angle(double turns_per_pos, int pos, float amp, float& c, float& s) {
    const double t = (double)pos * turns_per_pos;
    const float f = (float)(t - rint(t));
    sincospif(2.f * f, &s, &c);
    c *= amp;
    s *= amp;
}

constexpr double kInvTwoPi = 0.15915494309189533577;

template <typename T, int MODE>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t r = blockIdx.x;
    const int D = a.kv.head_dim, rot = a.rot;
    const int s = find_seq(a.batch.start, a.batch.n_seqs, r);
    if (s < 0) return;
    // Place in the cache: the row's index among its sequence's new tokens,
    // counted back from the sequence's length.
    const int64_t place = (int64_t)a.batch.len[s] - ((int64_t)a.batch.start[s + 1] - r);
    const int pos = a.pos ? a.pos[r] : (int)place;
    int64_t slot = -1;
    if (place >= 0 && place < (int64_t)INT32_MAX)
        slot = token_offset(a.kv, s, (int)place, a.err);
    else
        set_device_error(a.err, kDevIndex);

    const T* q = static_cast<const T*>(a.q) + (a.q ? r * a.q_stride : 0);
    const T* k = static_cast<const T*>(a.k) + r * a.k_stride;
    const T* v = static_cast<const T*>(a.v) + r * a.v_stride;
    T* qo = static_cast<T*>(a.q_out) + (a.q ? r * a.qo_stride : 0);
    T* kc = static_cast<T*>(a.kv.k) + (slot < 0 ? 0 : slot);
    T* vc = static_cast<T*>(a.kv.v) + (slot < 0 ? 0 : slot);
    const int hq = a.q ? a.q_heads : 0;
    const int h_end = slot < 0 ? hq : hq + a.kv.n_heads;   // heads to rotate

    // Items of a head: np rotated ones, then nt that pass.
    int np, nt;
    if (MODE == kRopeHalf) {
        np = rot / 16;
        nt = (D - rot) / 8;
    } else if (MODE == kRopeInterleaved) {
        np = (rot + 7) / 8;
        nt = D / 8 - np;
    } else {
        np = rot / 2;
        nt = D - rot;
    }
    const int items = np + nt;
    const int width = items < kAppendThreads ? items : kAppendThreads;
    const int subs = kAppendThreads / width;
    const int sub = threadIdx.x / width;
    const int h0 = blockIdx.y * subs + sub, dh = gridDim.y * subs;
    if (sub < subs) {
        for (int it = threadIdx.x - sub * width; it < items; it += width) {
            if (MODE == kRopeHalfScalar) {
                if (it < np) {
                    float c, sn;
                    rope_angle(a.freqs[it] * kInvTwoPi, pos, a.amp, c, sn);
                    for (int h = h0; h < h_end; h += dh) {
                        const T* src = h < hq ? q + (int64_t)h * D : k + (int64_t)(h - hq) * D;
                        T* dst = h < hq ? qo + (int64_t)h * D : kc + (int64_t)(h - hq) * a.kv.head_stride;
                        const float x = Elem<T>::load(src + it), y = Elem<T>::load(src + it + np);
                        dst[it] = Elem<T>::round(x * c - y * sn);
                        dst[it + np] = Elem<T>::round(y * c + x * sn);
                    }
                } else {
                    const int e = rot + it - np;
                    for (int h = h0; h < h_end; h += dh) {
                        const T* src = h < hq ? q + (int64_t)h * D : k + (int64_t)(h - hq) * D;
                        T* dst = h < hq ? qo + (int64_t)h * D : kc + (int64_t)(h - hq) * a.kv.head_stride;
                        dst[e] = src[e];
                    }
                }
                continue;
            }
            if (it >= np) {
                const int e = (MODE == kRopeHalf ? rot : 8 * np) + 8 * (it - np);
                for (int h = h0; h < h_end; h += dh) {
                    const T* src = h < hq ? q + (int64_t)h * D : k + (int64_t)(h - hq) * D;
                    T* dst = h < hq ? qo + (int64_t)h * D : kc + (int64_t)(h - hq) * a.kv.head_stride;
                    *reinterpret_cast<uint4*>(dst + e) = *reinterpret_cast<const uint4*>(src + e);
                }
                continue;
            }
            constexpr int F = MODE == kRopeHalf ? 8 : 4;       // angles of an item
            float c[F], sn[F];
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int f = F * it + i;
                c[i] = 1.f;
                sn[i] = 0.f;
                if (MODE == kRopeHalf || 2 * f < rot) rope_angle(a.freqs[f] * kInvTwoPi, pos, a.amp, c[i], sn[i]);
            }
            for (int h = h0; h < h_end; h += dh) {
                const T* src = h < hq ? q + (int64_t)h * D : k + (int64_t)(h - hq) * D;
                T* dst = h < hq ? qo + (int64_t)h * D : kc + (int64_t)(h - hq) * a.kv.head_stride;
                float x[8];
                unpack8<T>(*reinterpret_cast<const uint4*>(src + 8 * it), x);
                if (MODE == kRopeHalf) {
                    float y[8], u[8], w[8];
                    unpack8<T>(*reinterpret_cast<const uint4*>(src + 8 * it + rot / 2), y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        u[i] = x[i] * c[i % F] - y[i] * sn[i % F];
                        w[i] = y[i] * c[i % F] + x[i] * sn[i % F];
                    }
                    *reinterpret_cast<uint4*>(dst + 8 * it) = pack8<T>(u);
                    *reinterpret_cast<uint4*>(dst + 8 * it + rot / 2) = pack8<T>(w);
                } else {
                    float u[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // pairs past the rotated part keep their values, whatever they are
                        const bool turn = 8 * it + 2 * i < rot;
                        u[2 * i] = turn ? x[2 * i] * c[i % F] - x[2 * i + 1] * sn[i % F] : x[2 * i];
                        u[2 * i + 1] = turn ? x[2 * i + 1] * c[i % F] + x[2 * i] * sn[i % F] : x[2 * i + 1];
                    }
                    *reinterpret_cast<uint4*>(dst + 8 * it) = pack8<T>(u);
                }
            }
        }
    }
    if (slot < 0) return;
    const int vh = D / 8;                                       // chunks of a value head
    for (int i = blockIdx.y * kAppendThreads + threadIdx.x; i < a.kv.n_heads * vh; i += gridDim.y * kAppendThreads) {
        const int h = i / vh, e = 8 * (i - h * vh);
        *reinterpret_cast<uint4*>(vc + (int64_t)h * a.kv.head_stride + e) =
            *reinterpret_cast<const uint4*>(v + (int64_t)h * D + e);
    }
}

}  // namespace q4
