// Shared pieces of the token-mixing kernels (cache append, paged attention,
// linear attention): 16-bit element types, the ragged batch of new tokens and
// the paged cache as the kernels see them.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_common.cuh"

namespace q4 {

template <typename T>
struct Elem;
template <>
struct Elem<__half> {
    static constexpr uint32_t kExpMask = 0x7C00u;   // all ones: infinity or NaN
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
    static __device__ __forceinline__ __half round(float f) { return __float2half_rn(f); }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr uint32_t kExpMask = 0x7F80u;
    static __device__ __forceinline__ float2 unpack(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ __nv_bfloat16 round(float f) { return __float2bfloat16_rn(f); }
};

// Eight elements of one 16-byte chunk.
template <typename T>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = Elem<T>::unpack(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(Elem<T>::pack(f[0], f[1]), Elem<T>::pack(f[2], f[3]), Elem<T>::pack(f[4], f[5]),
                      Elem<T>::pack(f[6], f[7]));
}

// Whether any of eight 16-bit values is an infinity or NaN.
template <typename T>
__device__ __forceinline__ bool any_nonfinite(uint4 v) {
    constexpr uint32_t e = Elem<T>::kExpMask;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & e) == e || (w[i] & (e << 16)) == (e << 16);
    return bad;
}

// The new tokens of a batch of sequences: sequence s holds the rows
// [start[s], start[s + 1]).  Entries come from device memory and are not
// trusted: rows outside [0, rows) belong to no sequence.
struct RaggedArgs {
    const int32_t* start;   // [n_seqs + 1]
    const int32_t* len;     // [n_seqs] tokens in the cache, the new ones included
    int64_t rows;
    int n_seqs;
};

// Rows [first, first + n) of sequence s, clipped to the batch.
__device__ __forceinline__ void seq_rows(const RaggedArgs& b, int s, int64_t& first, int& n) {
    int64_t lo = b.start[s], hi = b.start[s + 1];
    if (lo < 0) lo = 0;
    if (hi > b.rows) hi = b.rows;
    first = lo;
    n = hi > lo ? (int)(hi - lo) : 0;
}

// The sequence that holds row r, found by a whole warp (32 probes a step); -1
// if none does.  With non-decreasing starts it is the last s with start[s] <= r
// (the empty sequences before it share its start); other starts give some s,
// which the bounds check at the end accepts or not.
__device__ __forceinline__ int find_seq(const int32_t* start, int n_seqs, int64_t r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lane * step;
        const bool le = at < n && (int64_t)start[lo + at] <= r;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, le);
        const int c = m ? 31 - __clz((int)m) : 0;
        lo += c * step;
        n = min(step, n - c * step);
    }
    if ((int64_t)start[lo] <= r && r < (int64_t)start[lo + 1]) return lo;
    return -1;
}

__device__ __forceinline__ int64_t div_floor(int64_t a, int b) {      // a >= 0, b > 0
    return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// A paged cache: token t of sequence s is in page table[s * table_stride +
// t / page_size], at row t % page_size.  Strides in elements.
struct KvArgs {
    void* k;
    void* v;
    const int32_t* table;
    int64_t page_stride, token_stride, head_stride, table_stride;
    int n_pages, table_cols, page_size, n_heads, head_dim;
    int page_shift;         // log2(page_size) if that is a power of two, else -1
};

__device__ __forceinline__ void split_page(const KvArgs& c, int t, int& page, int& row) {
    if (c.page_shift >= 0) {
        page = t >> c.page_shift;
        row = t & (c.page_size - 1);
    } else {
        page = t / c.page_size;
        row = t - page * c.page_size;
    }
}

// Element offset of token t (>= 0) of sequence s, head 0; -1 (and the error
// word) for a page outside the table's columns or the pool.
__device__ __forceinline__ int64_t token_offset(const KvArgs& c, int s, int t, int* err) {
    int page, row;
    split_page(c, t, page, row);
    int phys = -1;
    if (page < c.table_cols) phys = c.table[(int64_t)s * c.table_stride + page];
    if ((unsigned)phys >= (unsigned)c.n_pages) {
        set_device_error(err, kDevIndex);
        return -1;
    }
    return (int64_t)phys * c.page_stride + (int64_t)row * c.token_stride;
}

}  // namespace q4
