// Host side of the token-mixing calls of the q4gemv C ABI (see
// include/q4gemv.h): argument validation, kernel selection and launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "../../include/q4gemv.h"
#include "attn_split.cuh"
#include "attn_tc.cuh"
#include "ctx_view.h"
#include "kv_append.cuh"
#include "lin_chunk.cuh"
#include "lin_tc.cuh"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The handle's device for the duration of a call; the caller's is put back.
struct DeviceScope {
    int before = -1;
    bool ok = false;
    explicit DeviceScope(int device) {
        if (cudaGetDevice(&before) != cudaSuccess) return;
        ok = before == device || cudaSetDevice(device) == cudaSuccess;
        if (before == device) before = -1;
    }
    ~DeviceScope() {
        if (before >= 0) cudaSetDevice(before);
    }
};

int bad(q4gemv_t h, int status, const char* call, const char* what) {
    char buf[256];
    snprintf(buf, sizeof buf, "%s: %s", call, what);
    return q4::ctx_fail(h, status, buf);
}

int launch_status(q4gemv_t h, cudaError_t e, const char* call) {
    return e == cudaSuccess ? Q4_OK : bad(h, Q4_ECUDA, call, cudaGetErrorString(e));
}

// A launch whose start may overlap the end of the kernel before it: every
// kernel here waits for that one before it touches memory.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool head_dim_ok(int64_t d) { return d >= 8 && d <= Q4GEMV_MAX_HEAD_DIM && d % 8 == 0; }

// Rows of `heads` heads of `dim`, `stride` elements apart.
bool row_stride_ok(int64_t stride, int64_t heads, int64_t dim) {
    return stride % 8 == 0 && stride >= heads * dim && stride <= (int64_t(1) << 40);
}

int check_batch(q4gemv_t h, const char* call, int64_t rows, int64_t n_seqs, const int32_t* start,
                const int32_t* len, bool want_len) {
    if (rows < 0 || rows > Q4GEMV_MAX_ROWS) return bad(h, Q4_ESHAPE, call, "rows outside [0, 2^24]");
    if (n_seqs < 0 || n_seqs > Q4GEMV_MAX_SEQS) return bad(h, Q4_ESHAPE, call, "n_seqs outside [0, 65535]");
    if (n_seqs > 0 && (!start || (want_len && !len))) return bad(h, Q4_EINVAL, call, "null start or len");
    if (!aligned(start, 4) || !aligned(len, 4)) return bad(h, Q4_EALIGN, call, "start or len not 4-byte aligned");
    return Q4_OK;
}

int check_kv(q4gemv_t h, const char* call, const q4gemv_kv* kv) {
    if (!kv) return bad(h, Q4_EINVAL, call, "null cache");
    if (!kv->k || !kv->v || !kv->table) return bad(h, Q4_EINVAL, call, "null pointer in the cache");
    if (kv->dtype != Q4GEMV_F16 && kv->dtype != Q4GEMV_BF16) return bad(h, Q4_EINVAL, call, "unknown dtype");
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->table, 4))
        return bad(h, Q4_EALIGN, call, "misaligned cache pointer");
    if (!head_dim_ok(kv->head_dim)) return bad(h, Q4_ESHAPE, call, "head_dim is not a multiple of 8 in [8, 256]");
    if (kv->n_heads < 1 || kv->n_heads > Q4GEMV_MAX_HEADS) return bad(h, Q4_ESHAPE, call, "n_heads outside [1, 1024]");
    if (kv->n_pages < 1 || kv->n_pages > INT32_MAX) return bad(h, Q4_ESHAPE, call, "n_pages outside [1, 2^31)");
    if (kv->page_size < 1 || kv->page_size > (1 << 20)) return bad(h, Q4_ESHAPE, call, "page_size outside [1, 2^20]");
    if (kv->table_cols < 1 || kv->table_cols > INT32_MAX || kv->table_stride < kv->table_cols)
        return bad(h, Q4_ESHAPE, call, "table_cols outside [1, table_stride]");
    const int64_t s[3] = {kv->page_stride, kv->token_stride, kv->head_stride};
    for (int64_t x : s)
        if (x < 0 || x % 8 != 0 || x > (int64_t(1) << 40))
            return bad(h, Q4_ESHAPE, call, "a cache stride is negative or not a multiple of 8");
    if ((kv->n_heads > 1 && kv->head_stride < kv->head_dim) || (kv->page_size > 1 && kv->token_stride < kv->head_dim) ||
        (kv->n_pages > 1 && kv->page_stride < kv->head_dim))
        return bad(h, Q4_ESHAPE, call, "cache strides under head_dim");
    return Q4_OK;
}

q4::KvArgs kv_args(const q4gemv_kv& c) {
    q4::KvArgs k;
    k.k = c.k;
    k.v = c.v;
    k.table = c.table;
    k.page_stride = c.page_stride;
    k.token_stride = c.token_stride;
    k.head_stride = c.head_stride;
    k.table_stride = c.table_stride;
    k.n_pages = (int)c.n_pages;
    k.table_cols = (int)c.table_cols;
    k.page_size = (int)c.page_size;
    k.n_heads = (int)c.n_heads;
    k.head_dim = (int)c.head_dim;
    k.page_shift = -1;
    for (int b = 0; b <= 20; ++b)
        if (c.page_size == (int64_t(1) << b)) k.page_shift = b;
    return k;
}

q4::RaggedArgs ragged(int64_t rows, int64_t n_seqs, const int32_t* start, const int32_t* len) {
    q4::RaggedArgs b;
    b.start = start;
    b.len = len;
    b.rows = rows;
    b.n_seqs = (int)n_seqs;
    return b;
}

// Up to this many rows of a sequence always go to attn_split_kernel, and up to
// as many as keep all its tiles' reads (tiles of 16 rows x key heads x cached
// tokens, by the table's capacity) under kSplitReads.  Measured (us, that
// kernel / the tensor-core one): 320 rows of 8 key heads of 128 over 1000 tokens
// 32 / 36, 640 rows 48 / 36; 80 rows over 30000 tokens 111 / 90; 1024 rows of
// one key head of 64 over 8000 tokens 39 / 43.  With head sizes over 128 a read
// costs that kernel more: 512 rows of 4 key heads of 256 over 1000 tokens 60 /
// 38, 128 rows 36 / 38; 512 rows over none 13 / 17, 1024 rows 33 / 20.
constexpr int kSplitRowsMin = 64, kSplitRowsMax = 1024;
constexpr int64_t kSplitReads = 300000, kSplitReadsWide = 60000;
// Sequences of up to this many new tokens run token by token.  Measured, 40
// heads of 128 x 128: 0.65 us a token against 11 us for a chunk of up to 128;
// with 8 such sequences the two meet between 12 and 16 tokens.
constexpr int kLinRecurMax = 12;
// Chunks of a prompt's segment, at least.
constexpr int kLinSegChunks = 4;

// Places and rows of a sequence stay this far under 2^31: kernels round them up
// to tiles, and the cost of a tensor-core unit is its first row tile's keys
// plus up to a place for each new token (at most 2^24).
constexpr int64_t kSlack = 1 << 25;

int split_dp(int64_t d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <typename T, int DP>
cudaError_t split_launch_dp(const q4::SplitAttnArgs& g, int sms, cudaStream_t st) {
    return launch(q4::attn_split_kernel<T, DP>, dim3((unsigned)(sms * q4::split_ctas_per_sm(DP))), q4::kSplitThreads,
                  q4::split_smem(DP), st, g);
}
template <typename T>
cudaError_t split_launch(const q4::SplitAttnArgs& g, int sms, cudaStream_t st) {
    const int dp = split_dp(g.a.kv.head_dim);
    return dp == 64 ? split_launch_dp<T, 64>(g, sms, st)
                    : dp == 128 ? split_launch_dp<T, 128>(g, sms, st) : split_launch_dp<T, 256>(g, sms, st);
}
template <typename T, int DP>
cudaError_t split_setup() {
    return cudaFuncSetAttribute(q4::attn_split_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                q4::split_smem(DP));
}

// Tensor map of 16-bit elements in the 128-byte swizzle, boxes of 64 elements;
// false where the driver refuses it.
bool tensor_map(CUtensorMap* map, const void* base, int dtype, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                const cuuint32_t* box) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<Encode>(f);
    }();
    if (!encode) return false;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return encode(map, dtype == Q4GEMV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One half of a paged cache, boxes of `box` tokens.
bool page_map(CUtensorMap* map, void* base, const q4gemv_kv& c, int box) {
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.n_heads,
                                (cuuint64_t)c.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.token_stride * 2, (cuuint64_t)c.head_stride * 2,
                                   (cuuint64_t)c.page_stride * 2};
    const cuuint32_t b[4] = {64, (cuuint32_t)box, 1, 1};
    return tensor_map(map, base, c.dtype, 4, dims, strides, b);
}

// Rows of heads, boxes of a chunk's rows.
bool row_map(CUtensorMap* map, const void* base, int dtype, int64_t dim, int64_t heads, int64_t rows, int64_t stride) {
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t b[3] = {64, 1, (cuuint32_t)q4::kLtTokens};
    return tensor_map(map, base, dtype, 3, dims, strides, b);
}

template <typename T>
cudaError_t tc_launch(const q4::TcAttnArgs& g, int sms, cudaStream_t st) {
    const dim3 grid((unsigned)sms);
    const int dp = split_dp(g.a.kv.head_dim);
    return dp == 64 ? launch(q4::attn_tc_kernel<T, 64>, grid, q4::kTaThreads, q4::ta_smem(64), st, g)
         : dp == 128 ? launch(q4::attn_tc_kernel<T, 128>, grid, q4::kTaThreads, q4::ta_smem(128), st, g)
                     : launch(q4::attn_tc_kernel<T, 256>, grid, q4::kTaThreads, q4::ta_smem(256), st, g);
}
template <typename T, int DP>
cudaError_t tc_setup() {
    return cudaFuncSetAttribute(q4::attn_tc_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, q4::ta_smem(DP));
}

template <typename F>
cudaError_t smem_limit(F* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}
template <typename T>
cudaError_t setup_type() {
    for (cudaError_t e :
         {split_setup<T, 64>(), split_setup<T, 128>(), split_setup<T, 256>(), tc_setup<T, 64>(), tc_setup<T, 128>(),
          tc_setup<T, 256>(),
          smem_limit(q4::lin_chunk_kernel<T, 256, 4, true>, q4::lc_smem(256, 4, true)),
          smem_limit(q4::lin_chunk_kernel<T, 256, 4, false>, q4::lc_smem(256, 4, false)),
          smem_limit(q4::lin_tc_kernel<T, 64, true>, q4::lt_smem(64, true)),
          smem_limit(q4::lin_tc_kernel<T, 64, false>, q4::lt_smem(64, false)),
          smem_limit(q4::lin_tc_kernel<T, 128, true>, q4::lt_smem(128, true)),
          smem_limit(q4::lin_tc_kernel<T, 128, false>, q4::lt_smem(128, false))})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

// Loads a kernel now: its first launch may be in a graph's capture.
template <typename F>
cudaError_t load(F* kernel) {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kernel);
}
template <typename T>
cudaError_t load_type() {
    for (cudaError_t e :
         {load(q4::kv_append_kernel<T, q4::kRopeInterleaved>), load(q4::kv_append_kernel<T, q4::kRopeHalf>),
          load(q4::kv_append_kernel<T, q4::kRopeHalfScalar>), load(q4::lin_recur_kernel<T, 4>),
          load(q4::lin_recur_kernel<T, 8>), load(q4::lin_recur_kernel<T, 16>)})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

template <typename T>
cudaError_t append_launch(const q4::AppendArgs& a, bool interleaved, dim3 grid, cudaStream_t st) {
    if (interleaved)
        return launch(q4::kv_append_kernel<T, q4::kRopeInterleaved>, grid, q4::kAppendThreads, 0, st, a);
    if (a.rot % 16 == 0) return launch(q4::kv_append_kernel<T, q4::kRopeHalf>, grid, q4::kAppendThreads, 0, st, a);
    return launch(q4::kv_append_kernel<T, q4::kRopeHalfScalar>, grid, q4::kAppendThreads, 0, st, a);
}

}  // namespace

cudaError_t q4::mix_setup() {
    for (cudaError_t e : {setup_type<__half>(), setup_type<__nv_bfloat16>(), load_type<__half>(),
                          load_type<__nv_bfloat16>(), load(q4::lin_scan_kernel)})
        if (e != cudaSuccess) return e;
    return cudaSuccess;
}

void q4::mix_workspace(int sms, size_t* ws_bytes, size_t* cnt_bytes) {
    size_t floats = 0, ctas = 0;
    for (int dp : {64, 128, 256}) {
        const size_t n = (size_t)sms * q4::split_ctas_per_sm(dp);
        floats = std::max(floats, 2 * n * q4::split_slot(dp));
        ctas = std::max(ctas, n);
    }
    floats = std::max(floats, 2 * (size_t)sms * std::max(q4::ta_slot(128), q4::ta_slot(256)));
    *ws_bytes = floats * sizeof(float);
    *cnt_bytes = ctas * sizeof(int);
}

extern "C" {

int q4gemv_rope_freqs(int kind, int rot, double base, double factor, double trained, double lo, double hi,
                      double* freqs) {
    if (!freqs || kind < Q4GEMV_ROPE_PLAIN || kind > Q4GEMV_ROPE_BY_PARTS) return Q4_EINVAL;
    if (rot < 0 || rot > Q4GEMV_MAX_HEAD_DIM || rot % 2 != 0) return Q4_ESHAPE;
    if (!(base > 0) || !std::isfinite(base)) return Q4_EINVAL;
    if (kind != Q4GEMV_ROPE_PLAIN && (!(factor >= 1) || !std::isfinite(factor))) return Q4_EINVAL;
    if (kind == Q4GEMV_ROPE_BY_PARTS &&
        (!(trained > 0) || !std::isfinite(trained) || !(lo < hi) || !std::isfinite(lo) || !std::isfinite(hi)))
        return Q4_EINVAL;
    const double two_pi = 6.283185307179586476925;
    for (int f = 0; f < rot / 2; ++f) {
        double w = std::pow(base, -2.0 * f / rot);
        if (kind == Q4GEMV_ROPE_LINEAR) w /= factor;
        if (kind == Q4GEMV_ROPE_BY_PARTS) {
            double keep = (trained * w / two_pi - lo) / (hi - lo);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            w *= keep + (1 - keep) / factor;
        }
        freqs[f] = w;
    }
    return Q4_OK;
}

int q4gemv_kv_append(q4gemv_t h, const q4gemv_kv* kv, int64_t rows, int64_t n_seqs, const int32_t* start,
                     const int32_t* len, const int32_t* pos, const q4gemv_rope* rope, const void* q,
                     int64_t q_stride, int64_t q_heads, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, void* q_out, int64_t q_out_stride, q4gemv_stream_t stream) {
    static const char* const call = "kv_append";
    if (!h) return Q4_EINVAL;
    int rc = check_kv(h, call, kv);
    if (rc == Q4_OK) rc = check_batch(h, call, rows, n_seqs, start, len, true);
    if (rc != Q4_OK) return rc;
    const int64_t D = kv->head_dim;
    if (rope && (rope->rot < 0 || rope->rot > D || rope->rot % 2 != 0))
        return bad(h, Q4_ESHAPE, call, "rot is odd or outside [0, head_dim]");
    if (rope && rope->rot > 0 && !rope->freqs) return bad(h, Q4_EINVAL, call, "null freqs");
    if (rope && !std::isfinite(rope->amp)) return bad(h, Q4_EINVAL, call, "amp is not finite");
    if (rows > 0 && (!k || !v || (q && !q_out))) return bad(h, Q4_EINVAL, call, "null pointer");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || (q && !aligned(q_out, 16)) || !aligned(pos, 4) ||
        (rope && !aligned(rope->freqs, 8)))
        return bad(h, Q4_EALIGN, call, "misaligned pointer");
    if (!row_stride_ok(k_stride, kv->n_heads, D) || !row_stride_ok(v_stride, kv->n_heads, D))
        return bad(h, Q4_ESHAPE, call, "row stride of k or v");
    if (q) {
        if (q_heads < 1 || q_heads > Q4GEMV_MAX_HEADS) return bad(h, Q4_ESHAPE, call, "q_heads outside [1, 1024]");
        if (!row_stride_ok(q_stride, q_heads, D) || !row_stride_ok(q_out_stride, q_heads, D))
            return bad(h, Q4_ESHAPE, call, "row stride of q or q_out");
        if (q == q_out && q_stride != q_out_stride)
            return bad(h, Q4_EINVAL, call, "q_out is q with another stride");
    }
    const q4::CtxView cx = q4::ctx_view(h);
    if (rows == 0 || n_seqs == 0) return Q4_OK;
    if (cx.fail_launch) return bad(h, Q4_EFAULTINJ, call, "injected launch failure");
    DeviceScope dev(cx.device);
    if (!dev.ok) return bad(h, Q4_ECUDA, call, "cudaSetDevice");
    q4::AppendArgs a;
    a.batch = ragged(rows, n_seqs, start, len);
    a.kv = kv_args(*kv);
    a.pos = pos;
    a.rot = rope ? rope->rot : 0;
    a.freqs = a.rot ? rope->freqs : nullptr;
    a.amp = rope ? rope->amp : 1.f;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.qo_stride = q_out_stride;
    a.q_heads = q ? (int)q_heads : 0;
    a.err = cx.err;
    // A row's heads over several CTAs while the rows alone leave SMs idle.
    const int64_t heads = a.q_heads + kv->n_heads;
    int64_t ny = (4 * (int64_t)cx.sms + rows - 1) / rows;
    if (ny > (heads + 7) / 8) ny = (heads + 7) / 8;
    if (ny < 1) ny = 1;
    const dim3 grid((unsigned)rows, (unsigned)ny);
    const bool il = rope && rope->interleaved;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_status(h, kv->dtype == Q4GEMV_F16 ? append_launch<__half>(a, il, grid, st)
                                                    : append_launch<__nv_bfloat16>(a, il, grid, st), call);
}

int q4gemv_attn_paged(q4gemv_t h, const q4gemv_kv* kv, int64_t rows, int64_t n_seqs, const int32_t* start,
                      const int32_t* len, int64_t max_new, const void* q, int64_t q_stride, int64_t q_heads,
                      void* out, int64_t out_stride, float scale, int causal, int64_t window,
                      q4gemv_stream_t stream) {
    static const char* const call = "attn_paged";
    if (!h) return Q4_EINVAL;
    int rc = check_kv(h, call, kv);
    if (rc == Q4_OK) rc = check_batch(h, call, rows, n_seqs, start, len, true);
    if (rc != Q4_OK) return rc;
    if (max_new < 1) return bad(h, Q4_EINVAL, call, "max_new under 1");
    if (q_heads < 1 || q_heads > Q4GEMV_MAX_HEADS || q_heads % kv->n_heads != 0)
        return bad(h, Q4_ESHAPE, call, "q_heads is not a multiple of n_heads in [1, 1024]");
    if (rows * (q_heads / kv->n_heads) > INT32_MAX - kSlack)     // kernels count them in 32 bits
        return bad(h, Q4_ESHAPE, call, "rows times the query heads of a key head of 2^31 - 2^25 or more");
    if (rows > 0 && (!q || !out)) return bad(h, Q4_EINVAL, call, "null pointer");
    if (!aligned(q, 16) || !aligned(out, 16)) return bad(h, Q4_EALIGN, call, "misaligned pointer");
    if (!row_stride_ok(q_stride, q_heads, kv->head_dim) || !row_stride_ok(out_stride, q_heads, kv->head_dim))
        return bad(h, Q4_ESHAPE, call, "row stride of q or out");
    if (rows > 0 && q == out) return bad(h, Q4_EINVAL, call, "out is q");
    if (!std::isfinite(scale)) return bad(h, Q4_EINVAL, call, "scale is not finite");
    if (window < 0) return bad(h, Q4_EINVAL, call, "negative window");
    const q4::CtxView cx = q4::ctx_view(h);
    if (rows == 0 || n_seqs == 0) return Q4_OK;
    if (cx.fail_launch) return bad(h, Q4_EFAULTINJ, call, "injected launch failure");
    DeviceScope dev(cx.device);
    if (!dev.ok) return bad(h, Q4_ECUDA, call, "cudaSetDevice");
    q4::AttnArgs a;
    a.batch = ragged(rows, n_seqs, start, len);
    a.kv = kv_args(*kv);
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.o_stride = out_stride;
    a.q_heads = (int)q_heads;
    a.group = (int)(q_heads / kv->n_heads);
    a.scale_log2 = (float)((double)scale * 1.4426950408889634074);
    a.causal = causal ? 1 : 0;
    a.window = window > INT32_MAX ? INT32_MAX : (int)window;
    a.cap = (int)std::min<int64_t>(kv->table_cols * kv->page_size, INT32_MAX - kSlack);
    a.err = cx.err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f16 = kv->dtype == Q4GEMV_F16;
    // Sequences with many rows (new tokens times query heads of a key head) go
    // to the tensor-core kernel, those with few to the other; a batch that may
    // hold both runs both.
    const int64_t reads = kv->n_heads * n_seqs * (int64_t)a.cap;     // of one tile of each sequence
    const int64_t most = kv->head_dim > 128 ? kSplitReadsWide : kSplitReads;
    const int limit = (int)std::max<int64_t>(kSplitRowsMin, std::min<int64_t>(kSplitRowsMax, 16 * (most / reads)));
    const bool many = max_new > limit / a.group;
    const bool few = !many || n_seqs > 1;
    if (many) {
        q4::TcAttnArgs g;
        g.a = a;
        g.ws = cx.attn_ws;
        g.cnt = cx.attn_cnt;
        g.min_rows = few ? limit : 0;
        const int dp = split_dp(kv->head_dim);
        // Boxes of the largest power of two of tokens that divides a page, up
        // to a tile; under 8 they would be more than the 16-byte copies' work.
        g.box = (int)std::min<int64_t>(kv->page_size & -kv->page_size, q4::kTaKeys);
        if (g.box < 8) g.box = 0;
        if (g.box && !(page_map(&g.kmap, kv->k, *kv, g.box) && page_map(&g.vmap, kv->v, *kv, g.box))) g.box = 0;
        g.idesc_s = q4::tc_idesc_16(128, q4::kTaKeys, !f16, false);
        g.idesc_o = q4::tc_idesc_16(128, dp, !f16, true);
        const int e = launch_status(h, f16 ? tc_launch<__half>(g, cx.sms, st) : tc_launch<__nv_bfloat16>(g, cx.sms, st), call);
        if (e != Q4_OK || !few) return e;
    }
    q4::SplitAttnArgs g;
    g.a = a;
    g.ws = cx.attn_ws;
    g.cnt = cx.attn_cnt;
    g.max_rows = many ? limit : 0;
    return launch_status(h, f16 ? split_launch<__half>(g, cx.sms, st) : split_launch<__nv_bfloat16>(g, cx.sms, st), call);
}

}  // extern "C"

namespace {

template <typename T>
cudaError_t lin_recur_launch(const q4::LinArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)a.n_seqs, (unsigned)a.v_heads, (unsigned)((a.v_dim + q4::kLinCols - 1) / q4::kLinCols));
    if (a.k_dim <= 64) return launch(q4::lin_recur_kernel<T, 4>, grid, q4::kLinThreads, 0, st, a);
    if (a.k_dim <= 128) return launch(q4::lin_recur_kernel<T, 8>, grid, q4::kLinThreads, 0, st, a);
    return launch(q4::lin_recur_kernel<T, 16>, grid, q4::kLinThreads, 0, st, a);
}

template <typename T, bool OUT>
cudaError_t lin_chunks(const q4::LinTcArgs& ta, cudaStream_t st) {
    const q4::LinSegArgs& g = ta.g;
    const unsigned z = (unsigned)(g.a.n_seqs * g.segs), y = (unsigned)((g.a.v_dim + 127) / 128);
    if (g.tokens != q4::kLtTokens)
        return launch(q4::lin_chunk_kernel<T, 256, 4, OUT>, dim3((unsigned)g.a.v_heads, (unsigned)((g.a.v_dim + 63) / 64), z),
                      64 * 4, q4::lc_smem(256, 4, OUT), st, g);
    const dim3 grid((unsigned)g.a.v_heads, y, z);
    return g.a.k_dim <= 64 ? launch(q4::lin_tc_kernel<T, 64, OUT>, grid, q4::kLtThreads, q4::lt_smem(64, OUT), st, ta)
                           : launch(q4::lin_tc_kernel<T, 128, OUT>, grid, q4::kLtThreads, q4::lt_smem(128, OUT), st, ta);
}

// Prompts run in chunks, cut into segments where sequences and heads alone
// would leave SMs idle (a segment costs half as much again: its gain is
// computed first).
template <typename T>
cudaError_t lin_prompt_launch(const q4::LinArgs& a, int64_t qk_heads, int dtype, int64_t max_new, const q4::CtxView& cx,
                              cudaStream_t st) {
    q4::LinTcArgs ta;
    q4::LinSegArgs& g = ta.g;
    g.a = a;
    g.ws = cx.attn_ws;
    const bool bf16 = dtype == Q4GEMV_BF16;
    ta.idesc_a = ta.idesc_i = q4::tc_idesc_16(128, 128, bf16, false);
    ta.idesc_o = q4::tc_idesc_16(128, 128, bf16, true);
    ta.idesc_s = q4::tc_idesc_16(128, a.k_dim <= 64 ? 64 : 128, bf16, true) | q4::kTcAMmajor;
    // The tcgen05 kernel holds states of up to 128 x 128; it reads whole boxes
    // of rows by tensor map.
    const bool tc = a.k_dim <= 128 && a.rows > 0 &&
                    row_map(&ta.qmap, a.q, dtype, a.k_dim, qk_heads, a.rows, a.q_stride) &&
                    row_map(&ta.kmap, a.k, dtype, a.k_dim, qk_heads, a.rows, a.k_stride) &&
                    row_map(&ta.vmap, a.v, dtype, a.v_dim, a.v_heads, a.rows, a.v_stride) &&
                    row_map(&ta.omap, a.out, dtype, a.v_dim, a.v_heads, a.rows, a.o_stride);
    g.tokens = tc ? q4::kLtTokens : q4::kLcTokens;
    const int64_t slices = tc ? (a.v_dim + 127) / 128 : (a.v_dim + 63) / 64;
    const int64_t ctas = (int64_t)a.n_seqs * a.v_heads * slices;
    const int64_t chunks = (std::min(max_new, a.rows) + g.tokens - 1) / g.tokens;
    const int64_t room = (int64_t)(cx.attn_ws_bytes / sizeof(float)) /
                         ((int64_t)a.n_seqs * a.v_heads * ((int64_t)a.k_dim * a.v_dim + 1));
    const int64_t segs = std::min<int64_t>({cx.sms / ctas, chunks / kLinSegChunks, room, 65535 / a.n_seqs});
    g.segs = segs < 3 ? 1 : (int)segs;
    if (g.segs > 1) {
        cudaError_t e = lin_chunks<T, false>(ta, st);
        if (e != cudaSuccess) return e;
        const int64_t size = (int64_t)a.k_dim * a.v_dim;
        e = launch(q4::lin_scan_kernel, dim3((unsigned)((size / 4 + q4::kLinScanThreads - 1) / q4::kLinScanThreads),
                                             (unsigned)a.v_heads, (unsigned)a.n_seqs),
                   q4::kLinScanThreads, 0, st, g);
        if (e != cudaSuccess) return e;
    }
    return lin_chunks<T, true>(ta, st);
}

}  // namespace

extern "C" int q4gemv_linattn(q4gemv_t h, const q4gemv_linattn_args* args, int64_t rows, int64_t n_seqs,
                              const int32_t* start, int64_t max_new, q4gemv_stream_t stream) {
    static const char* const call = "linattn";
    if (!h) return Q4_EINVAL;
    if (!args) return bad(h, Q4_EINVAL, call, "null arguments");
    const int rc = check_batch(h, call, rows, n_seqs, start, nullptr, false);
    if (rc != Q4_OK) return rc;
    const q4gemv_linattn_args& p = *args;
    if (max_new < 1) return bad(h, Q4_EINVAL, call, "max_new under 1");
    if (p.dtype != Q4GEMV_F16 && p.dtype != Q4GEMV_BF16) return bad(h, Q4_EINVAL, call, "unknown dtype");
    if (!head_dim_ok(p.k_dim) || !head_dim_ok(p.v_dim))
        return bad(h, Q4_ESHAPE, call, "k_dim or v_dim is not a multiple of 8 in [8, 256]");
    if (p.qk_heads < 1 || p.v_heads < 1 || p.v_heads > Q4GEMV_MAX_HEADS || p.v_heads % p.qk_heads != 0)
        return bad(h, Q4_ESHAPE, call, "v_heads is not a multiple of qk_heads in [1, 1024]");
    if (p.n_slots < 0 || p.n_slots > INT32_MAX) return bad(h, Q4_ESHAPE, call, "n_slots outside [0, 2^31)");
    if (!p.slots && n_seqs > p.n_slots) return bad(h, Q4_ESHAPE, call, "fewer states than sequences");
    if (rows > 0 && (!p.q || !p.k || !p.v || !p.log_decay || !p.out)) return bad(h, Q4_EINVAL, call, "null pointer");
    if (n_seqs > 0 && !p.state_out) return bad(h, Q4_EINVAL, call, "null state_out");
    if (!aligned(p.q, 16) || !aligned(p.k, 16) || !aligned(p.v, 16) || !aligned(p.out, 16) ||
        !aligned(p.state_in, 16) || !aligned(p.state_out, 16) || !aligned(p.log_decay, 4) || !aligned(p.slots, 4))
        return bad(h, Q4_EALIGN, call, "misaligned pointer");
    if (!row_stride_ok(p.q_stride, p.qk_heads, p.k_dim) || !row_stride_ok(p.k_stride, p.qk_heads, p.k_dim) ||
        !row_stride_ok(p.v_stride, p.v_heads, p.v_dim) || !row_stride_ok(p.out_stride, p.v_heads, p.v_dim))
        return bad(h, Q4_ESHAPE, call, "row stride of q, k, v or out");
    if (p.decay_stride != 0 && (p.decay_stride < p.v_heads || p.decay_stride > (int64_t(1) << 40)))
        return bad(h, Q4_ESHAPE, call, "row stride of log_decay");
    if (rows > 0 && (p.out == p.q || p.out == p.k || p.out == p.v)) return bad(h, Q4_EINVAL, call, "out is an input");
    if (!std::isfinite(p.scale)) return bad(h, Q4_EINVAL, call, "scale is not finite");
    const q4::CtxView cx = q4::ctx_view(h);
    if (n_seqs == 0) return Q4_OK;
    if (cx.fail_launch) return bad(h, Q4_EFAULTINJ, call, "injected launch failure");
    DeviceScope dev(cx.device);
    if (!dev.ok) return bad(h, Q4_ECUDA, call, "cudaSetDevice");
    q4::LinArgs a;
    a.start = start;
    a.slots = p.slots;
    a.q = p.q;
    a.k = p.k;
    a.v = p.v;
    a.g = p.log_decay;
    a.state_in = p.state_in;
    a.state_out = p.state_out;
    a.out = p.out;
    a.rows = rows;
    a.q_stride = p.q_stride;
    a.k_stride = p.k_stride;
    a.v_stride = p.v_stride;
    a.g_stride = p.decay_stride;
    a.o_stride = p.out_stride;
    a.n_seqs = (int)n_seqs;
    a.n_slots = (int)p.n_slots;
    a.v_heads = (int)p.v_heads;
    a.each = (int)(p.v_heads / p.qk_heads);
    a.k_dim = (int)p.k_dim;
    a.v_dim = (int)p.v_dim;
    a.scale = p.scale;
    a.err = cx.err;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f16 = p.dtype == Q4GEMV_F16;
    if (max_new <= kLinRecurMax)
        return launch_status(h, f16 ? lin_recur_launch<__half>(a, st) : lin_recur_launch<__nv_bfloat16>(a, st), call);
    return launch_status(h, f16 ? lin_prompt_launch<__half>(a, p.qk_heads, p.dtype, max_new, cx, st)
                                : lin_prompt_launch<__nv_bfloat16>(a, p.qk_heads, p.dtype, max_new, cx, st), call);
}
