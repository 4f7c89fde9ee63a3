/*
 * q4gemv -- Q4_0 dequantise-and-multiply matrix-vector products on NVIDIA
 * B200 (sm_100a), the memory-bound core of quantised LLM decode.
 *
 * The operation (SwarmLLM coverage, originshq.com page, section "The Engine:
 * ~50 WGSL Kernels Written From Scratch"): decode reads every weight once per
 * token, dequantises the 4-bit values and accumulates the matrix-vector
 * product; speculative verification and prefill apply the same weights to a
 * handful of activation vectors (aipolix en-US page, section "Speculation is
 * used to amortize network round trips"; originshq.com page, section
 * "Multi-Device Performance and the Network Penalty", 16 tokens per round
 * trip).
 *
 *   y[m][n] = sum_k W[n][k] * x[m][k],   0 <= m < M, 0 <= n < N, 0 <= k < K
 *
 * W is Q4_0: the pages name the format (taozi.news page, section
 * "支持模型与限制") without laying it out; the GGUF block is used.  Each row
 * holds K/32 blocks of 18 bytes: an f16 scale d (little-endian) and 16 bytes
 * qs; weight j of a block has code q_j = qs[j] & 15 (j < 16) or
 * qs[j-16] >> 4 (j >= 16) and value (q_j - 8) * d.  x and y are row-major
 * IEEE binary16.
 *
 * Conventions for every entry point
 *  - All buffers are caller-owned device memory (except where a parameter
 *    says "host"); the library never frees them.  Pointers to device data
 *    must be 16-byte aligned.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 *    default stream) and perform no implicit device synchronisation, except
 *    q4gemv_create, q4gemv_destroy and q4gemv_sync_status.
 *  - Every call returns a q4gemv_status.  Arguments are validated on the host
 *    before anything is launched; an invalid call launches nothing.  The
 *    library throws no C++ exception across this interface and never traps
 *    on the device.  The text of the last error of a handle is available from
 *    q4gemv_last_error.
 *  - A handle owns a small device workspace (split-K partial sums, per-tile
 *    arrival counters, an error word) and the cached CUDA graph of
 *    q4gemv_run_stack.  Calls on one handle must not overlap on the GPU: keep
 *    them on one stream, or order them with events.  Use one handle per
 *    concurrent stream.  Overlap that the kernels detect is reported as
 *    Q4_ECONCURRENT by the next q4gemv_sync_status.
 */
#ifndef Q4GEMV_H
#define Q4GEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define Q4GEMV_API __attribute__((visibility("default")))
#else
#define Q4GEMV_API
#endif

typedef struct q4gemv_ctx* q4gemv_t;   /* opaque, library-owned */
typedef void* q4gemv_stream_t;         /* a cudaStream_t */

typedef enum {
    Q4_OK = 0,
    Q4_EINVAL = -1,        /* null handle or pointer, bad enum value */
    Q4_ESHAPE = -2,        /* K % 32 != 0, N or K <= 0, sizes beyond the limits */
    Q4_EALIGN = -3,        /* a device pointer is not 16-byte aligned */
    Q4_ENOMEM = -4,        /* device or host allocation failed */
    Q4_ECUDA = -5,         /* a CUDA runtime call failed (see q4gemv_last_error) */
    Q4_EUNSUPPORTED = -6,  /* M outside [1, 256], or the device is not sm_100 */
    Q4_ETIMEOUT = -7,      /* a bounded device-side wait gave up */
    Q4_EFAULTINJ = -8,     /* a host step failed on purpose (fault injection) */
    Q4_ECONCURRENT = -9,   /* kernels saw overlapping calls on one handle */
    Q4_EINDEX = -10        /* a page, place or state slot in device memory is out of range */
} q4gemv_status;

/* Limits checked by validation.  Besides these, ceil(N/32) * (K/32) must be
 * below 2^31. */
#define Q4GEMV_MAX_M 256            /* vectors per q4gemv_run call */
#define Q4GEMV_MAX_M_GEMV 16        /* above this, the tensor-core GEMM path */
#define Q4GEMV_MAX_N (1 << 22)     /* rows */
#define Q4GEMV_MAX_K (1 << 20)     /* columns */

/* Library version, (major << 16) | minor. */
Q4GEMV_API int q4gemv_version(void);

/* Creates a handle bound to CUDA device `device` (made current for the
 * call).  Queries the SM count and allocates the workspace.  Returns
 * Q4_EUNSUPPORTED on a device that is not compute capability 10.x. */
Q4GEMV_API int q4gemv_create(q4gemv_t* out, int device);

/* Synchronises the device, releases the workspace and cached graphs, frees
 * the handle.  Null is accepted (no-op). */
Q4GEMV_API int q4gemv_destroy(q4gemv_t h);

/* Bytes of a GGUF Q4_0 matrix: N * (K/32) * 18; 0 if the shape is invalid. */
Q4GEMV_API size_t q4gemv_gguf_bytes(int64_t N, int64_t K);

/* Bytes of the packed (repacked) matrix: Np * (K/32) * 18 with
 * Np = ceil(N/32)*32; 0 if the shape is invalid.
 *
 * Packed layout (the input of q4gemv_run).  Rows are padded to Np (padding
 * rows hold qs bytes 0x88 and d = +0, i.e. zero weights) and grouped into
 * tiles of 32 rows.  With KB = K/32, segment s = t*KB + b holds block b of
 * the rows of tile t and occupies the 576 bytes from 576*s; row
 * n = 32t + g + 8i (g in [0,8), i in [0,4)):
 *   segment bytes 16*(4g + c) + 4i + e  = qs[4c + e] of that block of row n
 *                                          (c, e in [0,4)), bytes [0, 512);
 *   segment bytes 512 + 8g + 2i, +1      = d of that block of row n
 *                                          (little-endian), bytes [512, 576).
 * A lane (g, c) of a warp thus finds qs word c of rows g, g+8, g+16, g+24 in
 * one 16-byte word and their four scales in one 8-byte word, and a run of
 * segments is one contiguous byte range (one bulk copy). */
Q4GEMV_API size_t q4gemv_packed_bytes(int64_t N, int64_t K);

/* Host-only check of q4gemv_run's arguments (no device access, no handle).
 * Returns the status q4gemv_run would return for these arguments before
 * launching anything. */
Q4GEMV_API int q4gemv_validate(int M, int64_t N, int64_t K, const void* W_packed,
                    const void* x, const void* y);

/* One-time repack of a GGUF Q4_0 matrix into the packed layout.
 *   gguf   : device, q4gemv_gguf_bytes(N, K) bytes (any alignment >= 2)
 *   packed : device, q4gemv_packed_bytes(N, K) bytes, 16-byte aligned,
 *            must not overlap gguf
 * Bit-exact: the packed bytes are a permutation of the GGUF bytes plus the
 * padding rows. */
Q4GEMV_API int q4gemv_repack(q4gemv_t h, const void* gguf, void* packed,
                  int64_t N, int64_t K, q4gemv_stream_t stream);

/* y[M][N] = W x[M][K]^T for a packed W.
 *   W_packed : device, q4gemv_packed_bytes(N, K) bytes
 *   x        : device, M*K binary16, row-major
 *   y        : device, M*N binary16, row-major (written, never read)
 * 1 <= M <= 256, K % 32 == 0.  Accumulation is fp32 or exact integer; y is
 * rounded to nearest even once.  Results beyond the binary16 range become
 * +-Inf; a non-finite x element makes the affected outputs NaN.  For M <= 2
 * the activations of each 32-column block are converted to 16-bit integers
 * with a power-of-two scale chosen so the block's largest magnitude is held
 * exactly (elements within a factor 16 of it are exact; others are rounded
 * to 2^-15 of the block maximum) and the per-block dot products are exact
 * integers.  Deterministic: the same inputs on the same device give the
 * same bits.
 * For 3 <= M <= 16 (and M <= 2 with K beyond the CUDA-core kernel's
 * activation staging) the mma.sync tensor-core kernel runs, as a grid of P
 * column panels whose
 * fp32 sums a second small kernel adds in panel order (P = 1 for large N and
 * K up to about 6,000 columns; more panels for narrow N, so a CTA stages a
 * short activation slice, and for wider K).  The panel sums live in a buffer
 * of P*M*N floats owned by the handle (preallocated for P*M*N <= 2^21; a
 * larger first call grows it, which synchronises the device and must not
 * happen during a stream capture).
 * With the environment variable Q4GEMV_SMALL_M=tcs (read at create) that
 * path runs on the tcgen05 tensor cores instead: kind::i8 MMAs, one per 128
 * rows x 32 columns, the weights dequantised to 16 (q - 8) in tensor memory
 * and the activations converted per block and vector to 15-bit integers X
 * (|X| <= 2^14, the block maximum exact) split into two signed bytes; the
 * int32 block sums are exact and scaled in fp32.  It keeps the same output
 * contract (non-finite inputs give NaN outputs for their vector) and uses
 * the same activation image buffer; it is slower than the mma.sync kernel on
 * the measured shapes and is kept for comparison.
 * For M = 17..256 (prefill chunks) a dense-contraction path on the tcgen05
 * tensor cores runs instead: "dequantise the weight tile, then multiply" --
 * each weight (q - 8) * d is split exactly into two binary16 parts (the
 * rounded value and its remainder), both multiply x (exact products), and
 * the sums accumulate in fp32.  Scales |d| >= 8192 overflow binary16 in the
 * split and give non-finite outputs.  A first kernel writes x into an
 * activation image owned by the handle (ceil(K/64) * Mp * 128 bytes, Mp = M
 * rounded up to 16; preallocated up to 16 MiB, grown like the panel sums);
 * the GEMM kernel covers 256 rows per CTA, and for narrow N splits K so the
 * grid fills the SMs, its fp32 split sums (P*M*N floats, the same buffer as
 * the panel sums) added in split order by the reduce kernel. */
Q4GEMV_API int q4gemv_run(q4gemv_t h, const void* W_packed, const void* x, void* y,
               int M, int64_t N, int64_t K, q4gemv_stream_t stream);

/* ---- Q8_0 matrices (the other GGUF format the pages name: taozi.news page,
 * section "支持模型与限制"; layout from GGUF).  A row holds K/32 blocks of 34
 * bytes: an f16 scale d (little-endian), then 32 signed 8-bit codes; weight
 * j of a block is qs[j] * d. */

/* The down GEMV fed directly by the gate+up GEMV: y[N] = W u for a packed
 * Q4_0 W (N x K), with u_k = SiLU(g_k) * up_k = g_k / (1 + e^-g_k) * up_k and
 * gate_up = [g | up] the 2K-entry binary16 output of the gate+up GEMV (gate
 * half first).  The pages name the model family (Qwen 3.8 27B: taozi.news
 * page, section "支持模型与限制"; originshq.com page, section "Limitations
 * and Open Questions") but not its FFN activation; this is that family's
 * gated unit.  u is computed in fp32 inside the kernel
 * (never written) and converted per 32-column block like any M = 1 input;
 * exact integer block sums, fp32 accumulation, y rounded once.
 *   gate_up : device, 2K binary16, 16-byte aligned
 *   y       : device, N binary16
 * Q4_EUNSUPPORTED for K beyond the M = 1 kernel's staging (K <= 36,864 and
 * its shared memory); otherwise errors as q4gemv_run.  Deterministic. */
Q4GEMV_API int q4gemv_run_swiglu(q4gemv_t h, const void* W_packed, const void* gate_up,
                      void* y, int64_t N, int64_t K, q4gemv_stream_t stream);

/* Bytes of a GGUF Q8_0 matrix: N * (K/32) * 34; 0 if the shape is invalid. */
Q4GEMV_API size_t q4gemv_q8_0_gguf_bytes(int64_t N, int64_t K);

/* Bytes of the packed Q8_0 matrix: Np * (K/32) * 34, Np = ceil(N/32)*32; 0 if
 * the shape is invalid.  Packed layout: rows padded to Np (padding rows hold
 * codes 0 and d = +0), tiles of 32 rows; segment s = t*KB + b (KB = K/32)
 * holds block b of the rows of tile t in the 1088 bytes from 1088*s; row
 * n = 32t + g + 8i (g in [0,8), i in [0,4)):
 *   segment bytes 32*(4g + c) + 8i + e      = qs[4c + e]       (c, e in [0,4))
 *   segment bytes 32*(4g + c) + 8i + 4 + e  = qs[16 + 4c + e]
 *   segment bytes 1024 + 8g + 2i, +1        = d (little-endian)
 * A lane (g, c) of a warp thus finds the codes it multiplies with the
 * activations' lane group c, for its four rows, in 32 contiguous bytes. */
Q4GEMV_API size_t q4gemv_q8_0_packed_bytes(int64_t N, int64_t K);

/* One-time repack of a GGUF Q8_0 matrix (arguments and errors as
 * q4gemv_repack; gguf any alignment >= 2).  Bit-exact. */
Q4GEMV_API int q4gemv_q8_0_repack(q4gemv_t h, const void* gguf, void* packed,
                       int64_t N, int64_t K, q4gemv_stream_t stream);

/* Host-only check of q4gemv_q8_0_run's arguments: Q4_EUNSUPPORTED for M
 * outside [1, 256], else as q4gemv_validate. */
Q4GEMV_API int q4gemv_q8_0_validate(int M, int64_t N, int64_t K, const void* W_packed,
                         const void* x, const void* y);

/* y[M][N] = W x[M][K]^T for a packed Q8_0 W, 1 <= M <= 256 (buffers as
 * q4gemv_run).  M <= 2 with M*K <= 36,864 (and the kernel's shared memory):
 * the activations are converted per 32-column block as for Q4_0 (exact for
 * the block maximum), each block's dot product with the 8-bit codes is an
 * exact integer, converted to fp32 once and scaled by d.  M <= 16 otherwise:
 * the mma.sync kernel of q4gemv_run's M = 3..16 path with Q8_0 segments (each
 * signed code exact in binary16, exact per-block sums in fp32, d applied once
 * per output and block; column panels for wide K).  M = 17..256: the
 * tcgen05 GEMM of q4gemv_run's M > 16 path runs with Q8_0 segments: each
 * weight q * d (up to 18 significant bits) is split exactly into two binary16
 * parts; scales |d| >= 512 overflow the split (non-finite outputs); its
 * activation image and split sums live in the same handle buffers.  fp32
 * accumulation; y rounded to binary16 once.  Deterministic. */
Q4GEMV_API int q4gemv_q8_0_run(q4gemv_t h, const void* W_packed, const void* x, void* y,
                    int M, int64_t N, int64_t K, q4gemv_stream_t stream);

/* One layer's packed matrices for q4gemv_run_stack. */
typedef struct {
    const void* qkv;      /* qkv_n  x hidden */
    const void* o;        /* hidden x hidden */
    const void* gate_up;  /* 2*ffn  x hidden (rows [0,ffn) gate, [ffn,2ffn) up) */
    const void* down;     /* hidden x ffn */
} q4gemv_layer;

/* One synthetic decode step (M = 1) through n_layers layers of four Q4_0
 * GEMVs each, the 27B-shaped workload of the pages (hidden 5120: taozi.news
 * page, section "技术架构"; 64 layers: originshq.com page, section "The
 * Architecture: Layers Distributed, Activations in Flight").  Every GEMV
 * output is rounded to binary16; the next GEMV reads its first K entries v
 * scaled to unit RMS by the real scalar s(v) = 1/sqrt(mean(v^2)) (0 for an
 * all-zero v), i.e. it computes f16(s(v) * (W v)):
 *     a = f16(QKV x),   b = f16(s(a') O a'),  a' = a[0:hidden]
 *     u = f16(s(b) gate_up b),   x' = f16(s(u') down u'),  u' = u[0:ffn]
 * and x_out = f16(s(x') x').  The pages give no layer math beyond the GEMVs,
 * so this chain (Q slice in place of attention, gate half without an
 * activation, a unit-RMS scale in place of the norm) is the reading adopted.
 * On the GPU s is taken in fp32: block sums of squares in a fixed binary tree,
 * blocks in a fixed order, the hardware's approximate reciprocal square root.
 *   layers  : HOST array of n_layers entries (device pointers inside)
 *   x_in    : hidden binary16 (not modified); device (16-byte aligned) or
 *             host memory, pinned or pageable: a host vector is copied to
 *             the device on `stream` inside the call
 *   x_out   : hidden binary16 (may alias x_in); device or host memory (a host
 *             vector is copied back on `stream` inside the call)
 *   trace_x : device or NULL; [4*n_layers][max(hidden, ffn)] binary16: the
 *             input vector of GEMV i = 4l + t (t = 0 QKV, 1 O, 2 gate_up,
 *             3 down), before its scale, in its first K_i entries
 *   trace_y : device or NULL; [4*n_layers][max(qkv_n, hidden, 2*ffn)]
 *             binary16: the raw output of GEMV i in its first N_i entries
 * Requires qkv_n >= hidden, qkv_n % 8 == 0, 1 <= n_layers <= 4096,
 * max(hidden, ffn) within one CTA's activation staging.  The step runs as ONE
 * cooperative persistent kernel (plus a 16-byte reset of its barrier words);
 * the first call with a given set of arguments uploads its descriptors and
 * must happen outside any stream capture, later calls only launch.  With the
 * environment variable Q4GEMV_STACK_MODE=kernels (read at create) the step
 * runs instead as a CUDA graph of one kernel per GEMV, captured on the first
 * call and replayed, or launched into the caller's capture when `stream` is
 * capturing; both modes give the same bits.  Host vectors are not accepted
 * while `stream` is capturing. */
Q4GEMV_API int q4gemv_run_stack(q4gemv_t h, const q4gemv_layer* layers, int n_layers,
                     int64_t hidden, int64_t qkv_n, int64_t ffn,
                     const void* x_in, void* x_out, void* trace_x,
                     void* trace_y, q4gemv_stream_t stream);

/* The decode step of q4gemv_run_stack with the feed-forward block's
 * activation: each layer's down GEMV takes u = SiLU(gate) * up of the whole
 * gate+up output (gate = rows [0, ffn), up = rows [ffn, 2 ffn); the pages
 * name the model family but not its activation -- taozi.news page, section
 * 支持模型与限制 -- so this is the common gated form, as in
 * q4gemv_run_swiglu), computed in fp32 inside the down GEMV's staging and
 * never written, and scaled to unit RMS like every input of the chain:
 * x' = f16(s(u) (down u)), s(u) = 1/sqrt(mean(u^2)).  Everything else,
 * arguments, modes and errors as q4gemv_run_stack (no traces). */
Q4GEMV_API int q4gemv_run_stack_gated(q4gemv_t h, const q4gemv_layer* layers, int n_layers,
                                      int64_t hidden, int64_t qkv_n, int64_t ffn,
                                      const void* x_in, void* x_out, q4gemv_stream_t stream);

/* ---- Row-sharded decode step over several GPUs (one process and one handle
 * per GPU).  The pages run the model split by contiguous layer ranges across
 * devices, passing the hidden state from one to the next (originshq.com page,
 * section "The Architecture: Layers Distributed, Activations in Flight";
 * taozi.news page, section "技术架构"); that pipelines tokens but does not
 * speed up one.  Here every GEMV of the step is split by output rows over
 * `world` GPUs and its output is all-gathered before the next GEMV, so one
 * token's step divides its weight bytes over the GPUs.
 *
 * Rows of an N-row matrix held by rank `rank`: [*row0, *row0 + *rows), whole
 * 32-row tiles, every rank holding *chunk = ceil(N / (32 world)) * 32 rows
 * or fewer (the last ranks: the remainder, possibly 0).  Host-only; no
 * device access.  Q4_EINVAL for N <= 0, world < 1 or rank outside
 * [0, world). */
Q4GEMV_API int q4gemv_shard_rows(int64_t N, int world, int rank, int64_t* row0, int64_t* rows,
                      int64_t* chunk);

/* An NCCL unique id (128 bytes, written to id) for q4gemv_comm_init: rank 0
 * calls it and sends the bytes to the other ranks.  NCCL (libnccl.so.2) is
 * loaded at run time; Q4_EUNSUPPORTED if it cannot be. */
Q4GEMV_API int q4gemv_comm_unique_id(void* id);

/* Binds the handle to rank `rank` of a `world`-GPU communicator created from
 * the unique id (every rank calls it with the same id; collective, blocks
 * until all ranks have joined).  Replaces an earlier communicator of the
 * handle. */
Q4GEMV_API int q4gemv_comm_init(q4gemv_t h, int world, int rank, const void* id);

/* Peer-memory exchange for the row-sharded step: instead of an NCCL
 * all-gather after every GEMV, each GEMV kernel stores its output rows
 * directly into every rank's gather buffer (CUDA IPC mappings over NVLink /
 * NVSwitch; plain stores, no multicast) and the next GEMV reads them there.
 * Every entry of a gather buffer is one 32-bit word, the binary16 value in
 * bits 0-15 and in bits 16-31 a stamp of the GEMV that wrote it: (steps run
 * x GEMVs per step + the GEMV's index in the step) mod 2^16.  A reader polls
 * (bounded) each word it needs until it carries the stamp it expects, so no
 * fence, flag or collective separates the GEMVs, and a GEMV starts (its
 * weights streaming) while the previous one ends.  The exchange buffer of a
 * rank (zeroed once) holds, for the four matrix types of the step (QKV, O,
 * gate+up, down), a gather buffer of world * chunk words (chunk from
 * q4gemv_shard_rows, rank r's rows at r * chunk), then the rank's step
 * count; offsets from q4gemv_peer_layout.
 *
 * Blob (Q4GEMV_PEER_BLOB_BYTES, little-endian): uint32 magic 0x51345045
 * ("EP4Q"), uint32 version 1, int32 world, int32 rank, int64 hidden, qkv_n,
 * ffn, uint64 buffer bytes, then the 64-byte cudaIpcMemHandle_t of the
 * buffer, zero padding to the end. */
#define Q4GEMV_PEER_BLOB_BYTES 128
#define Q4GEMV_PEER_MAX_WORLD 8

/* Byte offsets of the exchange buffer for these shapes: off[0..3] the gather
 * buffers of QKV, O, gate+up and down outputs, off[4] the step count, off[5]
 * the total size (six entries).  Host-only.  Q4_EINVAL for world outside
 * [1, Q4GEMV_PEER_MAX_WORLD] or non-positive shapes. */
Q4GEMV_API int q4gemv_peer_layout(int world, int64_t hidden, int64_t qkv_n, int64_t ffn,
                                  int64_t* off);

/* Checks `world` blobs (world * Q4GEMV_PEER_BLOB_BYTES bytes, rank order) for
 * one exchange: magic and version, the same world, shapes and buffer size in
 * all of them, blob r from rank r.  Host-only.  Q4_OK or Q4_EINVAL. */
Q4GEMV_API int q4gemv_peer_check(const void* blobs, int world);

/* Allocates (zeroed) this rank's exchange buffer for the step's shapes and
 * writes its blob.  Every rank calls it, sends its blob to all ranks (any
 * host channel) and then calls q4gemv_peer_open with all of them.  Replaces
 * an earlier exchange of the handle (synchronises the device). */
Q4GEMV_API int q4gemv_peer_export(q4gemv_t h, int world, int rank, int64_t hidden, int64_t qkv_n,
                                  int64_t ffn, void* blob);

/* Maps the other ranks' exchange buffers (cudaIpcOpenMemHandle) from the
 * `world` blobs of q4gemv_peer_export, in rank order, after q4gemv_peer_check
 * and a comparison with this handle's export.  From then on
 * q4gemv_run_stack_sharded with the exported shapes uses the peer-memory
 * exchange.  With world = 1 nothing is mapped (the rank's own buffer). */
Q4GEMV_API int q4gemv_peer_open(q4gemv_t h, const void* blobs);

/* Unmaps the peers' buffers and frees this rank's; every rank must stop
 * using the exchange first (no step of any rank in flight). */
Q4GEMV_API int q4gemv_peer_close(q4gemv_t h);

/* The decode step of q4gemv_run_stack, row-sharded: `layers` holds THIS
 * rank's row slices (q4gemv_shard_rows of each matrix, packed as q4gemv_run
 * matrices of `rows` rows; a slice of 0 rows may be NULL).  Per GEMV the rank
 * computes its rows f16(s(v) * W_slice v) from the full previous output v
 * (the M = 1 kernel; the scale as in q4gemv_run_stack), and every rank gets
 * the whole output: through the peer-memory exchange when it is open for
 * these shapes (stores by the GEMV kernel itself, above), else an NCCL
 * all-gather; x_out = f16(s(x') x') on every rank.  x_in, x_out: device
 * memory (hidden binary16), the same x_in on every rank.  Every rank must
 * make the same calls in the same order.  The step is captured as one CUDA
 * graph on the first call with these arguments (not inside the caller's
 * capture) and replayed.  Results agree with q4gemv_run_stack within the
 * GEMV tolerance (the row split changes the order of the partial sums, not
 * the arithmetic) and are the same bits on both exchanges.  Errors as
 * q4gemv_run_stack; Q4_EINVAL with neither a communicator nor an open
 * exchange for these shapes; a peer whose rows never come makes the waiting
 * GEMV report Q4_ETIMEOUT through q4gemv_sync_status (one time-out per step:
 * later waits of the step give up at once). */
Q4GEMV_API int q4gemv_run_stack_sharded(q4gemv_t h, const q4gemv_layer* layers_local,
                             int n_layers, int64_t hidden, int64_t qkv_n, int64_t ffn,
                             const void* x_in, void* x_out, q4gemv_stream_t stream);

/* Fixed limits of q4gemv_run_noalloc. */
#define Q4GEMV_NOALLOC_MAX_N (1 << 22)                 /* rows */
#define Q4GEMV_NOALLOC_SCRATCH_BYTES (2u << 20)        /* static device scratch */

/* q4gemv_run for M <= 2 without a handle and without allocating anything.
 * The paper has no counterpart; this is a library convenience.
 *
 * Who needs it: q4gemv_create obtains its workspace with cudaMalloc, which
 * some callers cannot do -- code that runs while a stream is captured in
 * global capture mode (cudaMalloc is then an error), threads that must not
 * take the implicit device synchronisation of cudaMalloc/cudaFree, and
 * plug-ins whose host application owns all device memory.  This entry point
 * runs the same kernel as q4gemv_run with its scratch (split-tile partial
 * sums, per-tile arrival counters, an error word) in one file-scope device
 * array of Q4GEMV_NOALLOC_SCRATCH_BYTES (2 MiB) that every GPU which loads
 * the library holds until the process exits.  It calls no cudaMalloc,
 * cudaFree or allocating library routine.
 *
 * Arguments as q4gemv_run (device pointers, 16-byte aligned, packed W), on
 * the current CUDA device, asynchronous on `stream`.  Limits: 1 <= M <= 2
 * (else Q4_EUNSUPPORTED); K % 32 == 0, N <= Q4GEMV_NOALLOC_MAX_N, and K <=
 * 24,896 for M = 1 or K <= 18,432 for M = 2 (the kernel's shared memory and
 * activation staging; else Q4_ESHAPE); at most 2560 warps are used.
 * Device-side error reports are not surfaced.
 *
 * The first call on a device sets that device up (resolves the array's
 * device address with cudaGetSymbolAddress, queries the SM count, sets the
 * kernels' shared-memory limit); make that first call before any stream
 * capture.  Every call shares the one array and clears its counters before
 * launching: calls that overlap on the GPU race and give wrong results, so
 * order them on one stream. */
Q4GEMV_API int q4gemv_run_noalloc(const void* W_packed, const void* x, void* y, int M,
                                  int64_t N, int64_t K, q4gemv_stream_t stream);

/* ---- Token mixing: what a layer does between its QKV and O products.  The
 * pages' trunk is a hybrid of attention layers and linear-attention layers
 * (taozi.news page, section "支持模型与限制"; originshq.com page, section
 * "Limitations and Open Questions") and gives no equations: the definitions
 * below are the common ones.
 *
 * A call takes the new tokens of a ragged batch of sequences: `rows` rows in
 * all, sequence s holding rows [start[s], start[s+1]) (device, n_seqs + 1
 * non-decreasing entries; a sequence may have none), and for the cached forms
 * len[s] (device, n_seqs entries), the tokens of sequence s in the cache with
 * the new ones counted.  New token t of n of sequence s thus has the place
 * len[s] - n + t.  Rows behind start[n_seqs] belong to no sequence: nothing
 * reads or writes them.  start, len, page tables and slots are read by the
 * kernels when they run, so a captured call follows later changes of them.
 * What they hold is checked on the device, never trusted: an entry out of
 * range is left out (each function says how) and the next q4gemv_sync_status
 * returns Q4_EINDEX.
 *
 * Elements are binary16 or bfloat16 (`dtype`, the same for every 16-bit
 * buffer of a call).  Strides are in elements; row strides of 16-bit buffers
 * are multiples of 8, so that rows keep the 16-byte alignment of their base;
 * the heads of a row lie one after the other.  Sums, softmax statistics and
 * states are in 32 bits, outputs rounded once.  All functions are
 * deterministic, may be captured into a graph from the first call on, and
 * launch nothing for rows == 0 (linattn: for n_seqs == 0). */
typedef enum { Q4GEMV_F16 = 0, Q4GEMV_BF16 = 1 } q4gemv_dtype;

#define Q4GEMV_MAX_HEAD_DIM 256      /* head_dim, k_dim, v_dim: multiples of 8 up to this */
#define Q4GEMV_MAX_HEADS 1024
#define Q4GEMV_MAX_SEQS 65535
#define Q4GEMV_MAX_ROWS (1 << 24)

/* A paged cache of keys and values (a host struct of device pointers, kept by
 * the caller).  Token t of sequence s is in page p = table[s * table_stride +
 * t / page_size], its head h at element p * page_stride +
 * (t % page_size) * token_stride + h * head_stride of both k and v.  Pages
 * that several sequences share may be read by all of them; a page that a
 * sequence appends to must be its own. */
typedef struct {
    void* k;                 /* 16-byte aligned */
    void* v;
    const int32_t* table;    /* [n_seqs][table_stride], pages of the pool */
    int64_t n_pages;         /* pages of the pool: 0 <= entry < n_pages */
    int64_t page_size;       /* tokens of a page, any count from 1 to 2^20 */
    int64_t n_heads;         /* key and value heads */
    int64_t head_dim;
    int64_t page_stride, token_stride, head_stride;   /* multiples of 8 */
    int64_t table_stride, table_cols;   /* between rows; entries of a row */
    int dtype;               /* q4gemv_dtype */
} q4gemv_kv;

/* Rotation of queries and keys by their positions.  The first `rot` (even)
 * elements of a head are rot/2 pairs: elements (f, f + rot/2) in the half
 * layout, (2f, 2f + 1) in the interleaved one; the rest passes.  Pair f of a
 * token at position p turns by p * freqs[f] radians: (a cos - b sin,
 * b cos + a sin) * amp.  Angles are taken in 64 bits. */
typedef struct {
    const double* freqs;     /* device, rot/2 entries (q4gemv_rope_freqs) */
    int rot;                 /* 0: no rotation */
    int interleaved;
    float amp;               /* factor of cos and sin; 1 for none */
} q4gemv_rope;

enum {
    Q4GEMV_ROPE_PLAIN = 0,      /* base^(-2f/rot) */
    Q4GEMV_ROPE_LINEAR = 1,     /* that / factor: positions interpolated */
    Q4GEMV_ROPE_BY_PARTS = 2    /* by the turns T that the pair takes in `trained` tokens:
                                 * under `lo` turns / factor, over `hi` unchanged, between
                                 * them mixed linearly in T */
};

/* Writes the rot/2 angular speeds of a rotation to `freqs` (HOST memory;
 * host-only, no device access).  factor, trained, lo and hi are used by the
 * scaled kinds only.  Q4_EINVAL for a null pointer, an unknown kind, base <= 0,
 * factor < 1, trained <= 0, lo >= hi or a value that is not finite; Q4_ESHAPE
 * for rot odd or outside [0, Q4GEMV_MAX_HEAD_DIM]. */
Q4GEMV_API int q4gemv_rope_freqs(int kind, int rot, double base, double factor, double trained,
                                 double lo, double hi, double* freqs);

/* Appends the new tokens' keys and values to the cache, keys rotated, and
 * rotates their queries.
 *   pos   : device, [rows] rotation positions, or NULL: the places
 *   rope  : host struct, or NULL: no rotation
 *   q     : device, [rows][q_heads][head_dim], rows q_stride apart, or NULL
 *           (then q_out is not used): the queries
 *   k, v  : device, [rows][n_heads][head_dim]
 *   q_out : device, rows q_out_stride apart; may be q (same stride), else it
 *           must not overlap the inputs
 * q, k and v may be slices of one row of the QKV product.  A row whose place
 * is negative, past the table's columns or in a page outside the pool is not
 * stored (Q4_EINDEX); its queries are rotated all the same. */
Q4GEMV_API int q4gemv_kv_append(q4gemv_t h, const q4gemv_kv* kv, int64_t rows, int64_t n_seqs,
                                const int32_t* start, const int32_t* len, const int32_t* pos,
                                const q4gemv_rope* rope, const void* q, int64_t q_stride,
                                int64_t q_heads, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, void* q_out, int64_t q_out_stride,
                                q4gemv_stream_t stream);

/* Attention of the new tokens over the cache (which holds their own keys and
 * values already):
 *   out = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale q.k_j),
 * j over the tokens that the new token at place p sees: j <= p if `causal`,
 * else every j < len[s]; with window > 0 only j > p - window.  Query head h
 * reads key head h / (q_heads / n_heads).  A row that sees no token (or whose
 * scores are all -Inf) gets zeros.  What a row does not see cannot reach it,
 * whatever it holds: tokens behind len[s] or behind the row's place, and
 * uninitialised parts of pages, may hold NaN.  Tokens in a page outside the
 * pool are left out (Q4_EINDEX).
 *   q     : device, [rows][q_heads][head_dim], rows q_stride apart
 *   out   : device, the same shape, rows out_stride apart; must not overlap
 *           q or the cache
 *   max_new : the most new tokens of a sequence, as far as the caller knows
 *           (1 <= max_new): it chooses the kernel, and results are right
 *           whatever it says
 * Tokens at places from 2^31 - 2^25 on are left out (Q4_EINDEX); rows times
 * the query heads of a key head stay under 2^31 - 2^25 (Q4_ESHAPE). */
Q4GEMV_API int q4gemv_attn_paged(q4gemv_t h, const q4gemv_kv* kv, int64_t rows, int64_t n_seqs,
                                 const int32_t* start, const int32_t* len, int64_t max_new,
                                 const void* q, int64_t q_stride, int64_t q_heads, void* out,
                                 int64_t out_stride, float scale, int causal, int64_t window,
                                 q4gemv_stream_t stream);

/* Linear attention with a decay for each head (a host struct of arguments):
 *   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   out_t = scale S_t^T q_t,
 * S the head's [k_dim][v_dim] state.  Value head h goes with query and key
 * head h / (v_heads / qk_heads). */
typedef struct {
    const void* q;           /* [rows][qk_heads][k_dim], rows q_stride apart */
    const void* k;           /* the same shape, rows k_stride apart */
    const void* v;           /* [rows][v_heads][v_dim], rows v_stride apart */
    const float* log_decay;  /* [rows][v_heads], rows decay_stride apart (any count, no
                              * alignment beyond 4 bytes); decay_stride 0: one row, fixed
                              * decays.  Entries <= 0 (-Inf clears the state) */
    const float* state_in;   /* [n_slots][v_heads][k_dim][v_dim]; NULL: zeros */
    float* state_out;        /* the same shape; may be state_in, else must not overlap it */
    const int32_t* slots;    /* device, [n_seqs]: the state of sequence s, no two the
                              * same; NULL: state s */
    void* out;               /* [rows][v_heads][v_dim], rows out_stride apart; must not
                              * overlap the inputs */
    int64_t q_stride, k_stride, v_stride, decay_stride, out_stride;
    int64_t n_slots, qk_heads, v_heads, k_dim, v_dim;
    float scale;
    int dtype;               /* q4gemv_dtype of q, k, v and out */
} q4gemv_linattn_args;

/* Runs the new tokens of every sequence through its state: reads state_in,
 * writes state_out (of the sequences' slots only; a sequence without new
 * tokens copies its state).  A sequence whose slot is outside [0, n_slots) is
 * left out, its rows unwritten (Q4_EINDEX).  max_new as in
 * q4gemv_attn_paged.  States are good up to magnitudes of 2^80 (many new tokens
 * are run in chunks that scale them by powers of two); an infinity in q, k or v
 * may come out as NaN wherever the formula takes it, and nowhere else. */
Q4GEMV_API int q4gemv_linattn(q4gemv_t h, const q4gemv_linattn_args* args, int64_t rows,
                              int64_t n_seqs, const int32_t* start, int64_t max_new,
                              q4gemv_stream_t stream);

/* A layer's token mixer in q4gemv_run_stack_mixed: attention over a paged cache
 * (table row 0 is the sequence's), or linear attention with fixed decays. */
enum { Q4GEMV_MIX_ATTENTION = 0, Q4GEMV_MIX_LINEAR = 1 };
typedef struct {
    int kind;
    q4gemv_kv kv;            /* attention: binary16, n_heads = kv_heads, head_dim = hidden/q_heads */
    const float* log_decay;  /* linear: device, [q_heads] */
    float* state;            /* linear: device, [q_heads][head_dim][head_dim], updated */
} q4gemv_mixer;

/* The decode step of q4gemv_run_stack_gated for one token of one sequence with
 * a token mixer between the QKV and the O product of every layer, in place of
 * the Q slice: the hybrid trunk's step.  With D = hidden / q_heads the QKV
 * product has hidden + 2 kv_heads D outputs a, and
 *   attention: a = [q | k | v] (q_heads, kv_heads, kv_heads heads of D); k
 *              (rotated) and v are appended to the layer's cache at place
 *              len[0] - 1 and the rotated q attends to the len[0] tokens there,
 *              scores times 1/sqrt(D): q4gemv_kv_append, q4gemv_attn_paged;
 *   linear:    a = [q | k | v] (kv_heads, kv_heads, q_heads heads of D):
 *              q4gemv_linattn with scale 1/sqrt(D) on the layer's state;
 * the mixer's output m (hidden binary16) goes to O, scaled to unit RMS like
 * every input of the chain: b = f16(s(m) O m).  Everything else as
 * q4gemv_run_stack_gated.
 *   layers, mixers : HOST arrays of n_layers entries (device pointers inside)
 *   rope    : host struct or NULL (device pointer inside), as q4gemv_kv_append
 *   len     : device, one entry: the sequence's tokens, the new one counted; the
 *             caller advances it between steps
 *   x_in, x_out : device, hidden binary16 (x_out may alias x_in)
 * Launches its kernels on `stream` (4 products and 1 or 2 mixer kernels a
 * layer), so it may be captured into a graph and replayed token by token; the
 * first call with larger sizes allocates (it waits for the device) and must
 * come outside a capture.  Arguments of all
 * layers are checked before anything is launched: errors of the parts it runs;
 * Q4_ESHAPE if q_heads does not divide hidden, kv_heads does not
 * divide q_heads, or a layer's cache has other heads. */
Q4GEMV_API int q4gemv_run_stack_mixed(q4gemv_t h, const q4gemv_layer* layers, const q4gemv_mixer* mixers,
                                      int n_layers, int64_t hidden, int64_t ffn, int64_t q_heads,
                                      int64_t kv_heads, const q4gemv_rope* rope, const int32_t* len,
                                      const void* x_in, void* x_out, q4gemv_stream_t stream);

/* Synchronises `stream`, then reads and clears the handle's device error
 * word: Q4_OK, Q4_ETIMEOUT, Q4_ECONCURRENT, Q4_EINDEX, or Q4_ECUDA if an earlier
 * asynchronous error is pending on the device. */
Q4GEMV_API int q4gemv_sync_status(q4gemv_t h, q4gemv_stream_t stream);

/* Static text for a status code. */
Q4GEMV_API const char* q4gemv_strerror(int status);

/* Text of the handle's last error (empty if none).  Valid until the next
 * call on the handle. */
Q4GEMV_API const char* q4gemv_last_error(q4gemv_t h);

/* Fault injection for tests.  which: "none"; "alloc" (workspace or buffer
 * allocation), "launch" (kernel launch) or "graph" (graph capture or
 * instantiation) make that host step of later calls fail with
 * Q4_EFAULTINJ; "timeout" makes later persistent decode steps
 * (q4gemv_run_stack) give every bounded device wait a budget of 1,024 polls
 * and ask their first inter-GEMV wait for a condition that never holds, so
 * the wait gives up, the kernel records Q4_ETIMEOUT in the handle's error
 * word, every CTA returns (after its copies in flight have landed) and the
 * next q4gemv_sync_status reports Q4_ETIMEOUT; the handle stays usable.  No
 * GPU fault, trap or unbounded wait is involved.  The environment variable
 * Q4GEMV_FAULT sets the initial value at q4gemv_create. */
Q4GEMV_API int q4gemv_set_fault(q4gemv_t h, const char* which);

#ifdef __cplusplus
}
#endif

#endif /* Q4GEMV_H */
