// Linear attention with decay over prompts on the 5th-generation tensor cores,
// 128 tokens at a time.  With b_i the sum of the log decays of a chunk's tokens
// up to i,
//   o_i = e^{b_i} q_i S + sum_{j <= i} e^{b_i - b_j} (q_i . k_j) v_j,
//   S'  = e^{b_C} S + sum_j e^{b_C - b_j} k_j v_j^T,
// a chunk is four products with all accumulators in tensor memory: the scores
// Q K^T, the part of the outputs from the state, the part from the chunk, and
// what the state gains (the state stays there, as S^T: a value column a lane).
//   warps 0-15 the passes between the products, a thread a quarter row: the state
//              to a 16-bit operand in shared memory and times its decay in
//              place; the scores times their decays, to the 16-bit operand in
//              their own place; the decayed keys k' = e^{b_C - b_j} k_j split
//              into 16-bit parts; values looked over; outputs out
//   warp 16    one thread issues the products
//   warp 17    one thread loads Q, K and V by tensor map, K a chunk ahead
//   warp 18    sums of the log decays, a chunk ahead
//   warp 19    the largest key of a chunk, a chunk ahead
// What bounds it: the passes between the products, 16 warps one after the
// other over 5 x 16384 values of a chunk: of its 4.5 us (f16, 40 heads of 128 x
// 128) the keys take 0.7, the state 1.0, the scores 0.9, the values 0.3, the
// outputs 0.8, and barriers and latencies the rest; the products alone are 2560
// cycles.  Outputs of whole chunks leave by tensor map (with stores by the
// passes: 9 % more).  Measured: three prompts of up to 16384 tokens 576 us (bf16
// 606), one of 8192 187 us, 115 TFLOP/s of the recurrence's products.
//
// Number formats.  State and sums are in 32 bits.  The split keys carry 22
// (binary16: two parts) or 24 (bfloat16: three) significant bits into the
// state; one part alone would leave it with 11 or 8.  The state's and the
// scores' operands of the output products are rounded once to the type, as the
// output itself is.  In binary16 powers of two keep them inside its range: of
// the chunk's largest key, of the state's largest value in a column, of a row's
// largest score.  Sums of log decays are in 64 bits (differences of far-apart
// sums).  A value that is not finite must not meet the zero weight of an
// earlier token: it is replaced by zero for the products, and the outputs and
// state columns that it does reach are set to NaN.
//
// Long sequences run as parallel segments (lin_seg.cuh).
#pragma once

#include <cuda.h>

#include "lin_seg.cuh"
#include "mma_common.cuh"
#include "tc_common.cuh"

namespace q4 {

constexpr int kLtTokens = 128;
constexpr int kLtPass = 512;                         // threads of the passes
constexpr int kLtParts = kLtPass / kLtTokens;        // threads of a row
constexpr int kLtThreads = kLtPass + 32 * 4;
constexpr uint32_t kLtHalf = kLtTokens * 128;        // [128 rows][64 elements]
constexpr int kLtDec = 4 * kLtTokens + 4;            // floats of a chunk's decays

__host__ __device__ constexpr int lt_kbytes(int dk) { return kLtTokens * dk * 2; }
// Two K's, the keys' second part, V, Q (or their third part), the state's operand,
// in whose place the outputs are laid in rows.
__host__ __device__ constexpr int lt_smem(int dk, bool out) {
    return 1024 + 4 * lt_kbytes(dk) + (out ? 4 : 2) * (int)kLtHalf + 2 * kLtDec * 4 +
           (2 * kLtParts * 128 + 128 + 2 * 128 + 32) * 4 + 256;
}

struct LinTcArgs {
    LinSegArgs g;
    uint32_t idesc_a, idesc_i, idesc_o, idesc_s;     // of the four products
    CUtensorMap qmap, kmap, vmap, omap;              // [row][head][element], boxes of 64 elements x 128 rows
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
                 : "memory");
}

// A box from shared memory, in this thread's next group of stores.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// This thread's stores have left shared memory; have been written.
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Sums of a chunk's log decays by one warp, four tokens a lane, in units of
// log2: [128] b_i high parts, [128] low parts, [128] e^{b_i}, [128] e^{b_C -
// b_i}, e^{b_C}, b_C.  Under -104 a decay is zero in 32 bits; padding tokens do
// not decay.
__device__ __forceinline__ void lt_decays(float4 g, float* out) {
    const int lane = threadIdx.x & 31;
    double b[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (b[i] < -104.0) b[i] = -104.0;
        if (i) b[i] += b[i - 1];
    }
    double p = b[3];
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(0xFFFFFFFFu, p, d);
        if (lane >= d) p += y;
    }
    const double before = p - b[3], all = __shfl_sync(0xFFFFFFFFu, p, 31);
    float hi[4], lo[4], e[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double x = b[i] + before, x2 = x * 1.4426950408889634074;
        hi[i] = (float)x2;
        lo[i] = (float)(x2 - hi[i]);
        e[i] = expf((float)x);
        w[i] = expf((float)(all - x));
    }
    float4* o = reinterpret_cast<float4*>(out) + lane;
    o[0] = make_float4(hi[0], hi[1], hi[2], hi[3]);
    o[32] = make_float4(lo[0], lo[1], lo[2], lo[3]);
    o[64] = make_float4(e[0], e[1], e[2], e[3]);
    o[96] = make_float4(w[0], w[1], w[2], w[3]);
    if (lane == 0) {
        out[4 * kLtTokens] = expf((float)all);
        out[4 * kLtTokens + 1] = (float)all;
    }
}

// max(m, |v.x|, |v.y|); a NaN is passed over.
__device__ __forceinline__ float max_abs(float m, float2 v) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(v.x), "f"(v.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

template <typename T, int DK, bool OUT>
__global__ void __launch_bounds__(kLtThreads, 1) lin_tc_kernel(const __grid_constant__ LinTcArgs ta) {
    constexpr bool kHalf16 = Elem<T>::kExpMask == Elem<__half>::kExpMask;
    constexpr bool kAhead = OUT && kHalf16;              // the largest keys come from warp 19
    constexpr int C = kLtTokens;
    constexpr uint32_t KB = lt_kbytes(DK);
    constexpr int CW = DK / kLtParts;                    // state columns of a thread: 32 or 16
    constexpr uint32_t kColA = 128, kColI = 256, kColO = 384;   // TMEM: state at 0, scores, outputs' two parts
    extern __shared__ uint8_t lt_raw[];
    const LinSegArgs& g = ta.g;
    const LinArgs& a = g.a;
    const uint32_t raw0 = smem_addr(lt_raw);
    const uint32_t sK = (raw0 + 1023u) & ~1023u;         // two
    const uint32_t sX = sK + 2 * KB;                     // the keys' second part
    const uint32_t sV = sX + KB;
    const uint32_t sQ = sV + 2 * kLtHalf;                // with OUT; the third part (bfloat16) in its place, or after V
    const uint32_t sS = sQ + KB;                         // the state's operand, with OUT
    float* fl = reinterpret_cast<float*>(lt_raw + (sS + (OUT ? 2 * kLtHalf : 0) - raw0));
    float* sx = fl + 2 * kLtDec;                         // [parts][128] row maxima: state, scores
    float* sy = sx + kLtParts * 128;
    float* colf = sy + kLtParts * 128;                              // [128] scale of a value column of the state's operand
    volatile int* badc = reinterpret_cast<volatile int*>(colf + 128);   // [2][128] first token with a bad value, or 128
    uint32_t* sMax = reinterpret_cast<uint32_t*>(colf + 384);           // [16] largest |k|: of two chunks, or of the warps' parts
    volatile int* any_bad = reinterpret_cast<volatile int*>(sMax + 16); // [2]
    volatile int* abort_flag = any_bad + 2;
    volatile int* never = any_bad + 3;
    uint32_t* tslot = sMax + 20;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sMax + 32);
    uint64_t *kfull = bars, *qfull = bars + 2, *vfull = bars + 3, *dfull = bars + 4, *dfree = bars + 6, *qkdone = bars + 8,
             *qfree = bars + 9, *odone = bars + 10, *kvdone = bars + 11, *sready = bars + 12, *pready = bars + 13,
             *kready = bars + 14, *oread = bars + 15, *idle = bars + 16, *kmax = bars + 17;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull + i, 1);
            mbar_init(dfull + i, 1);
            mbar_init(kmax + i, 1);
            mbar_init(dfree + i, kLtPass / 32);
            any_bad[i] = 0;
        }
        for (uint64_t* b : {qfull, vfull, qkdone, qfree, odone, kvdone, idle}) mbar_init(b, 1);
        for (uint64_t* b : {sready, pready, kready, oread}) mbar_init(b, kLtPass / 32);
        *abort_flag = *never = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < 256) badc[threadIdx.x] = C;
    if (warp == 16) tc_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    pdl_wait();
    pdl_launch_dependents();

    const int h = blockIdx.x, c0 = blockIdx.y * 128;
    const int s = blockIdx.z / g.segs, seg = blockIdx.z - s * g.segs;
    const int slot = a.slots ? a.slots[s] : s;
    const bool bad_slot = (unsigned)slot >= (unsigned)a.n_slots;
    if (bad_slot && threadIdx.x == 0) set_device_error(a.err, kDevIndex);
    int64_t t0 = 0, t1 = 0;
    bool last = false;
    if (!bad_slot) segment(g, s, seg, t0, t1, last);
    const bool work = !bad_slot && (OUT ? t0 < t1 || last : t0 < t1 && !last);
    const int nc = work ? (int)((t1 - t0 + C - 1) / C) : 0;
    const int hk = h / a.each;
    auto give_up = [&]() {
        *abort_flag = 1;
        set_device_error(a.err, kDevTimeout);
    };

    if (warp == 17) {
        // ---- loads ----
        if (lane == 0) {
            bool ok = true;
            int nk = 0, nq = 0, nv = 0;                  // loads begun
            for (int c = 0; c < nc && ok; ++c) {
                const int t = (int)(t0 + (int64_t)c * C);
                // K's buffer was chunk c - 2's, whose last product was waited for below.
                mbar_arrive_expect_tx(kfull + (c & 1), KB);
                for (int i = 0; i < DK / 64; ++i)
                    tma_load_3d(sK + (c & 1) * KB + i * kLtHalf, &ta.kmap, 64 * i, hk, t, kfull + (c & 1));
                ++nk;
                if (OUT && kHalf16) {
                    if (c > 0) ok = tc_wait_long(qfree, (c - 1) & 1, abort_flag);
                    if (!ok) break;
                    mbar_arrive_expect_tx(qfull, KB);
                    for (int i = 0; i < DK / 64; ++i) tma_load_3d(sQ + i * kLtHalf, &ta.qmap, 64 * i, hk, t, qfull);
                    ++nq;
                }
                if (c > 0) ok = tc_wait_long(kvdone, (c - 1) & 1, abort_flag);
                if (!ok) break;
                if (OUT && !kHalf16) {
                    mbar_arrive_expect_tx(qfull, KB);
                    for (int i = 0; i < DK / 64; ++i) tma_load_3d(sQ + i * kLtHalf, &ta.qmap, 64 * i, hk, t, qfull);
                    ++nq;
                }
                mbar_arrive_expect_tx(vfull, 2 * kLtHalf);
                for (int i = 0; i < 2; ++i) tma_load_3d(sV + i * kLtHalf, &ta.vmap, c0 + 64 * i, h, t, vfull);
                ++nv;
            }
            if (!ok) give_up();
            // Copies in flight land before the CTA ends (in vain only after a
            // wait that gave up).
            for (int i = 0; i < 2; ++i)
                if (nk > i) tc_wait_long(kfull + i, ((nk + 1 - i) / 2 - 1) & 1, never);
            if (nq > 0) tc_wait_long(qfull, (nq - 1) & 1, never);
            if (nv > 0) tc_wait_long(vfull, (nv - 1) & 1, never);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ---- decays ----
        double total = 0;
        bool ok = true;
        const float* gb = a.g + h;
        auto load = [&](int c) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = t0 + (int64_t)c * C + 4 * lane + i;
                v[i] = c < nc && t < t1 ? gb[t * a.g_stride] : 0.f;
            }
            return make_float4(v[0], v[1], v[2], v[3]);
        };
        float4 next = load(0);
        for (int c = 0; c < nc; ++c) {
            const float4 now = next;
            next = load(c + 1);
            if (c >= 2) ok = __all_sync(0xFFFFFFFFu, tc_wait_long(dfree + (c & 1), ((c >> 1) - 1) & 1, abort_flag));
            if (!ok) break;
            float* d = fl + (c & 1) * kLtDec;
            lt_decays(now, d);
            __syncwarp();
            total += d[4 * C + 1];
            if (lane == 0) mbar_arrive(dfull + (c & 1));
        }
        if (!ok) give_up();
        if (!OUT && work && lane == 0 && blockIdx.y == 0) *seg_decay(g, s, h, seg) = expf((float)total);
    } else if (warp == 19) {
        // ---- the chunks' largest keys, a chunk ahead (with OUT: without the
        // outputs a chunk is too short for one warp, and the passes look) ----
        if (kAhead) {
            bool ok = true;
            for (int c = 0; c < nc; ++c) {
                ok = __all_sync(0xFFFFFFFFu, tc_wait_long(kfull + (c & 1), (c >> 1) & 1, abort_flag));
                if (!ok) break;
                const int n = (int)min((int64_t)C, t1 - t0 - (int64_t)c * C);
                uint32_t m = 0;
#pragma unroll 1
                for (int x0 = lane; x0 < (int)KB / 16; x0 += 512) {
                    uint4 v[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) v[y] = lds128(sK + (c & 1) * KB + 16u * (x0 + 32 * y));
#pragma unroll
                    for (int y = 0; y < 16; ++y) m = __vmaxu2(m, (((x0 + 32 * y) >> 3) & 127) < n ? max_abs8(0u, v[y]) : 0u);
                }
                for (int x = 16; x; x >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                // The passes have read the last but one: its keys were freed
                // after them.
                if (lane == 0) {
                    sMax[c & 1] = max(m & 0xFFFFu, m >> 16);
                    mbar_arrive(kmax + (c & 1));
                }
                __syncwarp();
            }
            if (!ok) give_up();
        }
    } else if (warp == 16) {
        // ---- products ----
        if (lane == 0) {
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t par) {
                if (ok && !tc_wait_long(bar, par & 1, abort_flag)) ok = false;
                tc_fence_after();
                return ok;
            };
            for (int c = 0; c < nc && ok; ++c) {
                const uint32_t k = sK + (c & 1) * KB;
                if (OUT) {
                    wait(kfull + (c & 1), c >> 1);
                    if (!wait(qfull, c)) break;
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint32_t o = (uint32_t)(kk >> 2) * kLtHalf + 32u * (kk & 3);
                        tc_mma_f16(tmem + kColA, tc_sdesc_sw128(sQ + o), tc_sdesc_sw128(k + o), ta.idesc_a, kk != 0);
                    }
                    tc_commit(qkdone);
                    wait(sready, c);
                    if (c > 0) wait(oread, c - 1);
                    if (!ok) break;
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint32_t o = (uint32_t)(kk >> 2) * kLtHalf + 32u * (kk & 3);
                        tc_mma_f16(tmem + kColI, tc_sdesc_sw128(sQ + o), tc_sdesc_sw128(sS + o), ta.idesc_i, kk != 0);
                    }
                    tc_commit(qfree);
                    wait(vfull, c);
                    if (!wait(pready, c)) break;
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        tc_mma_f16_ta(tmem + kColO, tmem + kColA + 8u * kk, tc_sdesc_sw128_nmajor(sV + 2048u * kk, kLtHalf),
                                      ta.idesc_o, kk != 0);
                    tc_commit(odone);
                }
                wait(vfull, c);
                if (!wait(kready, c)) break;
                const uint32_t parts[3] = {k, sX, sQ};
#pragma unroll
                for (int p = 0; p < (kHalf16 ? 2 : 3); ++p)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk)
                        tc_mma_f16(tmem, tc_sdesc_sw128_nmajor(sV + 2048u * kk, kLtHalf),
                                   tc_sdesc_sw128_nmajor(parts[p] + 2048u * kk, kLtHalf), ta.idesc_s, 1u);
                tc_commit(kvdone);
            }
            if (!ok) give_up();
            tc_commit(idle);
            tc_wait_long(idle, 0, never);
        }
        __syncwarp();
    } else if (warp < 16 && work) {
        // ---- passes: lane quadrant warp % 4, column part warp / 4 ----
        const int row = 32 * (warp & 3) + lane, hc = warp >> 2, tid = threadIdx.x;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + (uint32_t)(hc * CW);
        const bool real = c0 + row < a.v_dim;            // this thread's value column, in the state's passes
        const int64_t so = ((int64_t)slot * a.v_heads + h) * a.k_dim * a.v_dim;
        const float* from = !OUT ? nullptr : g.segs > 1 ? seg_state(g, s, h, seg) : a.state_in ? a.state_in + so : nullptr;
        float* to = OUT ? (last ? a.state_out + so : nullptr) : seg_state(g, s, h, seg);
        if (from) from += c0 + row;
        if (to) to += c0 + row;
        auto load_state = [&](uint32_t (&v)[CW]) {
            if constexpr (CW == 32) tc_ld32(tS, reinterpret_cast<float(&)[32]>(v));
            else tc_ld16(tS, v);
            if constexpr (CW == 32) tc_wait_ld(reinterpret_cast<float(&)[32]>(v));
        };
        auto store_state = [&](const uint32_t (&v)[CW]) {
            if constexpr (CW == 32) tc_st32(tS, v);
            else tc_st16(tS, v);
        };
        // The first state.
        {
            uint32_t v[CW];
#pragma unroll
            for (int y = 0; y < CW; ++y)
                v[y] = from && real && hc * CW + y < a.k_dim ? __float_as_uint(from[(int64_t)(hc * CW + y) * a.v_dim]) : 0u;
            store_state(v);
            tc_wait_st();
            if (nc == 0 && to && real)
#pragma unroll
                for (int y = 0; y < CW; ++y)
                    if (hc * CW + y < a.k_dim) to[(int64_t)(hc * CW + y) * a.v_dim] = __uint_as_float(v[y]);
        }
        int E = 0;                                       // TMEM holds the state times 2^E
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t par) {
            if (ok && !tc_wait_long(bar, par & 1, abort_flag)) ok = false;
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) give_up();
        };
        auto tell = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        T* ob = static_cast<T*>(a.out) + (int64_t)h * a.v_dim + c0;
        auto bar = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kLtPass) : "memory"); };
        for (int c = 0; c < nc; ++c) {
            const int64_t t = t0 + (int64_t)c * C;
            const int n = (int)min((int64_t)C, t1 - t);
            const uint32_t k = sK + (c & 1) * KB;
            const float* dec = fl + (c & 1) * kLtDec;
            const int bad_now = 128 * (c & 1), bad_then = 128 * ((c & 1) ^ 1);

            // The chunk's largest key, and the common end after a wait that gave up.
            wait(kAhead ? kmax + (c & 1) : kfull + (c & 1), c >> 1);
            if (kHalf16 && !kAhead) {
                uint32_t m = 0;
#pragma unroll 4
                for (int x = tid; x < (int)KB / 16; x += kLtPass)
                    if (((x >> 3) & 127) < n) m = max_abs8(m, lds128(k + 16u * x));
                for (int x = 16; x; x >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                if (lane == 0) sMax[warp] = max(m & 0xFFFFu, m >> 16);
            }
            wait(dfull + (c & 1), c >> 1);
            if (!all_of<kLtPass>(ok)) break;
            int sk = 0;
            if (kHalf16) {
                uint32_t top = *reinterpret_cast<volatile uint32_t*>(sMax + (kAhead ? c & 1 : 0));
                if (!kAhead)
#pragma unroll
                    for (int y = 1; y < kLtPass / 32; ++y) top = max(top, sMax[y]);
                // The largest to [2^14, 2^15); with infinities or NaN, what suits any finite key.
                sk = top >= Elem<__half>::kExpMask ? -2
                                                   : to_2_14(__half2float(__ushort_as_half((unsigned short)top)), 24);
            }

            // The state: its operand, and its decay.
            if (c > 0) wait(kvdone, c - 1);
            tc_fence_after();
            const bool spoilt = any_bad[(c & 1) ^ 1] && badc[bad_then + row] < C;   // by the last chunk's values
            const float decay = dec[4 * C], f1 = exp2i(sk - E);
            float rp = 1.f;
            uint32_t sv[CW];
            load_state(sv);
            if (spoilt)
#pragma unroll
                for (int y = 0; y < CW; ++y) sv[y] = 0x7FFFFFFFu;
            auto pair = [&](int y) { return make_float2(__uint_as_float(sv[y]), __uint_as_float(sv[y + 1])); };
            if (OUT && kHalf16) {
                float m = 0.f;
#pragma unroll
                for (int y = 0; y < CW; y += 2) m = max_abs(m, pair(y));
                sx[128 * hc + row] = m;
            }
            if (OUT && tid == 0) tma_store_read();           // the operand's place is free of the last outputs
            bar();
            if (OUT && kHalf16) {
                float m = sx[row];
#pragma unroll
                for (int y = 1; y < kLtParts; ++y) m = fmaxf(m, sx[128 * y + row]);
                const int e = (__float_as_int(m) >> 23) - 127;
                const int rs = m == 0.f || e > 127 ? 0 : min(126, 14 - e);
                rp = exp2i(rs);
                if (hc == 0) colf[row] = exp2i(-rs - E);
            } else if (OUT && hc == 0) {
                colf[row] = 1.f;
            }
            if (hc == 0 && spoilt) badc[bad_then + row] = C;
            if (tid == 0) any_bad[(c & 1) ^ 1] = 0;
            if (OUT) {
#pragma unroll
                for (int x = 0; x < CW / 8; ++x) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float2 v = fmul2(pair(8 * x + 2 * y), both(rp));
                        w[y] = Elem<T>::pack(v.x, v.y);
                    }
                    const int ch = hc * (CW / 8) + x;    // 16-byte chunk of the row
                    sts128(sS + (uint32_t)(ch >> 3) * kLtHalf + (uint32_t)(row * 128 + (((ch & 7) ^ (row & 7)) << 4)),
                           make_uint4(w[0], w[1], w[2], w[3]));
                }
                fence_proxy_async_smem();
            }
#pragma unroll
            for (int y = 0; y < CW; y += 2) {
                const float2 v = fmul2(fmul2(pair(y), both(decay)), both(f1));
                sv[y] = __float_as_uint(v.x);
                sv[y + 1] = __float_as_uint(v.y);
            }
            store_state(sv);
            tc_wait_st();
            tc_fence_before();
            E = sk;
            tell(sready);

            // Values: rows behind the chunk's tokens to zero, and those that
            // are not finite, which are remembered.  They come after the last
            // chunk's products, in bfloat16 with the queries, so there is time
            // for the scores first where the queries are early.
            auto look_over = [&]() {
                wait(vfull, c);
                constexpr int N = (int)(2 * kLtHalf / 16) / kLtPass;
                uint32_t top = 0;
#pragma unroll
                for (int x = 0; x < N; ++x) top = max_abs8(top, lds128(sV + 16u * (tid + x * kLtPass)));
                if (n < C || (top & 0xFFFFu) >= Elem<T>::kExpMask || top >> 16 >= Elem<T>::kExpMask) {
                    for (int x = tid; x < (int)(2 * kLtHalf / 16); x += kLtPass) {
                        const int r = (x >> 3) & 127;
                        const uint4 v = lds128(sV + 16u * x);
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        if (r >= n) {
                            w[0] = w[1] = w[2] = w[3] = 0;
                        } else if (any_nonfinite<T>(v)) {
                            const int col = 64 * (x >> 10) + 8 * ((x & 7) ^ (r & 7));
#pragma unroll
                            for (int y = 0; y < 8; ++y)
                                if (((w[y >> 1] >> (16 * (y & 1))) & Elem<T>::kExpMask) == Elem<T>::kExpMask) {
                                    w[y >> 1] &= y & 1 ? 0xFFFFu : 0xFFFF0000u;
                                    atomicMin(const_cast<int*>(badc) + bad_now + col + y, r);
                                }
                            any_bad[c & 1] = 1;
                        }
                        sts128(sV + 16u * x, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                    fence_proxy_async_smem();
                }
            };
            if (!kHalf16 && OUT) look_over();

            float rowf = 1.f;
            if (OUT) {
                // Scores with their decays.
                wait(qkdone, c);
                tc_fence_after();
                float p[32];
                tc_ld32(tmem + lanes + kColA + 32u * hc, p);
                tc_wait_ld(p);
                float m = 0.f;
                if (hc <= (warp & 3)) {                  // else wholly above the diagonal
                    const float2 bh = both(dec[row]), bl = both(dec[C + row]), less = both(-1.f);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const float4 h4 = *reinterpret_cast<const float4*>(dec + 32 * hc + 4 * x);
                        const float4 l4 = *reinterpret_cast<const float4*>(dec + C + 32 * hc + 4 * x);
                        const float2 hj[2] = {make_float2(h4.x, h4.y), make_float2(h4.z, h4.w)};
                        const float2 lj[2] = {make_float2(l4.x, l4.y), make_float2(l4.z, l4.w)};
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float2 d = fadd2(ffma2(hj[y], less, bh), ffma2(lj[y], less, bl));
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d.x) : "f"(d.x));
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d.y) : "f"(d.y));
                            const int at = 4 * x + 2 * y;
                            const float2 v = fmul2(make_float2(p[at], p[at + 1]), d);
                            p[at] = v.x;
                            p[at + 1] = v.y;
                        }
                    }
                    if (hc == (warp & 3)) {              // on the diagonal
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            if (y > lane) p[y] = 0.f;
                    }
                    if (kHalf16)
#pragma unroll
                        for (int y = 0; y < 32; y += 2) m = max_abs(m, make_float2(p[y], p[y + 1]));
                } else {
#pragma unroll
                    for (int y = 0; y < 32; ++y) p[y] = 0.f;
                }
                float tp = 1.f;
                if (kHalf16) sy[128 * hc + row] = m;
                bar();                                   // a row's parts are read: the operand may go there
                if (kHalf16) {
                    m = sy[row];
#pragma unroll
                    for (int y = 1; y < kLtParts; ++y) m = fmaxf(m, sy[128 * y + row]);
                    const int e = (__float_as_int(m) >> 23) - 127;
                    const int rs = m == 0.f || e > 127 ? 0 : max(-126, min(126, 14 - e));
                    tp = exp2i(rs);
                    rowf = exp2i(-rs);
                }
                uint32_t w[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                    const float2 v = fmul2(make_float2(p[2 * y], p[2 * y + 1]), both(tp));
                    w[y] = Elem<T>::pack(v.x, v.y);
                }
                tc_st16(tmem + lanes + kColA + 16u * hc, w);
            }

            if (kHalf16 || !OUT) look_over();
            if (OUT) {
                tc_wait_st();
                tc_fence_before();
                tell(pready);
                if (!kHalf16) wait(qfree, c);            // Q's place is the third part's
            }

            // The decayed keys in parts, the first in the keys' own place.
            if (kAhead) wait(kfull + (c & 1), c >> 1);
            {
                const float pk = exp2i(sk);
#pragma unroll 2
                for (int x = tid; x < (int)KB / 16; x += kLtPass) {
                    const int r = (x >> 3) & 127;
                    const float w = dec[3 * C + r] * pk;
                    const uint4 kv = r < n ? lds128(k + 16u * x) : make_uint4(0, 0, 0, 0);
                    const uint32_t kw[4] = {kv.x, kv.y, kv.z, kv.w};
                    const float2 less = both(-1.f);
                    uint32_t p0[4], p1[4], p2[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float2 f = fmul2(Elem<T>::unpack(kw[y]), both(w));
                        p0[y] = Elem<T>::pack(f.x, f.y);
                        f = ffma2(Elem<T>::unpack(p0[y]), less, f);      // exact: what the part left
                        p1[y] = Elem<T>::pack(f.x, f.y);
                        if (!kHalf16) {
                            f = ffma2(Elem<T>::unpack(p1[y]), less, f);
                            p2[y] = Elem<T>::pack(f.x, f.y);
                        }
                    }
                    sts128(k + 16u * x, make_uint4(p0[0], p0[1], p0[2], p0[3]));
                    sts128(sX + 16u * x, make_uint4(p1[0], p1[1], p1[2], p1[3]));
                    if (!kHalf16) sts128(sQ + 16u * x, make_uint4(p2[0], p2[1], p2[2], p2[3]));
                }
                fence_proxy_async_smem();
                tell(kready);
            }

            if (OUT) {
                // Outputs.
                const float eb = dec[2 * C + row] * a.scale;
                rowf *= a.scale;
                wait(odone, c);
                tc_fence_after();
                const bool bad = any_bad[c & 1] != 0;
                // Into rows in the state operand's place, then out.
                {
                    float vi[32], vo[32];
                    tc_ld32(tmem + lanes + kColI + 32u * hc, vi);
                    tc_ld32(tmem + lanes + kColO + 32u * hc, vo);
                    tc_wait_ld(vi);
                    tc_wait_ld(vo);
                    tc_fence_before();
                    tell(oread);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float v[8];
                        const float4 f0 = *reinterpret_cast<const float4*>(colf + 32 * hc + 8 * y);
                        const float4 f4 = *reinterpret_cast<const float4*>(colf + 32 * hc + 8 * y + 4);
                        const float2 cf[4] = {make_float2(f0.x, f0.y), make_float2(f0.z, f0.w), make_float2(f4.x, f4.y),
                                              make_float2(f4.z, f4.w)};
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const int at = 8 * y + 2 * z;
                            const float2 u = fmul2(make_float2(vi[at], vi[at + 1]), cf[z]);
                            const float2 t = ffma2(u, both(eb), fmul2(make_float2(vo[at], vo[at + 1]), both(rowf)));
                            v[2 * z] = t.x;
                            v[2 * z + 1] = t.y;
                        }
                        if (bad)
#pragma unroll
                            for (int z = 0; z < 8; ++z)
                                if (badc[bad_now + 32 * hc + 8 * y + z] <= row) v[z] = __int_as_float(0x7FFFFFFF);
                        const int ch = 4 * hc + y;
                        sts128(sS + (uint32_t)(ch >> 3) * kLtHalf + (uint32_t)(row * 128 + (((ch & 7) ^ (row & 7)) << 4)),
                               pack8<T>(v));
                    }
                }
                if (n == C) {                            // a whole box
                    fence_proxy_async_smem();
                    bar();
                    if (tid == 0) {
                        for (int i = 0; i < 2; ++i)
                            if (c0 + 64 * i < a.v_dim) tma_store_3d(&ta.omap, sS + i * kLtHalf, c0 + 64 * i, h, (int)t);
                        tma_store_commit();
                    }
                } else {
                    bar();
#pragma unroll
                    for (int x = 0; x < C * 16 / kLtPass; ++x) {
                        const int r = (tid >> 4) + x * (kLtPass / 16), ch = tid & 15;
                        const uint4 v =
                            lds128(sS + (uint32_t)(ch >> 3) * kLtHalf + (uint32_t)(r * 128 + (((ch & 7) ^ (r & 7)) << 4)));
                        if (r < n && c0 + 8 * ch < a.v_dim) *reinterpret_cast<uint4*>(ob + (t + r) * a.o_stride + 8 * ch) = v;
                    }
                }
            }
            tell(dfree + (c & 1));
        }

        if (OUT && tid == 0) tma_store_done();

        // The last state.
        if (ok && nc > 0 && to) {
            wait(kvdone, nc - 1);
            tc_fence_after();
            const bool spoilt = any_bad[(nc - 1) & 1] && badc[128 * ((nc - 1) & 1) + row] < C;
            const float un = exp2i(-E);
            uint32_t v[CW];
            load_state(v);
#pragma unroll
            for (int y = 0; y < CW; ++y)
                if (real && hc * CW + y < a.k_dim)
                    to[(int64_t)(hc * CW + y) * a.v_dim] = spoilt ? __int_as_float(0x7FFFFFFF) : __uint_as_float(v[y]) * un;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

}  // namespace q4
