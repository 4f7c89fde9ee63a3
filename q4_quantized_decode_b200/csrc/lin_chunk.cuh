// Linear attention with decay over prompts, 64 tokens at a time on the tensor
// cores.  With b_i the sum of the log decays of a chunk's tokens up to i,
//   o_i = e^{b_i} S^T q_i + sum_{j <= i} e^{b_i - b_j} (q_i . k_j) v_j,
//   S'  = e^{b_C} S + sum_j e^{b_C - b_j} k_j v_j^T,
// so a chunk is four matrix products.  They are taken transposed, O^T = S^T Q^T
// + V^T A^T and S'^T = V^T K', because then a warp's accumulators of S^T (its
// 16 or 32 value columns as rows, all of k_dim as columns) are, register for
// register, the A operand of the next chunk's first product: the state never
// leaves the registers from the sequence's first token to its last.
//
// Number formats.  The state and all sums are in 32 bits.  Products run in
// binary16 (bfloat16 inputs are converted, exactly up to values 2^28 under the
// chunk's largest).  The decayed keys k' = e^{b_C - b_j} k_j are split into two
// binary16 parts, so what the state gains has 22 significant bits: one part
// alone would leave the state with binary16's 11.  The state's and the scores'
// operand of the output products are rounded to binary16 once, because the
// output is rounded to 16 bits itself.  Powers of two, taken from the chunk's
// largest magnitudes and the state rows', keep all of that inside binary16's
// range.  Sums of log decays are in 64 bits (differences of far-apart sums).
// (The state's unit is at most 2^40, so states up to 2^87 fit.)
// A chunk with infinities, NaN or magnitudes from 2^30 on is run token by token
// on the same registers instead, where a zero weight touches nothing.
#pragma once

#include "linattn.cuh"
#include "mma_common.cuh"

namespace q4 {

constexpr int kLcTokens = 64;
constexpr int kLcWarps = 4;
constexpr int kLcThreads = 32 * kLcWarps;

// Value columns of a CTA: 16 MT for each warp.
__host__ __device__ constexpr int lc_cols(int mt) { return 16 * mt * kLcWarps; }
__host__ __device__ constexpr int lc_qbytes(int dk, int mt) {        // Q, later the chunk's outputs
    return kLcTokens * 2 * (dk > lc_cols(mt) ? dk : lc_cols(mt));
}
__host__ __device__ constexpr int lc_smem(int dk, int mt) {
    return lc_qbytes(dk, mt) + 3 * kLcTokens * dk * 2 + kLcTokens * lc_cols(mt) * 2 + kLcTokens * kLcTokens * 2 +
           (4 * kLcTokens + 32) * 4;
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

__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {   // a: running, b: two 16-bit floats
    return __vmaxu2(a, b & 0x7FFF7FFFu);
}

// Two 16-bit values times a power of two, as binary16.
template <typename T>
__device__ __forceinline__ uint32_t to_half2(uint32_t v, float pw) {
    const float2 f = Elem<T>::unpack(v);
    return Elem<__half>::pack(f.x * pw, f.y * pw);
}

template <typename T, int DK, int MT>
__global__ void __launch_bounds__(kLcThreads, DK * MT <= 256 && DK <= 128 ? 2 : 1) lin_chunk_kernel(const LinArgs a) {
    constexpr bool kConvert = Elem<T>::kExpMask != Elem<__half>::kExpMask;   // bfloat16 inputs
    constexpr int C = kLcTokens;
    constexpr int DVS = lc_cols(MT);
    constexpr int KB = DK * 2, VB = DVS * 2;             // row bytes
    constexpr int NK = DK / 8;                           // 8-column tiles of the state
    extern __shared__ __align__(128) uint8_t lc_raw[];
    const uint32_t sQ = smem_addr(lc_raw);
    const uint32_t sK = sQ + lc_qbytes(DK, MT), sHi = sK + C * KB, sLo = sHi + C * KB, sV = sLo + C * KB,
                   sA = sV + C * VB;
    float* fl = reinterpret_cast<float*>(lc_raw + lc_smem(DK, MT) - (4 * C + 32) * 4);
    float* sBh = fl;              // b_i, high and low parts
    float* sBl = fl + C;
    float* sEb = fl + 2 * C;      // e^{b_i}
    float* sW = fl + 3 * C;       // e^{b_C - b_i}
    volatile float* sMisc = fl + 4 * C;                  // [0] e^{b_C}
    uint32_t* sMax = reinterpret_cast<uint32_t*>(fl + 4 * C + 4);   // [warp][3] largest |q|, |k|, |v|

    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, cc = lane & 3;
    const int h = blockIdx.x, c0 = blockIdx.y * DVS, s = blockIdx.z;
    const int slot = a.slots ? a.slots[s] : s;
    if ((unsigned)slot >= (unsigned)a.n_slots) {
        if (threadIdx.x == 0) set_device_error(a.err, kDevIndex);
        return;
    }
    int64_t t0 = a.start[s], t1 = a.start[s + 1];
    if (t0 < 0) t0 = 0;
    if (t1 > a.rows) t1 = a.rows;

    const T* qb = static_cast<const T*>(a.q) + (int64_t)(h / a.each) * a.k_dim;
    const T* kb = static_cast<const T*>(a.k) + (int64_t)(h / a.each) * a.k_dim;
    const T* vb = static_cast<const T*>(a.v) + (int64_t)h * a.v_dim + c0;
    T* ob = static_cast<T*>(a.out) + (int64_t)h * a.v_dim + c0;
    const float* gb = a.g + h;

    // The state: row warp * 16 MT + 16 mt + gr (+ 8) of its transpose, columns
    // 8 nk + 2 cc (+ 1).
    float S[MT][NK][4];
    const int64_t so = ((int64_t)slot * a.v_heads + h) * a.k_dim * a.v_dim;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nk = 0; nk < NK; ++nk)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int dv = c0 + (warp * MT + mt) * 16 + gr + 8 * (x >> 1), dk = 8 * nk + 2 * cc + (x & 1);
                S[mt][nk][x] = a.state_in && dv < a.v_dim && dk < a.k_dim
                                   ? a.state_in[so + (int64_t)dk * a.v_dim + dv] : 0.f;
            }
    int E = 0;                                           // S holds the state times 2^E

    for (int64_t t = t0; t < t1; t += C) {
        const int n = (int)(t1 - t < C ? t1 - t : C);
        for (int x = threadIdx.x; x < C * (DK / 8); x += kLcThreads) {
            const int r = x / (DK / 8), ch = x % (DK / 8);
            const bool in = r < n && 8 * ch < a.k_dim;
            const uint32_t dst = (uint32_t)(r * KB + ((ch ^ (r & 7)) << 4));
            cp_async16(sQ + dst, in ? qb + (t + r) * a.q_stride + 8 * ch : qb, in);
            cp_async16(sK + dst, in ? kb + (t + r) * a.k_stride + 8 * ch : kb, in);
        }
        for (int x = threadIdx.x; x < C * (DVS / 8); x += kLcThreads) {
            const int r = x / (DVS / 8), ch = x % (DVS / 8);
            const bool in = r < n && c0 + 8 * ch < a.v_dim;
            cp_async16(sV + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)), in ? vb + (t + r) * a.v_stride + 8 * ch : vb, in);
        }
        cp_async_commit();
        if (warp == 0) {
            // Sums of the log decays, two tokens a lane.  Under -104 a decay
            // is zero in 32 bits; padding tokens do not decay.
            double b0 = 0, b1 = 0;
            if (2 * lane < n) b0 = gb[(t + 2 * lane) * a.g_stride];
            if (2 * lane + 1 < n) b1 = gb[(t + 2 * lane + 1) * a.g_stride];
            if (b0 < -104.0) b0 = -104.0;
            if (b1 < -104.0) b1 = -104.0;
            b1 += b0;
            double p = b1;
            for (int d = 1; d < 32; d <<= 1) {
                const double y = __shfl_up_sync(0xFFFFFFFFu, p, d);
                if (lane >= d) p += y;
            }
            const double before = p - b1;                // exact enough: sums of 32-bit values in 64 bits
            b0 += before;
            b1 += before;
            const double all = __shfl_sync(0xFFFFFFFFu, p, 31);
            sBh[2 * lane] = (float)b0;
            sBh[2 * lane + 1] = (float)b1;
            sBl[2 * lane] = (float)(b0 - (float)b0);
            sBl[2 * lane + 1] = (float)(b1 - (float)b1);
            sEb[2 * lane] = expf((float)b0);
            sEb[2 * lane + 1] = expf((float)b1);
            sW[2 * lane] = expf((float)(all - b0));
            sW[2 * lane + 1] = expf((float)(all - b1));
            if (lane == 0) sMisc[0] = expf((float)all);
        }
        cp_async_wait<0>();
        __syncthreads();

        // Largest magnitudes of the chunk.
        {
            uint32_t mq = 0, mk = 0, mv = 0;
            for (int x = threadIdx.x; x < C * (DK / 8); x += kLcThreads) {
                const uint4 q = lds128(sQ + 16u * x), k = lds128(sK + 16u * x);
                mq = max_abs2(max_abs2(max_abs2(max_abs2(mq, q.x), q.y), q.z), q.w);
                mk = max_abs2(max_abs2(max_abs2(max_abs2(mk, k.x), k.y), k.z), k.w);
            }
            for (int x = threadIdx.x; x < C * (DVS / 8); x += kLcThreads) {
                const uint4 v = lds128(sV + 16u * x);
                mv = max_abs2(max_abs2(max_abs2(max_abs2(mv, v.x), v.y), v.z), v.w);
            }
            for (int x = 16; x; x >>= 1) {
                mq = __vmaxu2(mq, __shfl_xor_sync(0xFFFFFFFFu, mq, x));
                mk = __vmaxu2(mk, __shfl_xor_sync(0xFFFFFFFFu, mk, x));
                mv = __vmaxu2(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, x));
            }
            if (lane == 0) {
                sMax[3 * warp] = mq;
                sMax[3 * warp + 1] = mk;
                sMax[3 * warp + 2] = mv;
            }
        }
        __syncthreads();
        float big[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            uint32_t m = sMax[x];
#pragma unroll
            for (int y = 1; y < kLcWarps; ++y) m = __vmaxu2(m, sMax[3 * y + x]);
            const float2 f = Elem<T>::unpack(m);
            big[x] = fmaxf(f.x, f.y);
            if (!(f.x < 1073741824.f && f.y < 1073741824.f)) big[x] = INFINITY;        // NaN too
        }
        const float decay = sMisc[0];
        if (!(big[0] < INFINITY && big[1] < INFINITY && big[2] < INFINITY)) {
            // Token by token.
            const float un = exp2i(-E);
            E = 0;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nk = 0; nk < NK; ++nk)
#pragma unroll
                    for (int x = 0; x < 4; ++x) S[mt][nk][x] *= un;
            for (int r = 0; r < n; ++r) {
                const float d = expf(gb[(t + r) * a.g_stride]);
                float v[MT][2], o[MT][2];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int col = (warp * MT + mt) * 16 + gr + 8 * y;
                        uint32_t u;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u)
                                     : "r"(sV + (uint32_t)(r * VB + (((col >> 3) ^ (r & 7)) << 4) + ((col & 6) << 1))));
                        const float2 f = Elem<T>::unpack(u);
                        v[mt][y] = col & 1 ? f.y : f.x;
                        o[mt][y] = 0.f;
                    }
#pragma unroll
                for (int nk = 0; nk < NK; ++nk) {
                    uint32_t uq, uk;
                    const uint32_t at = (uint32_t)(r * KB + ((nk ^ (r & 7)) << 4) + 4 * cc);
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(uq) : "r"(sQ + at));
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(uk) : "r"(sK + at));
                    const float2 q = Elem<T>::unpack(uq), k = Elem<T>::unpack(uk);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            float& s0 = S[mt][nk][2 * y];
                            float& s1 = S[mt][nk][2 * y + 1];
                            s0 = fmaf(s0, d, k.x * v[mt][y]);
                            s1 = fmaf(s1, d, k.y * v[mt][y]);
                            if (8 * nk + 2 * cc < a.k_dim) {
                                o[mt][y] = fmaf(q.x * a.scale, s0, o[mt][y]);
                                o[mt][y] = fmaf(q.y * a.scale, s1, o[mt][y]);
                            }
                        }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float f = o[mt][y];
                        f += __shfl_xor_sync(0xFFFFFFFFu, f, 1);
                        f += __shfl_xor_sync(0xFFFFFFFFu, f, 2);
                        const int col = (warp * MT + mt) * 16 + gr + 8 * y;
                        if (cc == 0 && c0 + col < a.v_dim) ob[(t + r) * a.o_stride + col] = Elem<T>::round(f);
                    }
            }
            __syncthreads();
            continue;
        }

        // Powers: q, v (and k of the scores) times 2^sq, 2^sv (2^skk) in
        // binary16, the split keys times 2^sk, the scores times 2^-ta.
        const int sk = to_2_14(big[1], 24);
        const int sq = kConvert ? to_2_14(big[0], 24) : 0, sv = kConvert ? to_2_14(big[2], 16) : 0;
        const int skk = kConvert ? sk : 0;
        const float bound = (float)DK * (big[0] * exp2i(sq)) * (big[1] * exp2i(skk));   // of a score
        const int ta = bound == 0.f ? 0 : max(-100, (__float_as_int(bound) >> 23) - 127 - 14);
        {
            const float pk = exp2i(sk);
            for (int x = threadIdx.x; x < C * (DK / 8); x += kLcThreads) {
                const int r = x / (DK / 8);
                const uint4 k = lds128(sK + 16u * x);
                const float w = sW[r] * pk;
                const uint32_t kw[4] = {k.x, k.y, k.z, k.w};
                uint32_t hi[4], lo[4], kk[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float2 f = Elem<T>::unpack(kw[y]);
                    const float f0 = f.x * w, f1 = f.y * w;
                    hi[y] = Elem<__half>::pack(f0, f1);
                    const float2 hf = Elem<__half>::unpack(hi[y]);
                    lo[y] = Elem<__half>::pack(f0 - hf.x, f1 - hf.y);
                    if (kConvert) kk[y] = Elem<__half>::pack(f.x * pk, f.y * pk);
                }
                sts128(sHi + 16u * x, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                sts128(sLo + 16u * x, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                if (kConvert) {
                    sts128(sK + 16u * x, make_uint4(kk[0], kk[1], kk[2], kk[3]));
                    const uint4 q = lds128(sQ + 16u * x);
                    const float pq = exp2i(sq);
                    sts128(sQ + 16u * x, make_uint4(to_half2<T>(q.x, pq), to_half2<T>(q.y, pq), to_half2<T>(q.z, pq),
                                                    to_half2<T>(q.w, pq)));
                }
            }
            if (kConvert) {
                const float pv = exp2i(sv);
                for (int x = threadIdx.x; x < C * (DVS / 8); x += kLcThreads) {
                    const uint4 v = lds128(sV + 16u * x);
                    sts128(sV + 16u * x, make_uint4(to_half2<T>(v.x, pv), to_half2<T>(v.y, pv), to_half2<T>(v.z, pv),
                                                    to_half2<T>(v.w, pv)));
                }
            }
        }
        __syncthreads();

        // Scores of the ten 16 x 16 blocks on and under the diagonal, each
        // with its decays, as the transposed product's B operand [i][j].
        for (int blk = warp; blk < 10; blk += kLcWarps) {
            const int bi = blk == 0 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, bj = blk - bi * (bi + 1) / 2;
            if (16 * bi >= n) continue;
            float sc[2][4];
#pragma unroll
            for (int x = 0; x < 8; ++x) sc[x >> 2][x & 3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                uint32_t af[4], bf[4];
                const int ra = 16 * bi + (lane & 15), ca = 2 * kk + (lane >> 4);
                ldmatrix4(af, sQ + (uint32_t)(ra * KB + ((ca ^ (ra & 7)) << 4)));
                const int rb = 16 * bj + (lane & 7) + ((lane >> 4) << 3), cb = 2 * kk + ((lane >> 3) & 1);
                ldmatrix4(bf, sK + (uint32_t)(rb * KB + ((cb ^ (rb & 7)) << 4)));
                mma16816<__half>(sc[0], af, bf[0], bf[1]);
                mma16816<__half>(sc[1], af, bf[2], bf[3]);
            }
            const float pa = exp2i(-ta);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int i = 16 * bi + gr + 8 * r;
                const float bh = sBh[i], bl = sBl[i];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int j = 16 * bj + 8 * y + 2 * cc + x;
                        f[x] = j <= i ? sc[y][2 * r + x] * pa * __expf((bh - sBh[j]) + (bl - sBl[j])) : 0.f;
                    }
                    const uint32_t at = sA + (uint32_t)(i * (2 * C) + (((2 * bj + y) ^ (i & 7)) << 4) + 4 * cc);
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(Elem<__half>::pack(f[0], f[1])) : "memory");
                }
            }
        }

        // O^T = (S^T 2^row) Q^T, then brought to the scores' scale with the
        // decays e^{b_i}.
        float O[MT][C / 8][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < C / 8; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) O[mt][x][y] = 0.f;
        int rs[MT][2];
        float rp[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float m = 0.f;
#pragma unroll
                for (int nk = 0; nk < NK; ++nk) m = fmaxf(m, fmaxf(fabsf(S[mt][nk][2 * y]), fabsf(S[mt][nk][2 * y + 1])));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                const int e = (__float_as_int(m) >> 23) - 127;
                rs[mt][y] = m == 0.f || e > 127 ? 0 : min(126, 14 - e);
                rp[mt][y] = exp2i(rs[mt][y]);
            }
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk) {
            uint32_t af[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float* p = S[mt][2 * kk + (x >> 1)];
                    const float f = rp[mt][x & 1];
                    af[mt][x] = Elem<__half>::pack(p[2 * (x & 1)] * f, p[2 * (x & 1) + 1] * f);
                }
#pragma unroll
            for (int np = 0; np < C / 16; ++np) {
                uint32_t bf[4];
                const int rb = 16 * np + (lane & 7) + ((lane >> 4) << 3), cb = 2 * kk + ((lane >> 3) & 1);
                ldmatrix4(bf, sQ + (uint32_t)(rb * KB + ((cb ^ (rb & 7)) << 4)));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma16816<__half>(O[mt][2 * np], af[mt], bf[0], bf[1]);
                    mma16816<__half>(O[mt][2 * np + 1], af[mt], bf[2], bf[3]);
                }
            }
        }
        const int En = sk + sv;                          // the unit that this chunk's keys and values give
        {
            float rf[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int y = 0; y < 2; ++y) rf[mt][y] = exp2i(-rs[mt][y] - E + skk + sv - ta);
#pragma unroll
            for (int x = 0; x < C / 8; ++x) {
                const float2 eb = *reinterpret_cast<const float2*>(sEb + 8 * x + 2 * cc);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        O[mt][x][2 * y] *= rf[mt][y] * eb.x;
                        O[mt][x][2 * y + 1] *= rf[mt][y] * eb.y;
                    }
            }
            const float f1 = exp2i(En - E);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nk = 0; nk < NK; ++nk)
#pragma unroll
                    for (int x = 0; x < 4; ++x) S[mt][nk][x] = S[mt][nk][x] * decay * f1;
            E = En;
        }
        __syncthreads();

        // O^T += V^T A^T and S^T += V^T K' (both parts), 16 tokens at a time.
#pragma unroll
        for (int kt = 0; kt < C / 16; ++kt) {
            if (16 * kt < n) {
                uint32_t vf[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    // transposed blocks: value columns 0-7, 8-15 at tokens 0-7, then at 8-15
                    const int r = 16 * kt + (lane & 7) + ((lane >> 4) << 3);
                    const int ch = 2 * (warp * MT + mt) + ((lane >> 3) & 1);
                    ldmatrix4t(vf[mt], sV + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)));
                }
#pragma unroll
                for (int np = kt; np < C / 16; ++np) {
                    uint32_t bf[4];
                    const int rb = 16 * np + (lane & 7) + ((lane >> 4) << 3), cb = 2 * kt + ((lane >> 3) & 1);
                    if (16 * np < n) {
                        ldmatrix4(bf, sA + (uint32_t)(rb * (2 * C) + ((cb ^ (rb & 7)) << 4)));
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            mma16816<__half>(O[mt][2 * np], vf[mt], bf[0], bf[1]);
                            mma16816<__half>(O[mt][2 * np + 1], vf[mt], bf[2], bf[3]);
                        }
                    }
                }
#pragma unroll
                for (int np = 0; np < DK / 16; ++np) {
                    uint32_t hf[4], lf[4];
                    const int r = 16 * kt + (lane & 15), ch = 2 * np + (lane >> 4);
                    const uint32_t at = (uint32_t)(r * KB + ((ch ^ (r & 7)) << 4));
                    ldmatrix4t(hf, sHi + at);
                    ldmatrix4t(lf, sLo + at);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma16816<__half>(S[mt][2 * np], vf[mt], hf[0], hf[1]);
                        mma16816<__half>(S[mt][2 * np + 1], vf[mt], hf[2], hf[3]);
                        mma16816<__half>(S[mt][2 * np], vf[mt], lf[0], lf[1]);
                        mma16816<__half>(S[mt][2 * np + 1], vf[mt], lf[2], lf[3]);
                    }
                }
            }
        }

        // Outputs: transposed into the queries' place, then out in rows.
        const float fo = exp2i(ta - sq - skk - sv) * a.scale;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int np = 0; np < C / 16; ++np) {
                // blocks: (columns 0-7, tokens 0-7), (columns 8-15, tokens 0-7), the same of tokens 8-15
                uint32_t p[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float* o = O[mt][2 * np + (x >> 1)];
                    p[x] = Elem<T>::pack(o[2 * (x & 1)] * fo, o[2 * (x & 1) + 1] * fo);
                }
                const int r = 16 * np + (lane & 7) + ((lane >> 4) << 3);
                const int ch = 2 * (warp * MT + mt) + ((lane >> 3) & 1);
                stmatrix4t(sQ + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)), p[0], p[1], p[2], p[3]);
            }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < C * 2 * MT / 32; ++x) {
            const int r = (x * 32 + lane) / (2 * MT), ch = 2 * warp * MT + lane % (2 * MT);
            const uint4 v = lds128(sQ + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)));
            if (r < n && c0 + 8 * ch < a.v_dim)
                *reinterpret_cast<uint4*>(ob + (t + r) * a.o_stride + 8 * ch) = v;
        }
        __syncthreads();
    }

    const float un = exp2i(-E);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nk = 0; nk < NK; ++nk)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int dv = c0 + (warp * MT + mt) * 16 + gr + 8 * (x >> 1), dk = 8 * nk + 2 * cc + (x & 1);
                if (dv < a.v_dim && dk < a.k_dim) a.state_out[so + (int64_t)dk * a.v_dim + dv] = S[mt][nk][x] * un;
            }
}

}  // namespace q4
