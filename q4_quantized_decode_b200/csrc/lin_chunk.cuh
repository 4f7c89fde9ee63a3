// Linear attention with decay over prompts for k_dim over 128 (whose state does
// not fit the tensor memory beside the other accumulators), 64 tokens at a time
// on mma.sync.  With b_i the sum of the log decays of a chunk's tokens up to i,
//   o_i = e^{b_i} S^T q_i + sum_{j <= i} e^{b_i - b_j} (q_i . k_j) v_j,
//   S'  = e^{b_C} S + sum_j e^{b_C - b_j} k_j v_j^T,
// so a chunk is four matrix products.  They are taken transposed, O^T = S^T Q^T
// + V^T A^T and S'^T = V^T K', because then a warp's accumulators of S^T (16
// value columns as rows, half of k_dim as columns) are, register for register,
// the A operand of the next chunk's first product: the state never leaves the
// registers from a segment's first token to its last.  The two warps of 16
// value columns have their sums of O^T over their halves of k_dim and of the
// tokens, and exchange half of them through shared memory; with half the state
// each, 16 warps have room on an SM, which the products' latencies need (with 8
// warps of the whole k_dim a scheduler issued in 38 of 100 cycles).  Measured,
// 8192 tokens of 40 heads of 256 x 256: 1.94 ms (f16), 2.17 (bf16), 44 and 40
// TFLOP/s of the recurrence's products.
//
// The next chunk's rows are copied, and its decays summed, while this one's
// products run, and each thread looks over the magnitudes of what it copied
// itself, so a chunk has two barriers (three with conversions).
//
// Number formats.  The state and all sums are in 32 bits.  Products run in
// binary16 (bfloat16 inputs are converted, exactly up to values 2^28 under the
// chunk's largest).  The decayed keys k' = e^{b_C - b_j} k_j are split into two
// binary16 parts, so what the state gains has 22 significant bits: one part
// alone would leave the state with binary16's 11.  The state's and the scores'
// operand of the output products are rounded to binary16 once, because the
// output is rounded to 16 bits itself.  Powers of two, taken from the chunk's
// largest magnitudes and the state rows', keep all of that inside binary16's
// range (the state's unit is at most 2^40, so states up to 2^87 fit).  Sums of
// log decays are in 64 bits (differences of far-apart sums).
// A chunk with infinities, NaN or magnitudes from 2^30 on is run token by token
// on the same registers instead, where a zero weight touches nothing.
#pragma once

#include "lin_seg.cuh"
#include "mma_common.cuh"

namespace q4 {

constexpr int kLcTokens = 64;

// A CTA's value columns (16 for each of nw pairs of warps) and its shared memory:
// two buffers of Q (later the chunk's outputs), K and V, the split keys, the
// scores, and for the exchange 2 KB a warp (in K's place where that has room).
__host__ __device__ constexpr int lc_cols(int nw) { return 16 * nw; }
__host__ __device__ constexpr int lc_qbytes(int dk, int nw, bool out) {
    return !out ? 0 : kLcTokens * 2 * (dk > lc_cols(nw) ? dk : lc_cols(nw));
}
__host__ __device__ constexpr int lc_buf(int dk, int nw, bool out) {
    return lc_qbytes(dk, nw, out) + kLcTokens * 2 * (dk + lc_cols(nw));
}
constexpr int kLcDecay = 4 * kLcTokens + 4;          // floats of a chunk's decays
__host__ __device__ constexpr int lc_xbytes(int dk, int nw, bool out) {
    return !out || kLcTokens * 2 * dk >= 4096 * nw ? 0 : 4096 * nw;
}
__host__ __device__ constexpr int lc_smem(int dk, int nw, bool out) {
    return 2 * lc_buf(dk, nw, out) + 2 * kLcTokens * dk * 2 + (out ? kLcTokens * kLcTokens * 2 : 0) +
           lc_xbytes(dk, nw, out) + (2 * kLcDecay + 2 * 3 * 16) * 4;
}

// Two 16-bit values times a power of two, as binary16.
template <typename T>
__device__ __forceinline__ uint32_t to_half2(uint32_t v, float pw) {
    const float2 f = Elem<T>::unpack(v);
    return Elem<__half>::pack(f.x * pw, f.y * pw);
}

// Sums of a chunk's log decays by one warp, two tokens a lane: [64] b_i high
// parts, [64] low parts, [64] e^{b_i}, [64] e^{b_C - b_i}, e^{b_C}, b_C.  Under
// -104 a decay is zero in 32 bits; padding tokens do not decay.
__device__ __forceinline__ float2 decays_of(const float* g, int64_t stride, int64_t t, int64_t t1) {
    const int64_t i = t + 2 * (threadIdx.x & 31);
    return make_float2(i < t1 ? g[i * stride] : 0.f, i + 1 < t1 ? g[(i + 1) * stride] : 0.f);
}
__device__ __forceinline__ void chunk_decays(float2 g, float* out) {
    const int lane = threadIdx.x & 31;
    double b0 = g.x, b1 = g.y;
    if (b0 < -104.0) b0 = -104.0;
    if (b1 < -104.0) b1 = -104.0;
    b1 += b0;
    double p = b1;
    for (int d = 1; d < 32; d <<= 1) {
        const double y = __shfl_up_sync(0xFFFFFFFFu, p, d);
        if (lane >= d) p += y;
    }
    const double before = p - b1;
    b0 += before;
    b1 += before;
    const double all = __shfl_sync(0xFFFFFFFFu, p, 31);
    const int i = 2 * lane;
    *reinterpret_cast<float2*>(out + i) = make_float2((float)b0, (float)b1);
    *reinterpret_cast<float2*>(out + kLcTokens + i) = make_float2((float)(b0 - (float)b0), (float)(b1 - (float)b1));
    *reinterpret_cast<float2*>(out + 2 * kLcTokens + i) = make_float2(expf((float)b0), expf((float)b1));
    *reinterpret_cast<float2*>(out + 3 * kLcTokens + i) = make_float2(expf((float)(all - b0)), expf((float)(all - b1)));
    if (lane == 0) {
        out[4 * kLcTokens] = expf((float)all);
        out[4 * kLcTokens + 1] = (float)all;
    }
}

// OUT: a segment's outputs and last state from its first one; else what it adds
// to a state of zero, and its decay.
template <typename T, int DK, int NW, bool OUT>
__global__ void __launch_bounds__(64 * NW, 1) lin_chunk_kernel(const LinSegArgs g) {
    constexpr bool kConvert = Elem<T>::kExpMask != Elem<__half>::kExpMask;   // bfloat16 inputs
    constexpr int C = kLcTokens;
    constexpr int NT = 64 * NW;
    constexpr int W = 2 * NW;                            // warps
    constexpr int DVS = lc_cols(NW);
    constexpr int KB = DK * 2, VB = DVS * 2;             // row bytes
    constexpr int NK = DK / 16;                          // 8-column tiles of a warp's half of the state
    constexpr uint32_t BUF = lc_buf(DK, NW, OUT);
    constexpr int KCH = C * (DK / 8), VCH = C * (DVS / 8);   // 16-byte chunks of K (or Q) and V
    extern __shared__ __align__(128) uint8_t lc_raw[];
    const LinArgs& a = g.a;
    const uint32_t base = smem_addr(lc_raw);
    const uint32_t sHi = base + 2 * BUF, sLo = sHi + C * KB, sA = sLo + C * KB;
    float* fl = reinterpret_cast<float*>(lc_raw + lc_smem(DK, NW, OUT) - (2 * kLcDecay + 96) * 4);
    uint32_t* sMax = reinterpret_cast<uint32_t*>(fl + 2 * kLcDecay);   // [2][16 warps][3] largest |q|, |k|, |v|

    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, cc = lane & 3;
    const int vg = warp >> 1, half = warp & 1;           // 16 value columns, half of k_dim
    const int kcol = half * (DK / 2);
    const int h = blockIdx.x, c0 = blockIdx.y * DVS;
    const int s = blockIdx.z / g.segs, seg = blockIdx.z - s * g.segs;
    const int slot = a.slots ? a.slots[s] : s;
    if ((unsigned)slot >= (unsigned)a.n_slots) {
        if (threadIdx.x == 0) set_device_error(a.err, kDevIndex);
        return;
    }
    int64_t t0, t1;
    bool last;
    segment(g, s, seg, t0, t1, last);
    if (OUT ? t0 == t1 && !last : last || t0 == t1) return;

    const T* qb = static_cast<const T*>(a.q) + (int64_t)(h / a.each) * a.k_dim;
    const T* kb = static_cast<const T*>(a.k) + (int64_t)(h / a.each) * a.k_dim;
    const T* vb = static_cast<const T*>(a.v) + (int64_t)h * a.v_dim + c0;
    T* ob = static_cast<T*>(a.out) + (int64_t)h * a.v_dim + c0;
    const float* gb = a.g + h;
    const int64_t so = ((int64_t)slot * a.v_heads + h) * a.k_dim * a.v_dim;

    // The state: row vg * 16 + gr (+ 8) of its transpose, columns kcol + 8 nk +
    // 2 cc (+ 1); S holds it times 2^E.
    float S[NK][4];
    int E = 0;
    const float* from = !OUT ? nullptr : g.segs > 1 ? seg_state(g, s, h, seg) : a.state_in ? a.state_in + so : nullptr;
#pragma unroll
    for (int nk = 0; nk < NK; ++nk)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int dv = c0 + vg * 16 + gr + 8 * (x >> 1), dk = kcol + 8 * nk + 2 * cc + (x & 1);
            S[nk][x] = from && dv < a.v_dim && dk < a.k_dim ? from[(int64_t)dk * a.v_dim + dv] : 0.f;
        }

    const int tid = threadIdx.x;
    auto copy = [&](int64_t t, uint32_t buf) {
        const int n = (int)min((int64_t)C, t1 - t);
        const uint32_t sQ = buf, sK = buf + lc_qbytes(DK, NW, OUT), sV = sK + C * KB;
#pragma unroll 4
        for (int x = tid; x < KCH; x += NT) {
            const int r = x / (DK / 8), ch = x % (DK / 8);
            const bool in = r < n && 8 * ch < a.k_dim;
            const uint32_t dst = (uint32_t)(r * KB + ((ch ^ (r & 7)) << 4));
            if (OUT) cp_async16(sQ + dst, in ? qb + (t + r) * a.q_stride + 8 * ch : qb, in);
            cp_async16(sK + dst, in ? kb + (t + r) * a.k_stride + 8 * ch : kb, in);
        }
#pragma unroll 4
        for (int x = tid; x < VCH; x += NT) {
            const int r = x / (DVS / 8), ch = x % (DVS / 8);
            const bool in = r < n && c0 + 8 * ch < a.v_dim;
            cp_async16(sV + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)), in ? vb + (t + r) * a.v_stride + 8 * ch : vb, in);
        }
        cp_async_commit();
    };
    // Waits for this thread's copies and looks over them.
    auto arrived = [&](uint32_t buf, uint32_t* mx) {
        cp_async_wait<0>();
        const uint32_t sQ = buf, sK = buf + lc_qbytes(DK, NW, OUT), sV = sK + C * KB;
        uint32_t m[3] = {0, 0, 0};
#pragma unroll 4
        for (int x = tid; x < KCH; x += NT) {
            const int r = x / (DK / 8), ch = x % (DK / 8);
            const uint32_t at = (uint32_t)(r * KB + ((ch ^ (r & 7)) << 4));
            if (OUT) m[0] = max_abs8(m[0], lds128(sQ + at));
            m[1] = max_abs8(m[1], lds128(sK + at));
        }
#pragma unroll 4
        for (int x = tid; x < VCH; x += NT) {
            const int r = x / (DVS / 8), ch = x % (DVS / 8);
            m[2] = max_abs8(m[2], lds128(sV + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4))));
        }
#pragma unroll
        for (int y = 0; y < 3; ++y) {
            for (int x = 16; x; x >>= 1) m[y] = __vmaxu2(m[y], __shfl_xor_sync(0xFFFFFFFFu, m[y], x));
            if (lane == 0) mx[3 * warp + y] = m[y];
        }
    };
    // The pair of warps with the same value columns.
    auto bar_pair = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + vg) : "memory"); };
    const bool sums = warp == W - 1;                     // this warp sums the decays
    double total = 0;

    if (t0 < t1) {
        copy(t0, base);
        if (sums) chunk_decays(decays_of(gb, a.g_stride, t0, t1), fl);
        arrived(base, sMax);
    }
    __syncthreads();
    int par = 0;
    for (int64_t t = t0; t < t1; t += C, par ^= 1) {
        const int n = (int)min((int64_t)C, t1 - t);
        const uint32_t sQ = base + par * BUF, sK = sQ + lc_qbytes(DK, NW, OUT), sV = sK + C * KB;
        const float* dec = fl + par * kLcDecay;
        const float *sBh = dec, *sBl = dec + C, *sEb = dec + 2 * C, *sW = dec + 3 * C;
        if (t + C < t1) copy(t + C, base + (par ^ 1) * BUF);
        float2 g_next = make_float2(0.f, 0.f);
        if (sums) {
            g_next = decays_of(gb, a.g_stride, t + C, t1);
            total += dec[4 * C + 1];
        }
        auto next_decays = [&]() {
            if (sums && t + C < t1) chunk_decays(g_next, fl + (par ^ 1) * kLcDecay);
        };

        float big[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            uint32_t m = sMax[48 * par + x];
#pragma unroll
            for (int y = 1; y < W; ++y) m = __vmaxu2(m, sMax[48 * par + 3 * y + x]);
            const float2 f = Elem<T>::unpack(m);
            big[x] = fmaxf(f.x, f.y);
            if (!(f.x < 1073741824.f && f.y < 1073741824.f)) big[x] = INFINITY;        // NaN too
        }
        const float decay = dec[4 * C];
        if (!(big[0] < INFINITY && big[1] < INFINITY && big[2] < INFINITY)) {
            // Token by token.
            const float un = exp2i(-E);
            E = 0;
#pragma unroll
            for (int nk = 0; nk < NK; ++nk)
#pragma unroll
                for (int x = 0; x < 4; ++x) S[nk][x] *= un;
            next_decays();
            // The halves' sums of an output meet through the scores' place.
            float* px = reinterpret_cast<float*>(lc_raw + (sA - base)) + vg * 32;
            for (int r = 0; r < n; ++r) {
                const float d = expf(gb[(t + r) * a.g_stride]);
                float v[2], o[2] = {0.f, 0.f};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int c = vg * 16 + gr + 8 * y;
                    uint32_t u;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u)
                                 : "r"(sV + (uint32_t)(r * VB + (((c >> 3) ^ (r & 7)) << 4) + ((c & 6) << 1))));
                    const float2 f = Elem<T>::unpack(u);
                    v[y] = c & 1 ? f.y : f.x;
                }
#pragma unroll
                for (int nk = 0; nk < NK; ++nk) {
                    const int kc = kcol / 8 + nk;
                    const uint32_t at = (uint32_t)(r * KB + ((kc ^ (r & 7)) << 4) + 4 * cc);
                    uint32_t uq = 0, uk;
                    if (OUT) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(uq) : "r"(sQ + at));
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(uk) : "r"(sK + at));
                    const float2 q = Elem<T>::unpack(uq), k = Elem<T>::unpack(uk);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float& s0 = S[nk][2 * y];
                        float& s1 = S[nk][2 * y + 1];
                        s0 = fmaf(s0, d, k.x * v[y]);
                        s1 = fmaf(s1, d, k.y * v[y]);
                        if (OUT && 8 * kc + 2 * cc < a.k_dim) {
                            o[y] = fmaf(q.x * a.scale, s0, o[y]);
                            o[y] = fmaf(q.y * a.scale, s1, o[y]);
                        }
                    }
                }
                if constexpr (OUT) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        o[y] += __shfl_xor_sync(0xFFFFFFFFu, o[y], 1);
                        o[y] += __shfl_xor_sync(0xFFFFFFFFu, o[y], 2);
                        if (half && cc == 0) px[16 * (r & 1) + gr + 8 * y] = o[y];
                    }
                    bar_pair();
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int c = vg * 16 + gr + 8 * y;
                        if (!half && cc == 0 && c0 + c < a.v_dim)
                            ob[(t + r) * a.o_stride + c] = Elem<T>::round(o[y] + px[16 * (r & 1) + gr + 8 * y]);
                    }
                }
            }
        } else {
            // Powers: q, v (and k of the scores) times 2^sq, 2^sv (2^skk) in
            // binary16, the split keys times 2^sk, the scores times 2^-ta.
            const int sk = to_2_14(big[1], 24);
            const int sq = kConvert ? to_2_14(big[0], 24) : 0, sv = kConvert ? to_2_14(big[2], 16) : 0;
            const int skk = kConvert ? sk : 0;
            const float bound = (float)DK * (big[0] * exp2i(sq)) * (big[1] * exp2i(skk));   // of a score
            const int ta = bound == 0.f ? 0 : max(-100, (__float_as_int(bound) >> 23) - 127 - 14);
            const float pk = exp2i(sk);
            if (kConvert) {
                const float pv = exp2i(sv), pq = exp2i(sq);
                for (int x = tid; x < VCH; x += NT) {
                    const uint4 v = lds128(sV + 16u * x);
                    sts128(sV + 16u * x, make_uint4(to_half2<T>(v.x, pv), to_half2<T>(v.y, pv), to_half2<T>(v.z, pv),
                                                    to_half2<T>(v.w, pv)));
                }
                for (int x = tid; x < KCH; x += NT) {
                    if (OUT) {
                        const uint4 q = lds128(sQ + 16u * x);
                        sts128(sQ + 16u * x, make_uint4(to_half2<T>(q.x, pq), to_half2<T>(q.y, pq),
                                                        to_half2<T>(q.z, pq), to_half2<T>(q.w, pq)));
                    }
                }
            }
            // The split keys (and, converted, the scores' keys).
#pragma unroll 4
            for (int x = tid; x < KCH; x += NT) {
                const float w = sW[x / (DK / 8)] * pk;
                const uint4 k = lds128(sK + 16u * x);
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
                if (kConvert && OUT) sts128(sK + 16u * x, make_uint4(kk[0], kk[1], kk[2], kk[3]));
            }
            if (kConvert) __syncthreads();

            float O[OUT ? C / 8 : 1][4];
            if constexpr (OUT) {
                // Scores of the ten 16 x 16 blocks on and under the diagonal in
                // halves of eight columns, each with its decays, as the
                // transposed product's B operand [i][j].
                for (int hb = warp; hb < 20; hb += W) {
                    const int blk = hb >> 1;
                    const int bi = blk == 0 ? 0 : blk < 3 ? 1 : blk < 6 ? 2 : 3, bj = blk - bi * (bi + 1) / 2;
                    if (16 * bi >= n) continue;
                    float sc[4] = {0.f, 0.f, 0.f, 0.f};
                    const int jb = 16 * bj + 8 * (hb & 1);
#pragma unroll
                    for (int kk = 0; kk < DK / 16; kk += 2) {
                        uint32_t af[4], ag[4], bf[4];
                        const int ra = 16 * bi + (lane & 15), ca = 2 * kk + (lane >> 4);
                        ldmatrix4(af, sQ + (uint32_t)(ra * KB + ((ca ^ (ra & 7)) << 4)));
                        ldmatrix4(ag, sQ + (uint32_t)(ra * KB + (((ca + 2) ^ (ra & 7)) << 4)));
                        const int rb = jb + (lane & 7), cb = 2 * kk + (lane >> 3);
                        ldmatrix4(bf, sK + (uint32_t)(rb * KB + ((cb ^ (rb & 7)) << 4)));
                        mma16816<__half>(sc, af, bf[0], bf[1]);
                        mma16816<__half>(sc, ag, bf[2], bf[3]);
                    }
                    const float pa = exp2i(-ta);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int i = 16 * bi + gr + 8 * r;
                        const float bh = sBh[i], bl = sBl[i];
                        float f[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int j = jb + 2 * cc + x;
                            f[x] = j <= i ? sc[2 * r + x] * pa * __expf((bh - sBh[j]) + (bl - sBl[j])) : 0.f;
                        }
                        const uint32_t at = sA + (uint32_t)(i * (2 * C) + (((jb >> 3) ^ (i & 7)) << 4) + 4 * cc);
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(Elem<__half>::pack(f[0], f[1])) : "memory");
                    }
                }

                // O^T = (S^T 2^row) Q^T over this half of k_dim, then brought to
                // the scores' scale with the decays e^{b_i}.
#pragma unroll
                for (int x = 0; x < C / 8; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) O[x][y] = 0.f;
                int rs[2];
                float rp[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    float m = 0.f;
#pragma unroll
                    for (int nk = 0; nk < NK; ++nk) m = fmaxf(m, fmaxf(fabsf(S[nk][2 * y]), fabsf(S[nk][2 * y + 1])));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                    const int e = (__float_as_int(m) >> 23) - 127;
                    rs[y] = m == 0.f || e > 127 ? 0 : min(126, 14 - e);
                    rp[y] = exp2i(rs[y]);
                }
#pragma unroll
                for (int kk = 0; kk < DK / 32; ++kk) {
                    uint32_t af[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float* p = S[2 * kk + (x >> 1)];
                        const float f = rp[x & 1];
                        af[x] = Elem<__half>::pack(p[2 * (x & 1)] * f, p[2 * (x & 1) + 1] * f);
                    }
#pragma unroll
                    for (int np = 0; np < C / 16; ++np) {
                        uint32_t bf[4];
                        const int rb = 16 * np + (lane & 7) + ((lane >> 4) << 3), cb = kcol / 8 + 2 * kk + ((lane >> 3) & 1);
                        ldmatrix4(bf, sQ + (uint32_t)(rb * KB + ((cb ^ (rb & 7)) << 4)));
                        mma16816<__half>(O[2 * np], af, bf[0], bf[1]);
                        mma16816<__half>(O[2 * np + 1], af, bf[2], bf[3]);
                    }
                }
                float rf[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) rf[y] = exp2i(-rs[y] - E + skk + sv - ta);
#pragma unroll
                for (int x = 0; x < C / 8; ++x) {
                    const float2 eb = *reinterpret_cast<const float2*>(sEb + 8 * x + 2 * cc);
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        O[x][2 * y] *= rf[y] * eb.x;
                        O[x][2 * y + 1] *= rf[y] * eb.y;
                    }
                }
            }
            {
                const float f1 = exp2i(sk + sv - E);     // to the unit of this chunk's keys and values
#pragma unroll
                for (int nk = 0; nk < NK; ++nk)
#pragma unroll
                    for (int x = 0; x < 4; ++x) S[nk][x] = S[nk][x] * decay * f1;
                E = sk + sv;
            }
            next_decays();
            __syncthreads();

            // O^T += V^T A^T and S^T += V^T K' (both parts), 16 tokens at a time.
#pragma unroll
            for (int kt = 0; kt < C / 16; ++kt) {
                if (16 * kt < n) {
                    uint32_t vf[4];
                    {
                        // transposed blocks: value columns 0-7, 8-15 at tokens 0-7, then at 8-15
                        const int r = 16 * kt + (lane & 7) + ((lane >> 4) << 3);
                        const int ch = 2 * vg + ((lane >> 3) & 1);
                        ldmatrix4t(vf, sV + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)));
                    }
                    // Of the scores' product each warp of the pair takes half:
                    // tokens 0-15 and 48-63, or 16-47.
                    if (OUT && (kt == 0 || kt == 3) == (half == 0)) {
#pragma unroll
                        for (int np = kt; np < C / 16; ++np) {
                            const int rb = 16 * np + (lane & 7) + ((lane >> 4) << 3), cb = 2 * kt + ((lane >> 3) & 1);
                            if (16 * np < n) {
                                uint32_t bf[4];
                                ldmatrix4(bf, sA + (uint32_t)(rb * (2 * C) + ((cb ^ (rb & 7)) << 4)));
                                mma16816<__half>(O[2 * np], vf, bf[0], bf[1]);
                                mma16816<__half>(O[2 * np + 1], vf, bf[2], bf[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int np = 0; np < DK / 32; ++np) {
                        uint32_t hf[4], lf[4];
                        const int r = 16 * kt + (lane & 15), ch = kcol / 8 + 2 * np + (lane >> 4);
                        const uint32_t at = (uint32_t)(r * KB + ((ch ^ (r & 7)) << 4));
                        ldmatrix4t(hf, sHi + at);
                        ldmatrix4t(lf, sLo + at);
                        mma16816<__half>(S[2 * np], vf, hf[0], hf[1]);
                        mma16816<__half>(S[2 * np + 1], vf, hf[2], hf[3]);
                        mma16816<__half>(S[2 * np], vf, lf[0], lf[1]);
                        mma16816<__half>(S[2 * np + 1], vf, lf[2], lf[3]);
                    }
                }
            }

            if constexpr (OUT) {
                // The pair's sums: each warp gives the other its sums of 32 of the
                // tokens and finishes the 32 others (0-31 the first warp).
                float* xb = reinterpret_cast<float*>(lc_raw + ((lc_xbytes(DK, NW, OUT) ? sA + C * C * 2 : sK) - base));
                {
                    float4* px = reinterpret_cast<float4*>(xb + warp * 512) + lane;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        px[32 * x] = make_float4(half ? O[x][0] : O[4 + x][0], half ? O[x][1] : O[4 + x][1],
                                                 half ? O[x][2] : O[4 + x][2], half ? O[x][3] : O[4 + x][3]);
                    }
                }
                bar_pair();
                float M[4][4];
                {
                    const float4* px = reinterpret_cast<const float4*>(xb + (warp ^ 1) * 512) + lane;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 v = px[32 * x];
                        M[x][0] = (half ? O[4 + x][0] : O[x][0]) + v.x;
                        M[x][1] = (half ? O[4 + x][1] : O[x][1]) + v.y;
                        M[x][2] = (half ? O[4 + x][2] : O[x][2]) + v.z;
                        M[x][3] = (half ? O[4 + x][3] : O[x][3]) + v.w;
                    }
                }
                // Transposed into the queries' place, then out in rows.
                const float fo = exp2i(ta - sq - skk - sv) * a.scale;
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    // blocks: (columns 0-7, tokens 0-7), (columns 8-15, tokens 0-7), the same of tokens 8-15
                    uint32_t p[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float* o = M[2 * np + (x >> 1)];
                        p[x] = Elem<T>::pack(o[2 * (x & 1)] * fo, o[2 * (x & 1) + 1] * fo);
                    }
                    const int r = 32 * half + 16 * np + (lane & 7) + ((lane >> 4) << 3);
                    const int ch = 2 * vg + ((lane >> 3) & 1);
                    stmatrix4t(sQ + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)), p[0], p[1], p[2], p[3]);
                }
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 32 * half + 16 * x + (lane >> 1), ch = 2 * vg + (lane & 1);
                    const uint4 v = lds128(sQ + (uint32_t)(r * VB + ((ch ^ (r & 7)) << 4)));
                    if (r < n && c0 + 8 * ch < a.v_dim)
                        *reinterpret_cast<uint4*>(ob + (t + r) * a.o_stride + 8 * ch) = v;
                }
            }
        }
        if (t + C < t1) arrived(base + (par ^ 1) * BUF, sMax + 48 * (par ^ 1));
        __syncthreads();
    }

    if (!OUT && sums && lane == 0 && blockIdx.y == 0) *seg_decay(g, s, h, seg) = expf((float)total);
    float* to = OUT ? (last ? a.state_out + so : nullptr) : seg_state(g, s, h, seg);
    if (!to) return;
    const float un = exp2i(-E);
#pragma unroll
    for (int nk = 0; nk < NK; ++nk)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int dv = c0 + vg * 16 + gr + 8 * (x >> 1), dk = kcol + 8 * nk + 2 * cc + (x & 1);
            if (dv < a.v_dim && dk < a.k_dim) to[(int64_t)dk * a.v_dim + dv] = S[nk][x] * un;
        }
}

}  // namespace q4
