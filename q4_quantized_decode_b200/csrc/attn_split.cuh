// Attention of few new tokens (single tokens, drafted ones) over a paged
// cache: bound by the cache's bytes, so the cache is read once for all query
// heads of a key head, by the whole chip, whatever the batch looks like.
//
// The rows of a sequence (its new tokens times the query heads of one key
// head) form tiles of 16; a tile of one key head is a unit, and a unit's keys
// are counted in groups of 256.  The groups of all units, one after the other,
// are cut into equal runs, one for each CTA: a long sequence is split over
// many CTAs, short ones share one.  The cut is computed on the device from the
// lengths, so a captured call follows them.  A unit inside one run is finished
// there; the pieces of others go to a workspace (at most two a CTA) and the CTA
// that comes last joins them in order.
//
// Within a CTA each of four warps has its own 16 keys of a block, its own ring
// of asynchronous copies and its own softmax (running maximum and sum, 32
// bits); they meet once, at the end of a run's unit.  The products run on
// mma.sync m16n8k16: its rows are mostly empty for one token (5 of 16 with
// five query heads to a key head), but the tensor rate is not what bounds
// this.  Weights are rounded once to the 16-bit type for the second product
// (the first one's sums are not).
//
// Measured (40 query and 8 key heads of 128): one token of each of 32 sequences
// of up to 16384 (bf16), 171 us, 6.1 TB/s of keys and values; one token of one
// sequence of 4096, 15.7 us, which is latency: 2.2 us to read the lengths and
// cut, 1.2 to the first keys, 4 for a warp's four tiles, 2.6 to the workspace,
// 4 for the join.
#pragma once

#include "attn_rows.cuh"
#include "mma_common.cuh"

namespace q4 {

constexpr int kSplitWarps = 4;
constexpr int kSplitThreads = 32 * kSplitWarps;
constexpr int kSplitKeys = 16;                          // keys of a warp's tile
constexpr int kSplitBlock = kSplitKeys * kSplitWarps;   // keys of a CTA's step
constexpr int kSplitGroup = 4 * kSplitBlock;            // keys of a group
constexpr int kSplitRows = 16;
constexpr int kSplitStages = 3;
// CTAs of an SM at each padded head size (shared memory: stages * 4 warps * 16
// keys * 2 * size * 2 bytes, 48 / 96 / 192 KB).
__host__ __device__ constexpr int split_ctas_per_sm(int dp) { return dp == 64 ? 4 : dp == 128 ? 2 : 1; }
__host__ __device__ constexpr int split_smem(int dp) {
    return kSplitStages * kSplitWarps * kSplitKeys * 2 * dp * 2 + kSplitStages * kSplitWarps * 4;
}
// Floats of one workspace slot: 16 rows of sums, their maxima and weights' sums.
__host__ __device__ constexpr int split_slot(int dp) { return kSplitRows * (dp + 2); }

struct SplitAttnArgs {
    AttnArgs a;
    float* ws;          // [2 * gridDim.x] slots
    int* cnt;           // [gridDim.x] arrivals, zero between calls
    int max_rows;       // rows (tokens * group) of a sequence that this kernel takes; 0: any
};

// The units of sequence s: `tiles` row tiles (times the key heads), each of
// `groups` key groups (the count for the longest range of its rows).
struct SeqWork {
    int64_t first;      // first row of the batch
    int n, len;         // new tokens, tokens in the cache
    int tiles, groups;
    __device__ __forceinline__ int64_t all(int heads) const { return (int64_t)tiles * groups * heads; }
    int lo;             // first key that any row sees
};

__device__ __forceinline__ SeqWork seq_work(const SplitAttnArgs& g, int s) {
    const AttnArgs& a = g.a;
    SeqWork w;
    seq_rows(a.batch, s, w.first, w.n);
    w.len = a.batch.len[s];
    const int64_t rows = (int64_t)w.n * a.group;
    w.tiles = w.groups = w.lo = 0;
    if (w.n == 0 || (g.max_rows && rows > g.max_rows)) return w;
    w.tiles = (int)((rows + kSplitRows - 1) / kSplitRows);
    int hi, lo1;
    seen_range(a, w.len, w.n, 0, w.lo, hi);             // the first row starts lowest
    seen_range(a, w.len, w.n, w.n - 1, lo1, hi);        // the last one ends highest
    w.lo = w.lo / kSplitBlock * kSplitBlock;
    w.groups = hi > w.lo ? (hi - w.lo + kSplitGroup - 1) / kSplitGroup : 1;   // an empty range is one group
    return w;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kSplitThreads, split_ctas_per_sm(DP)) attn_split_kernel(const SplitAttnArgs g) {
    constexpr int CH = DP / 8;                            // 16-byte chunks of a padded head
    constexpr int ROWB = DP * 2;
    constexpr int TILEB = kSplitKeys * ROWB;              // one K or V tile of a warp
    extern __shared__ __align__(128) uint8_t split_smem_raw[];
    __shared__ int last_word;
    const AttnArgs& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.kv.head_dim;
    const uint32_t ring = smem_addr(split_smem_raw) + (uint32_t)(warp * kSplitStages * 2 * TILEB);
    volatile uint32_t* okw = reinterpret_cast<volatile uint32_t*>(
        split_smem_raw + kSplitStages * kSplitWarps * 2 * TILEB) + warp * kSplitStages;

    pdl_wait();
    pdl_launch_dependents();

    // Groups of all units, and this CTA's run of them.
    const int nh = a.kv.n_heads, n_seqs = a.batch.n_seqs;
    SeqWork w;
    w.tiles = w.groups = 0;
    int64_t total = 0, first_all = 0;                     // first_all: lane's sequence of the first 32
    for (int q = lane; q < n_seqs; q += 32) {
        const SeqWork x = seq_work(g, q);
        total += x.all(nh);
        if (q == lane) {
            w = x;
            first_all = x.all(nh);
        }
    }
    for (int x = 16; x; x >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, x);
    const int runs = (int)min((int64_t)gridDim.x, total);
    const int me = (int)blockIdx.x;
    if (me >= runs) return;
    const double ratio = (double)total / (double)runs;    // groups of a run; the same cuts in every CTA
    auto run_start = [&](int c) { return c >= runs ? total : (int64_t)((double)c * ratio); };
    const int64_t b0 = run_start(me), b1 = run_start(me + 1);

    // The sequence of group b0: prefix sums of 32 sequences at a time.
    int64_t seq_base = 0;                                 // groups before sequence s
    int s = 0;
    for (int c0 = 0; c0 < n_seqs; c0 += 32) {
        if (c0 > 0) {
            w.tiles = w.groups = 0;
            if (c0 + lane < n_seqs) w = seq_work(g, c0 + lane);
        }
        const int64_t x = c0 > 0 ? w.all(nh) : first_all;
        int64_t p = x;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, p, d);
            if (lane >= d) p += y;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, seq_base + p > b0);
        if (past) {
            const int l = __ffs((int)past) - 1;
            s = c0 + l;
            seq_base += __shfl_sync(0xFFFFFFFFu, p - x, l);
            w.first = __shfl_sync(0xFFFFFFFFu, w.first, l);
            w.n = __shfl_sync(0xFFFFFFFFu, w.n, l);
            w.len = __shfl_sync(0xFFFFFFFFu, w.len, l);
            w.tiles = __shfl_sync(0xFFFFFFFFu, w.tiles, l);
            w.groups = __shfl_sync(0xFFFFFFFFu, w.groups, l);
            w.lo = __shfl_sync(0xFFFFFFFFu, w.lo, l);
            break;
        }
        seq_base += __shfl_sync(0xFFFFFFFFu, p, 31);
    }

    for (int64_t b = b0; b < b1;) {
        while (b >= seq_base + w.all(nh) && s + 1 < n_seqs) {          // sequences without groups are passed
            seq_base += w.all(nh);
            w = seq_work(g, ++s);
        }
        const int64_t unit = div_floor(b - seq_base, max(1, w.groups));
        const int64_t ub = seq_base + unit * w.groups;                 // the unit's first group
        const int64_t be = b1 < ub + w.groups ? b1 : ub + w.groups;
        const int rt = (int)div_floor(unit, nh), hk = (int)(unit - (int64_t)rt * nh);
        const int n_rows = min(kSplitRows, w.n * a.group - rt * kSplitRows);

        // Ranges: this thread's rows lane / 4 and that + 8, the tile's union
        // and intersection.
        int rlo[2], rhi[2];
        int tlo = INT32_MAX, thi = 0, ilo = 0, ihi = INT32_MAX;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (lane >> 2) + 8 * i;
            rlo[i] = rhi[i] = 0;
            if (r < n_rows) {
                seen_range(a, w.len, w.n, (rt * kSplitRows + r) / a.group, rlo[i], rhi[i]);
                if (rlo[i] < rhi[i]) {
                    tlo = min(tlo, rlo[i]);
                    thi = max(thi, rhi[i]);
                }
                ilo = max(ilo, rlo[i]);
                ihi = min(ihi, rhi[i]);
            }
        }
        for (int x = 16; x; x >>= 1) {
            tlo = min(tlo, __shfl_xor_sync(0xFFFFFFFFu, tlo, x));
            thi = max(thi, __shfl_xor_sync(0xFFFFFFFFu, thi, x));
            ilo = max(ilo, __shfl_xor_sync(0xFFFFFFFFu, ilo, x));
            ihi = min(ihi, __shfl_xor_sync(0xFFFFFFFFu, ihi, x));
        }
        // This warp's tiles: keys k0 + 64 i .. + 16, i in [0, nt).
        const int from = w.lo + (int)(b - ub) * kSplitGroup;
        const int nt = min((int)(be - b) * (kSplitGroup / kSplitBlock), max(0, (thi - from + kSplitBlock - 1) / kSplitBlock));
        const int k0 = from + warp * kSplitKeys;

        // Key `lane & 15` of tile i: its element offset, or -1.
        const int64_t ho = (int64_t)hk * a.kv.head_stride;
        auto locate = [&](int i) -> int64_t {
            const int j = k0 + i * kSplitBlock + (lane & 15);
            int64_t off = -1;
            if (i < nt && j >= tlo && j < thi) off = token_offset(a.kv, s, j, a.err);
            return off < 0 ? -1 : off + ho;
        };
        auto issue = [&](int i, int64_t off) {
            if (i < nt) {
                const int st = i % kSplitStages;
                const uint32_t kt = ring + (uint32_t)(st * 2 * TILEB), vt = kt + TILEB;
                const unsigned ok = __ballot_sync(0xFFFFFFFFu, off >= 0) & 0xFFFFu;
                if (lane == 0) okw[st] = ok;
#pragma unroll
                for (int it = 0; it < CH / 2; ++it) {
                    const int ci = it * 32 + lane;
                    const int row = ci / CH, ch = ci % CH;
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
                    const bool in = o >= 0 && 8 * ch < D;
                    const int64_t e = in ? o + 8 * ch : 0;
                    const uint32_t dst = (uint32_t)(row * ROWB + ((ch ^ (row & 7)) << 4));
                    cp_async16(kt + dst, static_cast<const T*>(a.kv.k) + e, in);
                    cp_async16(vt + dst, static_cast<const T*>(a.kv.v) + e, in);
                }
            }
            cp_async_commit();
        };

        int64_t off = locate(0);
#pragma unroll
        for (int i = 0; i < kSplitStages - 1; ++i) {
            const int64_t cur = off;
            off = locate(i + 1);
            issue(i, cur);
        }

        // Queries as the first product's A operand.
        uint32_t qf[DP / 16][4];
        {
            const T* qp[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = rt * kSplitRows + (lane >> 2) + 8 * i;
                const int t = r / a.group, gh = r - t * a.group;
                qp[i] = (lane >> 2) + 8 * i < n_rows
                            ? static_cast<const T*>(a.q) + (w.first + t) * a.q_stride + (int64_t)(hk * a.group + gh) * D
                            : nullptr;
            }
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int col = 16 * kk + 8 * (x >> 1) + 2 * (lane & 3);
                    const T* p = qp[x & 1];
                    qf[kk][x] = p && col < D ? *reinterpret_cast<const uint32_t*>(p + col) : 0u;
                }
        }
        float o[DP / 8][4];
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int i = 0; i < nt; ++i) {
            {
                const int64_t cur = off;
                off = locate(i + kSplitStages);
                issue(i + kSplitStages - 1, cur);
            }
            cp_async_wait<kSplitStages - 1>();
            __syncwarp();
            const int st = i % kSplitStages;
            const uint32_t kt = ring + (uint32_t)(st * 2 * TILEB), vt = kt + TILEB;
            const uint32_t ok = okw[st];
            const int j0 = k0 + i * kSplitBlock;
            if (ok != 0) {
            // Scores of 16 rows x 16 keys.
            float sc[2][4];
#pragma unroll
            for (int x = 0; x < 8; ++x) sc[x >> 2][x & 3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                // matrices: keys 0-7 and 8-15, elements 16 kk .. + 8 and + 16
                uint32_t bf[4];
                const int row = (lane & 7) + ((lane >> 4) << 3), ch = 2 * kk + ((lane >> 3) & 1);
                ldmatrix4(bf, kt + (uint32_t)(row * ROWB + ((ch ^ (row & 7)) << 4)));
                mma16816<T>(sc[0], qf[kk], bf[0], bf[1]);
                mma16816<T>(sc[1], qf[kk], bf[2], bf[3]);
            }
            const bool mixed = ok != 0xFFFFu || j0 < ilo || j0 + kSplitKeys > ihi;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v = sc[y][x] * a.scale_log2;
                    if (mixed) {
                        const int c = 8 * y + 2 * (lane & 3) + (x & 1), j = j0 + c;
                        if (j < rlo[x >> 1] || j >= rhi[x >> 1] || !((ok >> c) & 1)) v = -INFINITY;
                    }
                    sc[y][x] = v;
                }
            float p[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]), fmaxf(sc[1][2 * r], sc[1][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                const float mn = fmaxf(m[r], mx);
                const float mu = mn == -INFINITY ? 0.f : mn;
                const float wt = exp2f(m[r] - mu);
                m[r] = mn;
                l[r] *= wt;
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        p[y][2 * r + x] = exp2f(sc[y][2 * r + x] - mu);
                        l[r] += p[y][2 * r + x];
                    }
                if (__any_sync(0xFFFFFFFFu, wt != 1.f)) {
#pragma unroll
                    for (int nn = 0; nn < DP / 8; ++nn) {
                        o[nn][2 * r] *= wt;
                        o[nn][2 * r + 1] *= wt;
                    }
                }
            }
            // A value that is not finite must not meet the zero weight of a
            // row that does not see its token (0 x Inf is NaN).  Tiles that
            // rows see in different parts are looked over first.
            bool slow = false;
            if (mixed) {
#pragma unroll
                for (int it = 0; it < CH / 2; ++it) slow |= any_nonfinite<T>(lds128(vt + (uint32_t)((it * 32 + lane) << 4)));
                slow = __any_sync(0xFFFFFFFFu, slow);
            }
            if (!slow) {
                uint32_t af[4];
                af[0] = Elem<T>::pack(p[0][0], p[0][1]);
                af[1] = Elem<T>::pack(p[0][2], p[0][3]);
                af[2] = Elem<T>::pack(p[1][0], p[1][1]);
                af[3] = Elem<T>::pack(p[1][2], p[1][3]);
#pragma unroll
                for (int nn = 0; nn < DP / 16; ++nn) {
                    // transposed: keys 0-7, 8-15 at elements 16 nn, the same at + 8
                    uint32_t bf[4];
                    const int row = lane & 15, ch = 2 * nn + (lane >> 4);
                    ldmatrix4t(bf, vt + (uint32_t)(row * ROWB + ((ch ^ (row & 7)) << 4)));
                    mma16816<T>(o[2 * nn], af, bf[0], bf[1]);
                    mma16816<T>(o[2 * nn + 1], af, bf[2], bf[3]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < kSplitKeys; ++c) {
                    const int from = (lane & ~3) | ((c & 7) >> 1);
                    const float p0 = __shfl_sync(0xFFFFFFFFu, p[c >> 3][c & 1], from);
                    const float p1 = __shfl_sync(0xFFFFFFFFu, p[c >> 3][2 + (c & 1)], from);
#pragma unroll
                    for (int nn = 0; nn < DP / 8; ++nn) {
                        uint32_t vv;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(vv)
                                     : "r"(vt + (uint32_t)(c * ROWB + ((nn ^ (c & 7)) << 4) + 4 * (lane & 3))));
                        const float2 v = Elem<T>::unpack(vv);
                        if (p0 != 0.f) {
                            o[nn][0] = fmaf(p0, v.x, o[nn][0]);
                            o[nn][1] = fmaf(p0, v.y, o[nn][1]);
                        }
                        if (p1 != 0.f) {
                            o[nn][2] = fmaf(p1, v.x, o[nn][2]);
                            o[nn][3] = fmaf(p1, v.y, o[nn][3]);
                        }
                    }
                }
            }
            }
            __syncwarp();                       // the stage may be filled again
        }
        cp_async_wait<0>();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
        }
        __syncthreads();                        // every warp is done with its ring
        // The warps' sums meet in shared memory: [4][16][DP], then m, l [4][16].
        float* so = reinterpret_cast<float*>(split_smem_raw);
        float* sm = so + kSplitWarps * kSplitRows * DP;
        float* sl = sm + kSplitWarps * kSplitRows;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
#pragma unroll
            for (int nn = 0; nn < DP / 8; ++nn)
                *reinterpret_cast<float2*>(so + (warp * kSplitRows + row) * DP + 8 * nn + 2 * (lane & 3)) =
                    make_float2(o[nn][2 * r], o[nn][2 * r + 1]);
            if ((lane & 3) == 0) {
                sm[warp * kSplitRows + row] = m[r];
                sl[warp * kSplitRows + row] = l[r];
            }
        }
        __syncthreads();
        const bool whole = b == ub && be == ub + w.groups;
        const bool first_seg = b == b0;
        float* slot = g.ws + ((int64_t)blockIdx.x * 2 + (first_seg ? 0 : 1)) * split_slot(DP);
        auto store_out = [&](int row, int c4, float4 v) {
            const int r = rt * kSplitRows + row, t = r / a.group, gh = r - t * a.group;
            if (4 * c4 >= D) return;
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (w.first + t) * a.o_stride +
                                      (int64_t)(hk * a.group + gh) * D + 4 * c4) =
                make_uint2(Elem<T>::pack(v.x, v.y), Elem<T>::pack(v.z, v.w));
        };
        for (int x = threadIdx.x; x < n_rows * (DP / 4); x += kSplitThreads) {
            const int row = x / (DP / 4), c4 = x % (DP / 4);
            float mx = -INFINITY;
#pragma unroll
            for (int y = 0; y < kSplitWarps; ++y) mx = fmaxf(mx, sm[y * kSplitRows + row]);
            const float mu = mx == -INFINITY ? 0.f : mx;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            float ls = 0.f;
#pragma unroll
            for (int y = 0; y < kSplitWarps; ++y) {
                const float wt = exp2f(sm[y * kSplitRows + row] - mu);
                const float4 u = *reinterpret_cast<const float4*>(so + (y * kSplitRows + row) * DP + 4 * c4);
                v.x += wt * u.x;
                v.y += wt * u.y;
                v.z += wt * u.z;
                v.w += wt * u.w;
                ls += wt * sl[y * kSplitRows + row];
            }
            if (whole) {
                const float inv = ls == 0.f ? 0.f : 1.f / ls;
                store_out(row, c4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
            } else {
                *reinterpret_cast<float4*>(slot + row * DP + 4 * c4) = v;
                if (c4 == 0) {
                    slot[kSplitRows * DP + row] = mx;
                    slot[kSplitRows * DP + kSplitRows + row] = ls;
                }
            }
        }
        if (!whole) {
            // The unit's pieces are in the CTAs c_lo .. c_hi; its count is kept
            // under c_lo, whose run no other unit leaves at its end.
            auto cta_of = [&](int64_t grp) {
                int c = min(runs - 1, (int)((double)grp / ratio));
                while (c + 1 < runs && run_start(c + 1) <= grp) ++c;
                while (c > 0 && run_start(c) > grp) --c;
                return c;
            };
            const int c_lo = cta_of(ub), c_hi = cta_of(ub + w.groups - 1);
            const int pieces = c_hi - c_lo + 1;
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) last_word = atom_add_acq_rel_gpu(g.cnt + c_lo, 1) == pieces - 1;
            __syncthreads();
            if (last_word) {
                __threadfence();
                if (threadIdx.x == 0) g.cnt[c_lo] = 0;
                // Every piece but the first begins its CTA's run: the first slot.
                const int64_t slot0 = 2 * (int64_t)c_lo + (run_start(c_lo) >= ub ? 0 : 1);
                auto piece = [&](int p) { return g.ws + (p ? 2 * (int64_t)(c_lo + p) : slot0) * split_slot(DP); };
                // Shared memory: the pieces' rows' weights [pieces][16], the
                // rows' 1 / sum.
                float* wts = reinterpret_cast<float*>(split_smem_raw);
                float* invs = wts + gridDim.x * kSplitRows;
                {
                    // Eight threads a row.
                    const int row = threadIdx.x >> 3, part = threadIdx.x & 7;
                    float mx = -INFINITY, ls = 0.f;
                    if (row < n_rows)
#pragma unroll 4
                        for (int p = part; p < pieces; p += 8) {
                            const float v = __ldcg(piece(p) + kSplitRows * DP + row);
                            const float sum = __ldcg(piece(p) + kSplitRows * DP + kSplitRows + row);
                            wts[p * kSplitRows + row] = v;
                            const float mn = fmaxf(mx, v), mu = mn == -INFINITY ? 0.f : mn;
                            ls = ls * exp2f(mx - mu) + sum * exp2f(v - mu);
                            mx = mn;
                        }
#pragma unroll
                    for (int x = 1; x < 8; x <<= 1) {
                        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, mx, x), l2 = __shfl_xor_sync(0xFFFFFFFFu, ls, x);
                        const float mn = fmaxf(mx, m2), mu = mn == -INFINITY ? 0.f : mn;
                        ls = ls * exp2f(mx - mu) + l2 * exp2f(m2 - mu);
                        mx = mn;
                    }
                    const float mu = mx == -INFINITY ? 0.f : mx;
                    if (row < n_rows)
                        for (int p = part; p < pieces; p += 8)
                            wts[p * kSplitRows + row] = exp2f(wts[p * kSplitRows + row] - mu);
                    if (part == 0) invs[row] = ls == 0.f ? 0.f : 1.f / ls;
                }
                __syncthreads();
                for (int x = threadIdx.x; x < n_rows * (DP / 4); x += kSplitThreads) {
                    const int row = x / (DP / 4), c4 = x % (DP / 4);
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float* at = g.ws + row * DP + 4 * c4;
#pragma unroll 16
                    for (int p = 0; p < pieces; ++p) {
                        const float wt = wts[p * kSplitRows + row];
                        const float4 u = __ldcg(reinterpret_cast<const float4*>(
                            at + (p ? 2 * (int64_t)(c_lo + p) : slot0) * split_slot(DP)));
                        v.x += wt * u.x;
                        v.y += wt * u.y;
                        v.z += wt * u.z;
                        v.w += wt * u.w;
                    }
                    const float inv = invs[row];
                    store_out(row, c4, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
                }
            }
        }
        __syncthreads();                        // shared memory is free for the next unit
        b = be;
    }
}

}  // namespace q4
