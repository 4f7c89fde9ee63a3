// Attention of many new tokens (chunks of prompts) over a paged cache on the
// 5th-generation tensor cores.
//
// The rows of a sequence (its new tokens times the query heads of one key
// head) form tiles of 256, two accumulators of 128: a tile of one key head is
// a unit.  For every 128 keys a CTA computes S = Q K^T of both accumulators,
// turns S into weights P = 2^(S - m) and adds P V to both sums:
//   warps 0-3, 4-7  the softmax of one accumulator each, a thread a row: S from
//              tensor memory, the running maximum m and sum (32 bits), P back
//              into S's place in the 16-bit type (the one rounding before the
//              output's), the sums brought to a new m when it has risen by more
//              than 2^8 (until then P may pass 1 and stays far from overflow);
//   warp 8     one thread issues the products: S of one accumulator runs while
//              the other one's softmax does;
//   warps 9-10 the pages' rows into a ring of 128-key tiles, in the 128-byte
//              swizzle that the products read (K as rows of K, V as an N-major
//              operand): tiles that every row sees whole by tensor map, where
//              pages of a multiple of 8 tokens allow it, the others by asynchronous
//              16-byte copies, because pages may end anywhere in a tile and
//              keys that no row sees have to be zeros.
// Two products of 128 x 128 x head_dim for each accumulator and tile, 16384
// powers of two: the tensor pipe and the exponential unit need about the same
// time, 2048 cycles for a CTA's tile at head size 128, under which the two
// groups' chain of S, maximum, powers, P and P V takes 4400.  Measured (f16, 40
// query and 8 key heads of 128): 4096 new tokens behind 12288, 1.20 ms, 1000
// TFLOP/s; four prompts' chunks of up to 1024 (bf16, 16 / 4 heads of 64, pages
// of 24) 196 us, 346 TFLOP/s.  Part of the powers by a polynomial of degree 4 on
// the FMA units was slower (a quarter of them: 2.30 against 2.20 ms): the
// issue slots are as busy.
//
// Head sizes over 128 leave room for the sums of one accumulator beside S (256
// and 128 of 512 columns): units of 128 rows, of which the two groups take 64
// keys of a tile and half of the sums' columns each; a warp and its fellow of
// the other group meet once a tile, to agree on the row maxima.  Measured, 32 /
// 4 heads of 256: 4096 new tokens behind 8192, 1.45 ms, 946 TFLOP/s; 16 / 4
// heads, 2048 behind 2048, 168 us (16 rows at a time on mma.sync: 1924).
//
// The units' key tiles are cut over the CTAs on the device: with few units
// each is split over several CTAs, with many the units' costs (which grow with
// the rows' places, when causal) form one line that is cut into equal runs.
// Pieces of a unit go to the workspace, at most two a CTA, and the CTA that
// comes last joins them in order.
//
// What rows do not see cannot reach them: a weight of zero times a value that
// is not finite would (and a page outside the pool has no keys at all), so the
// copying warps look at values in tiles that rows see in different parts, and
// a unit with such a value, or with a bad page, is taken row by row at the end.
#pragma once

#include <cuda.h>

#include "attn_rows.cuh"
#include "mma_common.cuh"
#include "tc_common.cuh"

namespace q4 {

constexpr int kTaKeys = 128;                 // keys of a tile
constexpr int kTaLoaders = 2;
constexpr int kTaThreads = 32 * 12;
constexpr int kTaSegs = 4;                   // parts told ahead
constexpr int kTaOver = 128;                 // a unit's fixed cost in keys: its start and end

// Ring slots (a K or a V tile each) beside the queries.
__host__ __device__ constexpr int ta_slots(int dp) { return dp == 64 ? 8 : dp == 128 ? 4 : 2; }
// Rows of a unit, 128 for each accumulator.
__host__ __device__ constexpr int ta_rows(int dp) { return dp == 256 ? 128 : 256; }
__host__ __device__ constexpr int ta_smem(int dp) {
    return 1024 + ta_rows(dp) * dp * 2 + ta_slots(dp) * kTaKeys * dp * 2 + 512 + (dp == 256 ? 2 * 2 * 128 * 4 : 0);
}
// Floats of a workspace slot: sums [dp / 4][rows][4], maxima, weights' sums.
__host__ __device__ constexpr int ta_slot(int dp) { return ta_rows(dp) * (dp + 2); }

struct TcAttnArgs {
    AttnArgs a;
    float* ws;           // [2 * gridDim.x] slots
    int* cnt;            // [gridDim.x] arrivals, zero between calls
    int min_rows;        // sequences of at most this many rows are another kernel's
    uint32_t idesc_s, idesc_o;
    int box;             // tokens of a tensor-map box (8..128, dividing page_size), 0: no maps
    CUtensorMap kmap, vmap;   // [page][head][token][element], boxes of 64 elements x `box` tokens
};

// The units of a sequence: `tiles` row tiles, of cost c0 + c1 rt each.
struct TaSeq {
    int64_t first;
    int n, len, tiles, c0, c1;
    __device__ __forceinline__ int64_t before(int64_t rt) const { return rt * c0 + c1 * (rt * (rt - 1) / 2); }
};

template <int ROWS>
__device__ __forceinline__ TaSeq ta_seq(const TcAttnArgs& g, int s) {
    TaSeq q;
    seq_rows(g.a.batch, s, q.first, q.n);
    q.len = g.a.batch.len[s];
    const int64_t rows = (int64_t)q.n * g.a.group;
    q.tiles = q.c0 = q.c1 = 0;
    if (rows <= g.min_rows) return q;
    q.tiles = (int)((rows + ROWS - 1) / ROWS);
    int lo, hi;
    if (g.a.causal && (g.a.window == 0 || g.a.window >= q.len)) {
        seen_range(g.a, q.len, q.n, min(q.n - 1, (ROWS - 1) / g.a.group), lo, hi);
        q.c1 = ROWS / g.a.group;
    } else {
        seen_range(g.a, q.len, q.n, q.n - 1, lo, hi);
    }
    q.c0 = hi - lo + kTaOver;
    return q;
}

// A CTA's part of one unit, as the other warps get it.
struct TaSeg {
    int more;            // 0: no further part, the rest is not set
    int s, hk, len, n;
    int n_rows;          // rows of the unit
    int t0, g0;          // token and query head (of the key head's) of its first row
    int64_t first;       // the sequence's first row in the batch
    int j0, nt;          // first key of the part (a multiple of 128), its 128-key tiles
    int tlo, thi;        // keys that any row of the unit sees
    int pieces, c_lo;    // pieces of the unit, the CTA of the first
    int slot, slot0;     // workspace slots of this piece and of the first
};

// Walks over a CTA's units (one warp, all lanes alike).
struct TaWalk {
    double ratio;        // cost of a run
    int64_t total, b0, b1, b, seq_base;
    int runs, s, k;      // k > 0: few units, k CTAs for each
    bool done;
    TaSeq q;

    __device__ __forceinline__ int64_t cut(int c) const { return c >= runs ? total : (int64_t)((double)c * ratio); }
};

// The sequence whose units (by count, or by cost) hold place x.
template <int ROWS>
__device__ __forceinline__ void ta_find(const TcAttnArgs& g, int64_t x, bool by_units, int& s, int64_t& base) {
    const int lane = threadIdx.x & 31, nh = g.a.kv.n_heads, n_seqs = g.a.batch.n_seqs;
    base = 0;
    s = 0;
    for (int c0 = 0; c0 < n_seqs; c0 += 32) {
        int64_t v = 0;
        if (c0 + lane < n_seqs) {
            const TaSeq q = ta_seq<ROWS>(g, c0 + lane);
            v = (by_units ? q.tiles : q.before(q.tiles)) * nh;
        }
        int64_t p = v;
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, p, d);
            if (lane >= d) p += y;
        }
        const unsigned past = __ballot_sync(0xFFFFFFFFu, base + p > x);
        if (past) {
            const int l = __ffs((int)past) - 1;
            s = c0 + l;
            base += __shfl_sync(0xFFFFFFFFu, p - v, l);
            return;
        }
        base += __shfl_sync(0xFFFFFFFFu, p, 31);
    }
}

// Place x of sequence q's cost (from its beginning): row tile, key head, place
// within the unit.
__device__ __forceinline__ void ta_unit(const TaSeq& q, int nh, int64_t x, int& rt, int& hk, int& in) {
    const int64_t xh = div_floor(x, nh);
    int64_t r;
    if (q.c1 == 0) {
        r = div_floor(xh, max(1, q.c0));
    } else {
        const float c1 = (float)q.c1, m = (float)q.c0 - 0.5f * c1;
        r = (int64_t)((sqrtf(m * m + 2.f * c1 * (float)xh) - m) / c1);
    }
    r = max((int64_t)0, min(r, (int64_t)q.tiles - 1));
    while (r > 0 && q.before(r) > xh) --r;
    while (r + 1 < q.tiles && q.before(r + 1) <= xh) ++r;
    const int cu = q.c0 + q.c1 * (int)r;
    const int64_t rest = x - q.before(r) * nh;
    rt = (int)r;
    hk = (int)div_floor(rest, max(1, cu));
    in = (int)(rest - (int64_t)hk * cu);
}

// Keys of row tile rt (the first row starts lowest, the last ends highest):
// the first 128-key tile's first key, the tiles.
template <int ROWS>
__device__ __forceinline__ int ta_tiles(const TcAttnArgs& g, const TaSeq& q, int rt, int& tlo, int& thi, int& base) {
    const int t0 = (int)div_floor((int64_t)rt * ROWS, g.a.group);
    const int t1 = min(q.n - 1, (int)div_floor((int64_t)(rt + 1) * ROWS - 1, g.a.group));
    int lo1, hi0;
    seen_range(g.a, q.len, q.n, t0, tlo, hi0);
    seen_range(g.a, q.len, q.n, t1, lo1, thi);
    base = tlo / kTaKeys * kTaKeys;
    return thi > tlo ? (thi - base + kTaKeys - 1) / kTaKeys : 0;
}

// Where a cut at place `in` of a unit with T tiles and cost cu falls: before
// tile T * in / cu, or at the unit's begin (0) or end (T) where that leaves a
// piece of under kTaPiece tiles: its way through the workspace costs more than
// an uneven run.
constexpr int kTaPiece = 6;
__device__ __forceinline__ int ta_snap(int T, int in, int cu) {
    const int i = (int)div_floor((int64_t)T * in, max(1, cu));
    if (2 * i <= T) return i < kTaPiece ? 0 : T - i < kTaPiece ? T : i;
    return T - i < kTaPiece ? T : i < kTaPiece ? 0 : i;
}

// Moves a cut to where ta_snap puts it; sets the walk's sequence to the one
// that holds it.
template <int ROWS>
__device__ __forceinline__ int64_t ta_snapped(const TcAttnArgs& g, TaWalk& w, int c) {
    if (c == 0) return 0;
    if (c >= w.runs) return w.total;
    const int64_t x = w.cut(c);
    int s, rt, hk, in, lo, hi, base;
    int64_t sb;
    ta_find<ROWS>(g, x, false, s, sb);
    const TaSeq q = ta_seq<ROWS>(g, s);
    ta_unit(q, g.a.kv.n_heads, x - sb, rt, hk, in);
    const int T = ta_tiles<ROWS>(g, q, rt, lo, hi, base), cu = q.c0 + q.c1 * rt;
    const int i = ta_snap(T, in, cu);
    return i == 0 ? x - in : i >= T ? x - in + cu : x;
}

template <int ROWS>
__device__ __forceinline__ TaWalk ta_start(const TcAttnArgs& g) {
    TaWalk w;
    const int lane = threadIdx.x & 31, nh = g.a.kv.n_heads, n_seqs = g.a.batch.n_seqs;
    int64_t units = 0, cost = 0;
    for (int s = lane; s < n_seqs; s += 32) {
        const TaSeq q = ta_seq<ROWS>(g, s);
        units += (int64_t)q.tiles * nh;
        cost += q.before(q.tiles) * nh;
    }
    for (int x = 16; x; x >>= 1) {
        units += __shfl_xor_sync(0xFFFFFFFFu, units, x);
        cost += __shfl_xor_sync(0xFFFFFFFFu, cost, x);
    }
    w.total = cost;
    w.done = units == 0;
    w.k = 0;
    w.b0 = w.b = w.b1 = 0;
    if (w.done) return w;
    const int c = blockIdx.x;
    if (2 * units <= (int64_t)gridDim.x) {
        w.k = (int)(gridDim.x / (unsigned)units);
        w.runs = 0;
        const int u = c / w.k;
        w.done = u >= units;
        if (w.done) return w;
        ta_find<ROWS>(g, u, true, w.s, w.seq_base);
        w.q = ta_seq<ROWS>(g, w.s);
        w.b = u - w.seq_base;                 // the unit within the sequence
        return w;
    }
    w.runs = (int)gridDim.x;
    w.ratio = (double)cost / (double)w.runs;
    w.b0 = w.b = ta_snapped<ROWS>(g, w, c);
    w.b1 = ta_snapped<ROWS>(g, w, c + 1);
    w.done = w.b >= w.b1;
    if (w.done) return w;
    ta_find<ROWS>(g, w.b, false, w.s, w.seq_base);
    w.q = ta_seq<ROWS>(g, w.s);
    return w;
}

// The next part of this CTA's run; e.more = 0 at its end.
template <int ROWS>
__device__ __forceinline__ void ta_next(const TcAttnArgs& g, TaWalk& w, TaSeg& e) {
    e.more = 0;
    const int nh = g.a.kv.n_heads;
    int rt, hk, in = 0, base, i0, i1;
    if (w.done) return;
    if (w.k) {
        w.done = true;
        rt = (int)div_floor(w.b, nh);
        hk = (int)(w.b - (int64_t)rt * nh);
        const int T = ta_tiles<ROWS>(g, w.q, rt, e.tlo, e.thi, base);
        // As many pieces as leave a piece about as many tiles as there are
        // pieces to join.
        int k = 1;
        while (k < w.k && (k + 1) * (k + 1) <= T) ++k;
        const int p = (int)(blockIdx.x % (unsigned)w.k);
        if (p >= k) return;
        i0 = (int)((int64_t)T * p / k);
        i1 = (int)((int64_t)T * (p + 1) / k);
        e.c_lo = (int)blockIdx.x - p;
        e.pieces = k;
        e.slot = 2 * (int)blockIdx.x;
        e.slot0 = 2 * e.c_lo;
    } else {
        if (w.b >= w.b1) {
            w.done = true;
            return;
        }
        while (w.b >= w.seq_base + w.q.before(w.q.tiles) * nh && w.s + 1 < g.a.batch.n_seqs) {
            w.seq_base += w.q.before(w.q.tiles) * nh;
            w.q = ta_seq<ROWS>(g, ++w.s);
        }
        ta_unit(w.q, nh, w.b - w.seq_base, rt, hk, in);
        const int cu = w.q.c0 + w.q.c1 * rt;
        const int64_t ub = w.b - in, ue = ub + cu;
        const int64_t stop = w.b1 < ue ? w.b1 : ue;
        const int T = ta_tiles<ROWS>(g, w.q, rt, e.tlo, e.thi, base);
        i0 = in == 0 ? 0 : (int)div_floor((int64_t)T * in, cu);
        i1 = stop == ue ? T : (int)div_floor((int64_t)T * (stop - ub), cu);
        // The runs that begin inside the unit are consecutive; the run before
        // the first of them has the unit's first piece.
        int c = (int)((double)ub / w.ratio);
        c = max(0, min(c, w.runs - 1));
        while (c > 0 && w.cut(c) > ub) --c;
        while (c + 1 < w.runs && w.cut(c + 1) <= ub) ++c;
        ++c;
        int inside = 0, c_first = 0;
        for (; c < w.runs && w.cut(c) < ue; ++c) {
            const int i = ta_snap(T, (int)(w.cut(c) - ub), cu);
            if (i > 0 && i < T) {
                if (inside++ == 0) c_first = c;
            }
        }
        e.pieces = inside + 1;
        e.c_lo = inside ? c_first - 1 : (int)blockIdx.x;
        e.slot = 2 * (int)blockIdx.x + (w.b == w.b0 ? 0 : 1);
        e.slot0 = e.slot;
        if (inside) e.slot0 = 2 * e.c_lo + (ta_snapped<ROWS>(g, w, e.c_lo) < ub ? 1 : 0);
        w.b = stop;
    }
    e.more = 1;
    e.s = w.s;
    e.hk = hk;
    e.len = w.q.len;
    e.n = w.q.n;
    e.first = w.q.first;
    e.n_rows = (int)min((int64_t)ROWS, (int64_t)w.q.n * g.a.group - (int64_t)rt * ROWS);
    e.t0 = (int)div_floor((int64_t)rt * ROWS, g.a.group);
    e.g0 = (int)((int64_t)rt * ROWS - (int64_t)e.t0 * g.a.group);
    e.j0 = base + i0 * kTaKeys;
    e.nt = i1 - i0;
}

// A box of a 4-dimensional tensor map into shared memory; its bytes count on
// `bar`.  x is a multiple of 64 elements.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
                 : "memory");
}

// Whether both warps of pair `pair` (64 threads) are well; they meet here.
__device__ __forceinline__ bool pair_ok(int pair, bool ok) {
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.and.pred q, %2, 64, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"((uint32_t)ok), "r"(2 + pair) : "memory");
    return all != 0;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kTaThreads, 1) attn_tc_kernel(const __grid_constant__ TcAttnArgs g) {
    constexpr int NS = ta_slots(DP);
    constexpr int CH = DP / 8;
    constexpr uint32_t kHalf = kTaKeys * 128;            // one 64-element part of a 128-row tile
    constexpr uint32_t kTile = kHalf * (DP / 64);
    constexpr int ROWS = ta_rows(DP), NA = ROWS / 128;   // accumulators
    // One accumulator: the two groups of softmax warps share its rows, 64 keys
    // of a tile and half of the output's columns each.
    constexpr bool kPair = NA == 1;
    constexpr int NV = kPair ? 64 : 128;                 // scores of a thread
    constexpr int DO = kPair ? DP / 2 : DP;              // output columns of a thread
    constexpr int kLag = NS > 2 ? 2 : 1;                 // copies in flight behind the newest
    constexpr uint32_t kColO = 256;                      // TMEM columns: S at 0 and 128, sums from 256
    extern __shared__ uint8_t ta_raw[];
    const uint32_t raw0 = smem_addr(ta_raw);
    const uint32_t sQ = (raw0 + 1023u) & ~1023u;         // NA tiles of 128 rows
    const uint32_t sRing = sQ + NA * kTile;
    uint64_t* full = reinterpret_cast<uint64_t*>(ta_raw + (sRing - raw0) + NS * kTile);   // [NS]
    uint64_t* empty = full + NS;                         // [NS]
    uint64_t* qfull = empty + NS;                        // queries in place
    uint64_t* sfull = qfull + 1;                         // [2] S computed
    uint64_t* pfull = sfull + 2;                         // [2] P written
    uint64_t* phalf = pfull + 2;                         // [2] the first 64 keys of P written
    uint64_t* ofull = phalf + 2;                         // [2] the piece's sums complete
    uint64_t* pfull_seg = ofull + 2;                     // [kTaSegs] a part is told
    uint64_t* pempty_seg = pfull_seg + kTaSegs;          // [kTaSegs] every working warp is done with it
    uint64_t* idle = pempty_seg + kTaSegs;               // every product done
    uint32_t* tslot = reinterpret_cast<uint32_t*>(idle + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    volatile int* never = abort_flag + 1;                // stays 0
    volatile int* last_word = abort_flag + 2;
    volatile int* odd = abort_flag + 3;                  // [16] of the pieces with keys, in order: take it row by row
    float* meet = reinterpret_cast<float*>(ta_raw + (sRing - raw0) + NS * kTile + 512);   // [2][2][128], kPair

    const AttnArgs& a = g.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.kv.head_dim;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, kTaLoaders);
            mbar_init(empty + i, 1);
        }
        mbar_init(qfull, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 4);
            mbar_init(phalf + i, kPair ? 8 : 4);
            mbar_init(ofull + i, 1);
        }
        for (int i = 0; i < 16; ++i) odd[i] = 0;
        for (int i = 0; i < kTaSegs; ++i) {
            mbar_init(pfull_seg + i, 1);
            mbar_init(pempty_seg + i, 8 + 1 + kTaLoaders);
        }
        mbar_init(idle, 1);
        *abort_flag = *never = 0;
        fence_barrier_init();
    }
    if (warp == 8) tc_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    pdl_wait();
    pdl_launch_dependents();

    __shared__ TaSeg segs[kTaSegs];
    // Every working warp goes through the parts in order: told_part() waits for the
    // next one, drop() frees its place.
    uint32_t part_no = 0;
    auto told_part = [&]() {
        return __all_sync(0xFFFFFFFFu,
                          tc_wait_long(pfull_seg + part_no % kTaSegs, (part_no / kTaSegs) & 1, abort_flag));
    };
    auto drop = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(pempty_seg + part_no % kTaSegs);
        ++part_no;
    };
    auto give_up = [&]() {
        *abort_flag = 1;
        set_device_error(a.err, kDevTimeout);
    };

    if (warp >= 8) {
    // Registers go to the softmax, which holds a row of S: 256 x 184 + 128 x 120
    // of the 384 x 168 that the kernel starts with (checked at setup).
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp > 8) {
        if (warp < 9 + kTaLoaders) {
        // ---- copies ----
        const int lw = warp - 9;
        uint32_t u = 0;                                  // tiles begun
        uint32_t told = 0;                               // tiles whose arrival was signalled
        uint32_t look = 0, mark = 0;                     // of the tiles in flight: V tiles to look over, their pieces
        int seg_no = 0;
        bool ok = true;
        // This warp's 64 keys of a tile, two a lane; copies of a tile are
        // CH per 32 keys, `ch` of every 32 / CH-th row.
        constexpr int RPI = 32 / CH;                     // rows of a copy instruction
        const int ch = lane % CH;
        const uint32_t col = (uint32_t)(ch >> 3) * kHalf;
        auto place = [&](int rr) { return col + (uint32_t)(rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)); };
        auto signal = [&](uint32_t upto) {
            for (; told < upto; ++told) {
                const uint32_t st = told % NS;
                if (look >> (told & 7) & 1) {
                    // this thread's own chunks of a V tile
                    bool bad = false;
                    const uint32_t vt = sRing + st * kTile;
#pragma unroll 8
                    for (int x = 0; x < 64 / RPI; ++x)
                        bad |= any_nonfinite<T>(lds128(vt + place(64 * lw + x * RPI + lane / CH)));
                    if (bad) odd[(mark >> (4 * (told & 7))) & 15] = 1;
                    look &= ~(1u << (told & 7));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + st);
            }
        };
        while (ok && (ok = told_part())) {
            const TaSeg& e = segs[part_no % kTaSegs];
            if (!e.more) break;
            const int64_t ho = (int64_t)e.hk * a.kv.head_stride;
            // Keys that every row of the unit sees: tiles inside need no look.
            const int t0 = e.t0, t1 = e.t0 + (e.g0 + e.n_rows - 1) / a.group;
            int ilo, ihi, x0;
            seen_range(a, e.len, e.n, t1, ilo, x0);
            seen_range(a, e.len, e.n, t0, x0, ihi);
            const int j_first = e.j0, nt = e.nt, tlo = e.tlo, thi = e.thi, seq = e.s;
            const int hk = e.hk;
            // A tile that all rows see whole comes by tensor map, a page (or
            // its part) a box; the others by 16-byte copies, which leave keys
            // that no row sees zero.
            auto by_map = [&](int j) { return g.box && j >= ilo && j + kTaKeys <= ihi; };
            // Pages of the next tile, as read (not yet checked, so nothing waits
            // for them), with the rows in them: of boxes lane / parts (and that
            // of lane + 32), or of keys lane, lane + 32 of this warp's; row -1 for
            // a key that no row sees.
            const int parts = DP / 64, items = g.box ? kTaKeys / g.box * parts : 0;
            const int32_t* table = a.kv.table + (int64_t)seq * a.kv.table_stride;
            int pg[2], pr[2] = {-1, -1};
            auto lookup = [&](int j) {
                const bool map = by_map(j);
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int key = map ? j + (lane + 32 * y) / parts * g.box : j + 64 * lw + 32 * y + lane;
                    pr[y] = -1;
                    if (map ? lane + 32 * y < items : key >= tlo && key < thi) {
                        int page;
                        split_page(a.kv, key, page, pr[y]);
                        pg[y] = table[page];             // inside the columns: key < cap
                    }
                }
            };
            if (nt > 0) lookup(j_first);
            for (int i = 0; i < nt && ok; ++i) {
                const int j = j_first + i * kTaKeys;
                const bool mapped = by_map(j);
                int pgn[2], prn[2];                      // of this tile, checked
                int64_t off0 = -1, off1 = -1;
                bool page_bad = false;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    prn[y] = pr[y];
                    pgn[y] = pr[y] < 0 ? 0 : pg[y];
                    if ((unsigned)pgn[y] >= (unsigned)a.kv.n_pages) {
                        page_bad = true;
                        pgn[y] = 0;
                        if (!mapped) prn[y] = -1;
                    }
                }
                if (!mapped) {
                    if (prn[0] >= 0) off0 = (int64_t)pgn[0] * a.kv.page_stride + (int64_t)prn[0] * a.kv.token_stride + ho;
                    if (prn[1] >= 0) off1 = (int64_t)pgn[1] * a.kv.page_stride + (int64_t)prn[1] * a.kv.token_stride + ho;
                }
                if (page_bad) {
                    set_device_error(a.err, kDevIndex);
                    odd[seg_no & 15] = 1;
                }
                if (i + 1 < nt) lookup(j + kTaKeys);     // the next tile's pages, on their way meanwhile
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++u) {
                    const uint32_t st = u % NS;
                    if (u >= NS) {
                        const uint32_t par = ((u / NS) - 1) & 1;
                        if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(empty + st, par))) {
                            cp_async_wait<0>();          // nothing more to begin: hand over what is there
                            signal(u);
                            ok = __all_sync(0xFFFFFFFFu, tc_wait_long(empty + st, par, abort_flag));
                            if (!ok) break;
                        }
                    }
                    const uint32_t dst = sRing + st * kTile;
                    if (mapped) {
                        if (told < u) {
                            cp_async_wait<0>();
                            signal(u);
                        }
                        told = u + 1;
                        if (lane == 0) {
                            if (lw == 0) mbar_arrive_expect_tx(full + st, kTile);
                            else mbar_arrive(full + st);
                        }
                        __syncwarp();
                        if (lw == 0)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int it = lane + 32 * y, box = it / parts, part = it - box * parts;
                                if (it < items)
                                    tma_load_4d(dst + (uint32_t)part * kHalf + (uint32_t)(box * g.box) * 128u,
                                                kv ? &g.vmap : &g.kmap, 64 * part, prn[y], hk, pgn[y], full + st);
                            }
                        continue;
                    }
                    const T* src = static_cast<const T*>(kv ? a.kv.v : a.kv.k) + 8 * ch;
                    const bool chin = 8 * ch < D;
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int x = 0; x < CH; ++x) {
                            const int row = x * RPI + lane / CH;           // of 32
                            const int64_t o = __shfl_sync(0xFFFFFFFFu, y ? off1 : off0, row);
                            const bool in = o >= 0 && chin;
                            cp_async16(dst + place(64 * lw + 32 * y + row), in ? src + o : static_cast<const T*>(a.kv.k), in);
                        }
                    cp_async_commit();
                    if (kv && (j < ilo || j + kTaKeys > ihi)) {
                        look |= 1u << (u & 7);
                        mark = (mark & ~(15u << (4 * (u & 7)))) | ((uint32_t)(seg_no & 15) << (4 * (u & 7)));
                    }
                    if (u + 1 > told + kLag) {
                        cp_async_wait<kLag>();
                        signal(u + 1 - kLag);
                    }
                }
            }
            if (nt > 0) ++seg_no;
            drop();
        }
        cp_async_wait<0>();
        signal(u);
        if (!ok) give_up();
        } else {
            // ---- the walk over this CTA's parts ----
            TaWalk w = ta_start<ROWS>(g);
            for (uint32_t n = 0;; ++n) {
                TaSeg e;
                ta_next<ROWS>(g, w, e);
                if (n >= kTaSegs && !__all_sync(0xFFFFFFFFu, tc_wait_long(pempty_seg + n % kTaSegs, (n / kTaSegs - 1) & 1,
                                                                     abort_flag))) {
                    give_up();
                    break;
                }
                if (lane == 0) {
                    segs[n % kTaSegs] = e;
                    mbar_arrive(pfull_seg + n % kTaSegs);
                }
                __syncwarp();
                if (!e.more) break;
            }
        }
    } else {
        // ---- products ----
        uint32_t u = 0, np[2] = {0, 0};                  // ring tiles used, P's waited for
        int seg_no = 0;
        bool ok = true;
        while (ok && (ok = told_part())) {
            const TaSeg& e = segs[part_no % kTaSegs];
            if (!e.more) break;
            const int nt = e.nt;
            drop();
            if (nt == 0) continue;
            if (lane == 0) {
                auto wait = [&](uint64_t* bar, uint32_t par) {
                    if (ok && !tc_wait_long(bar, par, abort_flag)) ok = false;
                    tc_fence_after();
                };
                auto scores = [&](int acc, uint32_t st) {
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        const uint32_t o = (uint32_t)(kk >> 2) * kHalf + 32u * (kk & 3);
                        tc_mma_f16(tmem + 128u * acc, tc_sdesc_sw128(sQ + acc * kTile + o),
                                   tc_sdesc_sw128(sRing + st * kTile + o), g.idesc_s, kk != 0);
                    }
                    tc_commit(sfull + acc);
                };
                wait(qfull, seg_no & 1);
                wait(full + u % NS, (u / NS) & 1);
                if (ok) {
                    scores(0, u % NS);
                    if (NA > 1) scores(1, u % NS);
                    tc_commit(empty + u % NS);
                }
                for (int i = 0; i < nt && ok; ++i) {
                    const uint32_t uv = u + 1, uk = u + 2;
                    wait(full + uv % NS, (uv / NS) & 1);
#pragma unroll
                    for (int acc = 0; acc < NA; ++acc) {
                        auto weighted = [&](int kk) {
                            tc_mma_f16_ta(tmem + kColO + 128u * acc, tmem + 128u * acc + 8u * kk,
                                          tc_sdesc_sw128_nmajor(sRing + (uv % NS) * kTile + 2048u * kk, kHalf),
                                          g.idesc_o, (i | kk) != 0);
                        };
                        wait(phalf + acc, np[acc] & 1);
                        if (ok)
#pragma unroll
                            for (int kk = 0; kk < kTaKeys / 32; ++kk) weighted(kk);
                        wait(pfull + acc, np[acc] & 1);
                        ++np[acc];
                        if (ok) {
#pragma unroll
                            for (int kk = kTaKeys / 32; kk < kTaKeys / 16; ++kk) weighted(kk);
                            if (acc == NA - 1) tc_commit(empty + uv % NS);
                            if (i + 1 == nt) tc_commit(ofull + acc);
                        }
                        if (i + 1 < nt) {
                            if (acc == 0) wait(full + uk % NS, (uk / NS) & 1);
                            if (ok) {
                                scores(acc, uk % NS);
                                if (acc == NA - 1) tc_commit(empty + uk % NS);
                            }
                        }
                    }
                    u += 2;
                }
                if (!ok) give_up();
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
            ++seg_no;
        }
        if (lane == 0) {
            // The products in flight end before the tensor memory is freed.
            tc_commit(idle);
            tc_wait_long(idle, 0, never);
        }
        __syncwarp();
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ---- softmax: a thread has row `row` of accumulator `acc`, or the part
        // `part` of the one accumulator's row: keys 64 part .. + 64, columns
        // 128 part .. + 128 ----
        const int grp = warp >> 2, acc = kPair ? 0 : grp, part = kPair ? grp : 0, row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + 128u * acc + 64u * part, tO = tmem + lanes + kColO + 128u * grp;
        const uint32_t tP = tmem + lanes + 128u * acc + 32u * part;
        uint32_t ns = 0;                                 // S's waited for
        int q_no = 0;                                    // pieces with keys
        bool ok = true;
        const bool neg = a.scale_log2 < 0.f, flat = a.scale_log2 == 0.f;
        const float sc = flat ? 1.f : fabsf(a.scale_log2);
        for (;; drop()) {
            // The eight warps go on, or end, together.
            if (!told_part()) ok = false;
            if (!ok) give_up();
            if (!all_of<256>(ok)) break;
            const TaSeg& e = segs[part_no % kTaSegs];
            if (!e.more) break;
            const int xr = acc * 128 + row;              // of the unit's rows
            const int cb = part * DO;                    // first output column
            if (e.nt > 0) {
                // Queries of this accumulator: a thread's chunk of every
                // kHands / CH-th row.
                constexpr int kHands = kPair ? 256 : 128;    // threads of an accumulator's queries
                const int hand = (int)threadIdx.x % kHands, ch = hand % CH;
#pragma unroll 4
                for (int rr = hand / CH; rr < 128; rr += kHands / CH) {
                    const int x = acc * 128 + rr, gx = e.g0 + x, t = gx / a.group, gh = gx - t * a.group;
                    const bool in = x < e.n_rows && 8 * ch < D;
                    const T* src = static_cast<const T*>(a.q) +
                                   (in ? (e.first + e.t0 + t) * a.q_stride + (int64_t)(e.hk * a.group + gh) * D + 8 * ch : 0);
                    cp_async16(sQ + acc * kTile + (uint32_t)(ch >> 3) * kHalf +
                                   (uint32_t)(rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)),
                               src, in);
                }
                cp_async_commit();
                cp_async_wait<0>();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
                ++q_no;
            }
            // Keys that this row sees, and that all rows of the warp see.
            const bool real = xr < e.n_rows;
            const int tr = (e.g0 + xr) / a.group;        // its token, from the unit's first
            int lo = 0, hi = 0;
            if (real) seen_range(a, e.len, e.n, e.t0 + tr, lo, hi);
            int wlo = real ? lo : 0, whi = real ? hi : INT32_MAX;
            for (int x = 16; x; x >>= 1) {
                wlo = max(wlo, __shfl_xor_sync(0xFFFFFFFFu, wlo, x));
                whi = min(whi, __shfl_xor_sync(0xFFFFFFFFu, whi, x));
            }
            T* out = static_cast<T*>(a.out) + (e.first + e.t0 + tr) * a.o_stride +
                     (int64_t)(e.hk * a.group + (e.g0 + xr - tr * a.group)) * D;
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < e.nt && ok; ++i) {
                ok = __all_sync(0xFFFFFFFFu, tc_wait_long(sfull + acc, ns & 1, abort_flag));
                ++ns;
                if (!kPair && !ok) break;                // (a pair ends together)
                tc_fence_after();
                float v[NV / 32][32];                    // the row's scores (its part's)
#pragma unroll
                for (int x = 0; x < NV / 32; ++x) tc_ld32(tS + 32u * x, v[x]);
#pragma unroll
                for (int x = 0; x < NV / 32; ++x) tc_wait_ld(v[x]);
                const int j = e.j0 + i * kTaKeys;
                if (neg || flat) {
#pragma unroll
                    for (int x = 0; x < NV / 32; ++x)
#pragma unroll
                        for (int y = 0; y < 32; ++y) v[x][y] = neg ? -v[x][y] : 0.f * v[x][y];
                }
                if (j < wlo || j + kTaKeys > whi) {
                    const int c0 = lo - j - 64 * part, c1 = hi - j - 64 * part;
#pragma unroll
                    for (int x = 0; x < NV / 32; ++x)
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            if (32 * x + y < c0 || 32 * x + y >= c1) v[x][y] = -INFINITY;
                }
                float mx[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    mx[x] = v[0][x];
#pragma unroll
                    for (int y = 8; y < NV; y += 8) mx[x] = fmaxf(mx[x], v[(x + y) >> 5][(x + y) & 31]);
                }
                float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                  fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sc;
                if (kPair) {
                    // The row's other part, read as well by now: P may go into
                    // S's place.
                    float* mt = meet + 256 * (ns & 1);
                    mt[128 * part + row] = top;
                    tc_fence_before();
                    ok = pair_ok(warp & 3, ok);
                    if (!ok) break;
                    tc_fence_after();
                    top = fmaxf(mt[row], mt[128 + row]);
                }
                float f = 1.f;
                if (i == 0) {
                    m = top;
                } else if (top > m + 8.f) {
                    f = exp2f(m - top);
                    m = top;
                    l *= f;
                }
                if (__any_sync(0xFFFFFFFFu, f != 1.f)) {
                    // S came after the last P V, so the sums are at rest.
#pragma unroll 1
                    for (int x = 0; x < DO / 16; ++x) {
                        uint32_t o[16];
                        tc_ld16(tO + 16u * x, o);
#pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                        tc_st16(tO + 16u * x, o);
                    }
                }
                if (kPair && part == 1) {                // its columns are ready for the product
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(phalf + acc);
                }
                const float mu = m == -INFINITY ? 0.f : m;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                const float2 sc2 = make_float2(sc, sc), mu2 = make_float2(-mu, -mu);
#pragma unroll
                for (int x = 0; x < NV / 32; ++x) {
                    uint32_t pw[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        float2 t = ffma2(make_float2(v[x][2 * y], v[x][2 * y + 1]), sc2, mu2);
                        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(t.x));
                        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(t.y));
                        sum[y & 1] = fadd2(sum[y & 1], t);
                        pw[y] = Elem<T>::pack(t.x, t.y);
                    }
                    tc_st16(tP + 16u * x, pw);
                    if (!kPair && x == 1) {
                        // The first 64 keys' weights: their product may begin.
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(phalf + acc);
                    }
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive((kPair && part == 0 ? phalf : pfull) + acc);
            }
            if (ok && e.nt > 0) {
                ok = __all_sync(0xFFFFFFFFu, tc_wait_long(ofull + acc, (q_no - 1) & 1, abort_flag));
                tc_fence_after();
            }
            if (kPair) {                                 // the row's weights, both parts'
                float* mt = meet + 256 * ((ns + 1) & 1);
                mt[128 * part + row] = l;
                ok = pair_ok(warp & 3, ok);
                l = mt[row] + mt[128 + row];
            }
            // The copying warps' marks on this piece reach here through the
            // products' barriers; they are at most five pieces ahead.
            const bool rows_apart = e.nt > 0 && odd[(q_no - 1) & 15] != 0;
            float* slot = g.ws + (int64_t)e.slot * ta_slot(DP);
            if (e.pieces == 1) {
                if (!rows_apart) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
                    for (int x = 0; x < DO / 32; ++x) {
                        float o[32];
                        if (e.nt > 0) {
                            tc_ld32(tO + 32u * x, o);
                            tc_wait_ld(o);
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            float v[8];
#pragma unroll
                            for (int z = 0; z < 8; ++z) v[z] = e.nt > 0 ? o[8 * y + z] * inv : 0.f;
                            if (real && cb + 32 * x + 8 * y < D)
                                *reinterpret_cast<uint4*>(out + cb + 32 * x + 8 * y) = pack8<T>(v);
                        }
                    }
                }
            } else {
                // A piece: sums as [column / 4][row][4], so a warp's stores are
                // 512 contiguous bytes.  The mark for a row-by-row unit is a
                // weights' sum of -1.
                const int rr = xr;
#pragma unroll
                for (int x = 0; x < DO / 32; ++x) {
                    float o[32];
                    if (e.nt > 0) {
                        tc_ld32(tO + 32u * x, o);
                        tc_wait_ld(o);
#pragma unroll
                        for (int y = 0; y < 8; ++y)
                            *reinterpret_cast<float4*>(slot + ((cb / 4 + 8 * x + y) * ROWS + rr) * 4) =
                                make_float4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
                    }
                }
                if (part == 0) {
                    slot[ROWS * DP + rr] = m;
                    slot[ROWS * DP + ROWS + rr] = rows_apart ? -1.f : l;
                }
                __threadfence();
                bar_first256();
                if (threadIdx.x == 0) *last_word = atom_add_acq_rel_gpu(g.cnt + e.c_lo, 1) == e.pieces - 1;
                bar_first256();
            }
            tc_fence_before();           // the sums were read: the next piece's products may come
            bool apart = e.pieces == 1 && rows_apart;
            if (e.pieces > 1 && *last_word) {
                __threadfence();
                if (threadIdx.x == 0) g.cnt[e.c_lo] = 0;
                // Piece 0 may be in its CTA's second slot, the others are in
                // their CTAs' first.
                auto piece = [&](int p) {
                    return g.ws + (int64_t)(p ? 2 * (e.c_lo + p) : e.slot0) * ta_slot(DP) + xr * 4;
                };
                constexpr int kM = ROWS * DP;         // maxima, then sums
                float top = -INFINITY, sum = 0.f;
#pragma unroll 4
                for (int p = 0; p < e.pieces; ++p) {
                    const float* sp = piece(p) - 3 * xr + kM;
                    top = fmaxf(top, __ldcg(sp));
                    if (__ldcg(sp + ROWS) == -1.f) apart = true;
                }
                const float mu = top == -INFINITY ? 0.f : top;
#pragma unroll 4
                for (int p = 0; p < e.pieces; ++p) {
                    const float* sp = piece(p) - 3 * xr + kM;
                    sum += exp2f(__ldcg(sp) - mu) * __ldcg(sp + ROWS);
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
                for (int x = 0; x < DO / 64; ++x) {
                    float4 o[16];
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                    for (int p = 0; p < e.pieces; ++p) {
                        const float* sp = piece(p);
                        const float wt = exp2f(__ldcg(sp - 3 * xr + kM) - mu);
                        float4 v[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            v[y] = __ldcg(reinterpret_cast<const float4*>(sp + (cb / 4 + 16 * x + y) * (4 * ROWS)));
                        if (wt == 0.f) continue;         // no keys: the slot's sums were not written
#pragma unroll
                        for (int y = 0; y < 16; ++y) {
                            o[y].x += wt * v[y].x;
                            o[y].y += wt * v[y].y;
                            o[y].z += wt * v[y].z;
                            o[y].w += wt * v[y].w;
                        }
                    }
                    if (real)
#pragma unroll
                        for (int y = 0; y < 16; ++y)
                            if (cb + 64 * x + 4 * y < D)
                                *reinterpret_cast<uint2*>(out + cb + 64 * x + 4 * y) =
                                    make_uint2(Elem<T>::pack(o[y].x * inv, o[y].y * inv),
                                               Elem<T>::pack(o[y].z * inv, o[y].w * inv));
                }
            }
            bar_first256();               // everyone has read this piece's mark and the word above
            if (threadIdx.x == 0 && e.nt > 0) odd[(q_no - 1) & 15] = 0;
            if (apart) {
                for (int x = warp; x < e.n_rows; x += 8) {
                    const int t = (e.g0 + x) / a.group;
                    int l0, h0;
                    seen_range(a, e.len, e.n, e.t0 + t, l0, h0);
                    attend_row<T>(a, e.s, e.first + e.t0 + t, e.hk * a.group + (e.g0 + x - t * a.group), l0, h0);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tc_dealloc(tmem, 512);
    }
}

}  // namespace q4
