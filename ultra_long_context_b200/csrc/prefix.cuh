// prefix.cuh -- how the shared-prefix decode divides its work: shared by its kernels (prefix_few.cu,
// prefix_wide.cu) and the join of their partials (prefix.cu).
//
// For a query row q and its visible keys, out = sum_k exp(s_k - m) v_k / sum_k exp(s_k - m) with
// s = scale q.k. The keys are cut into tiles of 128 (two pages). A SEGMENT is a run of tiles of one page list
// (the prefix's, or a request's own) for one key head and up to 64 or 256 query rows: rows of the whole batch that
// read the key head, for the prefix; the request's own rows, for its own pages. Over a segment a row keeps a reference m
// (see prefix_few.cu), its sum l = sum exp(s - m) and output O = sum exp(s - m) v, and the segments' (m, l, O) of a row
// are joined at the end. So a prefix page is read once for as many rows, and both kinds of work are the same.
#pragma once

#include <cuda.h>

#include "launch.h"
#include "tc.cuh"

namespace hsa {

constexpr int kPfTile = 128;      // keys per tile = 2 pages
constexpr int kPfFewRows = 64;    // rows per segment at most: in the few-rows kernel,
constexpr int kPfWideRows = 256;  // in the wide kernel
constexpr int kPfCtas = 148;      // at most: one per SM; the workspace is sized for it
constexpr int kPfItems = 4 * kPfCtas;  // prefix segments at most (or one per head and row group)
// Tiles that are summed in the products' accumulator at most. It adds by cutting: 2^-24 of the sum are lost with each product, eight
// a tile (V = 1: 0.8% over 14,000 tiles, 8% over 114,000). A longer run is walked in pieces, each of which is added to
// the partial that is there, in fp32 by rounding. 512 tiles lose some 2^-12, a sixteenth of the result's rounding, and
// take 300 us and more, so that a piece's start and end do not show. Even, so that every piece's items alternate between the
// wide kernel's streams alike.
constexpr int kPfPiece = 512;
// Costs in half tiles: a tile, and what a segment's start and end take beside its tiles, some 5000 cycles (24 requests x 4
// tokens over 20K: 35.7 us; with 3 and 4 for the two 36.2, with 3 and 5 40.8; other shapes within 1%)
constexpr int kPfTileCost = 2, kPfPrefixCost = 5, kPfOwnCost = 5;

// a / b for a >= 0, b > 0, in 32 bits where they suffice (a 64-bit division takes several times as long)
__device__ __forceinline__ int64_t pf_div(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// The division of one kernel's work; every CTA computes the same, CTA 0 stores it for the join.
//   prefix: per key head and row group (a unit), `nsplit` runs of `run` tiles; segment i = run i / units of unit
//   i % units goes to CTA i % ctas, so that the row groups of one run, which read the same keys, do so at about the
//   same time, through L2;
//   own: the stretches of all (request, key head, row group), weight = cost of their tiles + kPfOwnCost each, laid
//   end to end on an axis, and the axis cut into one interval per CTA such that prefix and own work
//   add up evenly: the first `lo_ctas` CTAs, which have one prefix segment more, get `cap_lo`, the others `cap_hi`.
struct PfPlan {
    int ctas, P, tiles, run, nsplit, items, lo_ctas, pad;  // P: the prefix's tokens
    int64_t cap_lo, cap_hi, axis;
    __device__ int64_t start(int i) const {
        const int64_t x = i <= lo_ctas ? i * cap_lo : lo_ctas * cap_lo + (i - lo_ctas) * cap_hi;
        return x < axis ? x : axis;
    }
    __device__ int cta_of(int64_t x) const {
        return x < lo_ctas * cap_lo ? (int)pf_div(x, cap_lo) : lo_ctas + (int)pf_div(x - lo_ctas * cap_lo, cap_hi);
    }
};

// Sizes that follow from the call's arguments alone.
struct PfDims {
    bool wide;             // the prefix goes to the wide kernel (the requests' own pages to the few-rows kernel always)
    int Rp, gp, Rgp;       // prefix rows per key head, in Rgp groups of gp
    int Ro, Rgo;           // own rows per request and key head, in groups of kPfFewRows
    int strideP, strideO;  // rows of one segment's partials (in the wide kernel, two streams may each keep one of the same rows)
    int max_items, max_slots, blocks;  // blocks: of 32 requests
    // Which kernel ends the prefix sooner? A tile of 128 keys takes the few-rows kernel 0.94 us (D = 128; 0.77 with D = 64)
    // for 64 rows, the wide one 2.05 us (1.65) for 256 and 1.4 us (1.07) for up to 128, and that is a launch of its own with
    // larger tiles to fill: 15 us (8). Both sides measured, D = 128: 512 rows x 4 heads over 14208 / 28416 / 56832 tokens
    // 38 / 61 / 110 us and 43 / 56 / 81, 1024 rows 66 / 110 / 208 and 63 / 89 / 135, 128 rows x 8 heads over 28416 / 59136
    // 42 / 67 and 48 / 66; D = 64: 512 rows 36 / 54 / 93 and 37 / 46 / 65. The tiles are those of the table, since the
    // length is not known here: a short prefix in a long table pays for the wide kernel's start (128 rows x 8 heads over 2048
    // tokens 21 to 25 us with a table of their size, 29 to 31 with one for 2^20).
    static bool pf_wide(int Rp, int Hkv, int D, int tiles) {
        const bool d128 = D == 128;
        const double per_sm = (double)Hkv * tiles / kPfCtas;
        const double few = per_sm * ((Rp + kPfFewRows - 1) / kPfFewRows) * (d128 ? 0.94 : 0.77);
        const double wide_tile = Rp > kPfTile ? (d128 ? 2.05 : 1.65) : (d128 ? 1.4 : 1.07);
        const double wide = (d128 ? 15.0 : 8.0) + per_sm * ((Rp + kPfWideRows - 1) / kPfWideRows) * wide_tile;
        return Rp > kPfFewRows && wide < few;
    }
    PfDims(int B, int H, int Hkv, int Tq, int D, int max_prefix_pages) {
        Ro = H / Hkv * Tq;
        Rp = B * Ro;
        const int tiles = (max_prefix_pages + 1) / 2;
        wide = pf_wide(Rp, Hkv, D, tiles);
        gp = wide ? kPfWideRows : kPfFewRows;
        Rgp = (Rp + gp - 1) / gp;
        Rgo = (Ro + kPfFewRows - 1) / kPfFewRows;
        strideP = wide ? kPfWideRows : Rp < kPfFewRows ? Rp : kPfFewRows;
        strideO = Ro < kPfFewRows ? Ro : kPfFewRows;
        const int units = Hkv * Rgp;
        int ns = kPfItems / units;
        ns = ns < 1 ? 1 : ns;
        ns = ns < tiles ? ns : tiles;
        max_items = units * ns;
        max_slots = B * Hkv * Rgo + kPfCtas;
        blocks = (B + 31) / 32;
    }
};

struct PfWork {
    int32_t *err;
    PfPlan *planP, *planO;   // of the kernel that takes the prefix / the own pages
    int32_t *status;         // [2][kPfCtas]: a kernel's CTAs; nonzero where a wait ran out
    int32_t *bcum;           // [blocks + 1] weights of the requests before each block
    float *Op, *mlp;         // prefix partials [max_items][strideP][D], [..][2] (m * scale * log2(e), l)
    float *Oo, *mlo;         // own partials [max_slots][strideO][D], [..][2]
};

__device__ __forceinline__ int64_t pf_clamp_len(int64_t n, int pages) { return min(n, (int64_t)pages * kChunk); }
__device__ __forceinline__ int pf_tiles(int64_t n) { return n > 0 ? (int)((n + kPfTile - 1) / kPfTile) : 0; }
__device__ __forceinline__ int pf_weight(int64_t n) { return n > 0 ? kPfTileCost * pf_tiles(n) + kPfOwnCost : 0; }
// Tile boundary of a place on a stretch: 0 at its start, the number of tiles at its end, never decreasing.
__device__ __forceinline__ int pf_tile_at(int64_t at) { return (int)(max(at - kPfOwnCost + kPfTileCost - 1, (int64_t)0) / kPfTileCost); }

struct PfSeg {
    int h, b;            // key head; request (own segments; -1: prefix)
    int r0, nr;          // its rows among the key head's (prefix) or the request's (own)
    int tile0, nt;       // run of tiles
    int len;             // tokens of the sequence
    int part;            // index of its partials; ~index in a later piece of its run, which is added to what stands there
    const int32_t *table;
    __device__ bool added() const { return part < 0; }
    __device__ int place() const { return part < 0 ? ~part : part; }
};

// Which of the 32 pages of a segment's tiles t .. t + 15 are there? A warp's lanes look one up each and vote; fetch() of the
// next 16 tiles comes that much earlier. (Handed over by the copying warp, through shared memory, the answer was 400 cycles
// late, behind the other warps' exponentials; so were lookups for every tile by every thread.)
struct PfPages {
    const int32_t *table;
    int end, num_pages;  // the first page that is not the segment's
    __device__ PfPages(const PfSeg &s, int pages) : table(s.table), end(min((s.len + kChunk - 1) / kChunk, 2 * (s.tile0 + s.nt))), num_pages(pages) {}
    __device__ int fetch(int tile) const {  // (in the sequence)
        const int p = 2 * tile + (threadIdx.x & 31);
        return p < end ? table[p] : -1;
    }
    __device__ uint32_t there(int id) const { return __ballot_sync(0xffffffffu, id >= 0 && id < num_pages); }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)), "l"(reinterpret_cast<uint64_t &>(c)));
    return reinterpret_cast<float2 &>(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return reinterpret_cast<float2 &>(r);
}

// What the copying warp, which walks the segments, announces of one to the other warps, through a ring in shared
// memory; nr = 0 ends the walk.
constexpr int kPfRing = 4;
struct PfNote {
    PfSeg s;
    int n0;  // number of its first tile among the CTA's
    int i0;  // wide: number of its first item (a tile for one of the two streams) among the CTA's
};

// Walks a CTA's segments; by a whole warp, its lanes holding the lengths of a block of 32 requests.
struct PfWalk {
    const PrefixArgs &a;
    const PfPlan &p;
    const int32_t *bcum;
    const PfDims &d;
    int item, lane, blk, len, weight, before;
    int rest;  // tiles of the present run behind its piece
    int64_t x, end;
    __device__ PfWalk(const PrefixArgs &a_, const PfPlan &p_, const int32_t *bcum_, const PfDims &d_)
        : a(a_), p(p_), bcum(bcum_), d(d_), item(blockIdx.x), lane(threadIdx.x & 31), blk(-1), len(0), weight(0), before(0), rest(0),
          x(p_.start(blockIdx.x)), end(p_.start(blockIdx.x + 1)) {}
    __device__ void load_block(int k) {
        blk = k;
        const int b = 32 * k + lane;
        const int64_t n = b < a.B ? pf_clamp_len(a.own_len[b], a.max_pages) : -1;
        len = n > 0 ? (int)n : 0;
        weight = pf_weight(n);
        int sum = weight;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        before = bcum[k] + sum - weight;
    }
    // `s`: the segment before, and then the next one
    __device__ bool next(PfSeg &s) {
        if (rest > 0) {
            s.tile0 += s.nt;
            s.part = ~s.place();
            s.nt = min(rest, kPfPiece);
            rest -= s.nt;
            return true;
        }
        if (!next_run(s)) return false;
        if (s.nt > kPfPiece) {
            rest = s.nt - kPfPiece;
            s.nt = kPfPiece;
        }
        return true;
    }
    __device__ bool next_run(PfSeg &s) {
        if (item < p.items) {
            const int units = a.Hkv * d.Rgp, k = item / units, u = item - k * units;
            s.h = d.Rgp == 1 ? u : u / d.Rgp;
            s.b = -1;
            s.r0 = (u - s.h * d.Rgp) * d.gp;
            s.nr = min(d.gp, d.Rp - s.r0);
            s.tile0 = k * p.run;
            s.nt = min(p.run, p.tiles - s.tile0);
            s.len = p.P;
            s.part = item;
            s.table = a.prefix_table;
            item += p.ctas;
            return true;
        }
        const int hr_n = a.Hkv * d.Rgo;
        while (x < end) {
            const int xw = (int)pf_div(x, hr_n);  // on the axis of the requests' weights alone
            int lo = 0, hi = d.blocks;       // the block that holds it (blocks of no weight are passed over)
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (bcum[m] <= xw) lo = m;
                else hi = m;
            }
            if (lo != blk) load_block(lo);
            const unsigned at_or_before = __ballot_sync(0xffffffffu, weight > 0 && before <= xw);
            const int l = 31 - __clz(at_or_before);
            const int w = __shfl_sync(0xffffffffu, weight, l);
            const int64_t rest = x - (int64_t)__shfl_sync(0xffffffffu, before, l) * hr_n;
            s.len = __shfl_sync(0xffffffffu, len, l);
            const int hr = (int)pf_div(rest, w), from = (int)(rest - (int64_t)hr * w);
            const int to = (int)min((int64_t)w, from + (end - x));
            x += to - from;
            const int t0 = pf_tile_at(from), t1 = pf_tile_at(to);
            if (t1 <= t0) continue;
            s.b = 32 * lo + l;
            s.h = hr / d.Rgo;
            s.r0 = hr % d.Rgo * kPfFewRows;
            s.nr = min(kPfFewRows, d.Ro - s.r0);
            s.tile0 = t0;
            s.nt = t1 - t0;
            s.part = s.b * hr_n + hr + (int)blockIdx.x;
            s.table = a.block_table + (int64_t)s.b * a.max_pages;
            return true;
        }
        return false;
    }
};

// Copies the q rows `first` .. of a segment to dst(0, chunk), dst(1, chunk), .. below `end` by cp.async, by a whole warp; zeros for the
// rows from `rows` on, which are nobody's, and for the empty rows of a padded batch: whatever stands there must not look
// like a large logit. A lane looks up one row of 32 (row by row, each behind its request's length, 128 rows took a
// warp 10600 cycles).
template <int D, class Dst>
__device__ __forceinline__ void pf_copy_q(const PrefixArgs &a, const PfDims &d, const PfSeg &s, int first, int rows, int end, Dst dst) {
    constexpr int CPR = D / 8, RPW = 32 / CPR;  // 16-byte chunks per row, rows per warp-wide copy
    const int lane = threadIdx.x & 31, rsub = lane / CPR, ch = lane % CPR;
    for (int r0 = 0; r0 < end; r0 += 32) {
        const int r = s.r0 + first + r0 + lane;
        int row = -1;  // rows stay below 2^31 / D
        if (r0 + lane < rows) {
            const int request = s.b < 0 ? r / d.Ro : s.b, rem = s.b < 0 ? r - request * d.Ro : r;
            if (s.b >= 0 || a.own_len[request] >= 0) row = (request * a.Hkv + s.h) * d.Ro + rem;
        }
#pragma unroll
        for (int j = 0; j < CPR; ++j) {
            const int rr = j * RPW + rsub, from = __shfl_sync(0xffffffffu, row, rr);
            if (r0 + rr < end)
                cp_async16_u32(dst(r0 + rr, ch), from >= 0 ? a.q + (int64_t)from * D + ch * 8 : a.q, from >= 0 ? 16 : 0);
        }
    }
}

// Two partials of a row: the reference of their sum and the factors that bring each to it. (0 for one that has seen nothing: what
// stands there may be anything.)
struct PfSum {
    float m, f0, f1;
    __device__ PfSum(float m0, float m1)
        : m(fmaxf(m0, m1)), f0(m0 > -INFINITY ? ex2_approx(m0 - m) : 0.0f), f1(m1 > -INFINITY ? ex2_approx(m1 - m) : 0.0f) {}
};
__device__ __forceinline__ float pf_add(float x0, float f0, float x1, float f1) {
    return (f0 > 0.0f ? f0 * x0 : 0.0f) + (f1 > 0.0f ? f1 * x1 : 0.0f);
}

// 32 bytes in one store: a whole sector, where two of 16 make the memory system handle it twice.
__device__ __forceinline__ void pf_store8(float *p, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// Tokens of the segment's sequence that its row rr sees. The empty rows of a padded batch compute something that
// is never read (no limit, so that they do not slow the others' tiles).
__device__ __forceinline__ int pf_limit(const PrefixArgs &a, const PfSeg &s, const PfDims &d, int rr) {
    const int r = s.r0 + rr;
    if (s.b >= 0) return max(0, s.len - a.Tq + (a.Tq == 1 ? 0 : r % a.Tq) + 1);
    const int64_t own = pf_clamp_len(a.own_len[r / d.Ro], a.max_pages);
    if (own < 0) return INT32_MAX;
    return max(0, s.len + min((int)own - a.Tq + (a.Tq == 1 ? 0 : r % d.Ro % a.Tq) + 1, 0));  // prefix tokens not seen
}
// A bound from below for all rows of the segment.
__device__ __forceinline__ int pf_min_limit(const PrefixArgs &a, const PfSeg &s) { return max(0, s.len - a.Tq + 1); }

// The division of the work, by the whole block of NT threads, into shared memory: the plan and bcum.
// `idle` is run by the other warps while the first makes the plan.
template <int NT, class Idle>
__device__ void pf_schedule(const PrefixArgs &a, const PfDims &d, bool prefix, bool own, PfPlan *plan, int32_t *bcum, Idle idle) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ctas = gridDim.x;
    for (int k = warp; k < d.blocks; k += NT / 32) {
        const int b = 32 * k + lane;
        const int w = own && b < a.B ? pf_weight(pf_clamp_len(a.own_len[b], a.max_pages)) : 0;
        const int sum = __reduce_add_sync(0xffffffffu, w);
        if (lane == 0) bcum[k] = sum;
    }
    int64_t plen = 0;
    if (warp == 0 && prefix && a.max_prefix_pages > 0) plen = pf_clamp_len(a.prefix_len[0], a.max_prefix_pages);
    __syncthreads();
    if (warp == 0) {
        int total = 0;
        for (int k0 = 0; k0 < d.blocks; k0 += 32) {
            const int k = k0 + lane, w = k < d.blocks ? bcum[k] : 0;
            int x = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (k < d.blocks) bcum[k] = total + x - w;
            total += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) bcum[d.blocks] = total;
        const int64_t axis = (int64_t)total * a.Hkv * d.Rgo;
        const int P = plen > 0 ? (int)plen : 0, tiles = pf_tiles(P);
        const int units = a.Hkv * d.Rgp;
        PfPlan p{};
        p.ctas = ctas;
        p.P = P;
        p.tiles = tiles;
        p.axis = axis;
        p.run = 1;
        p.nsplit = 1;
        if (tiles > 0) {
            // a number of runs per lane: 1 .. 16, and what fills 1/4 .. 4 waves; the one that ends the work soonest,
            // both kinds of it counted (fewer runs win a tie). An estimate: in floats, whose quotients are quick
            const int ns_max = min(max(kPfItems / units, 1), tiles);
            const float quarter = (float)ctas * 0.25f / (float)units;
            const int ns = min(max(lane < 16 ? lane + 1 : (int)((float)(lane - 15) * quarter), 1), ns_max);
            const float run = ceilf(__fdividef((float)tiles, (float)ns) - 1e-3f), cost = kPfTileCost * run + kPfPrefixCost;
            const float items = (float)units * ceilf(__fdividef((float)tiles, run) - 1e-3f);
            const float waves = ceilf(__fdividef(items, (float)ctas) - 1e-3f) * cost;
            const float even = __fdividef(items * cost + (float)axis, (float)ctas);
            // costs are positive, so their bits order as they do; the last five say whose it is
            const uint32_t key = __reduce_min_sync(0xffffffffu, (__float_as_uint(fmaxf(waves, even)) & ~31u) | (uint32_t)lane);
            const int best = __shfl_sync(0xffffffffu, ns, (int)(key & 31u));
            p.run = (tiles + best - 1) / best;
            p.nsplit = (tiles + p.run - 1) / p.run;
            p.items = units * p.nsplit;
        }
        const int64_t cost = kPfTileCost * p.run + kPfPrefixCost;
        const int waves = p.items / ctas;
        p.lo_ctas = p.items - waves * ctas;
        const int64_t pc_hi = waves * cost, pc_lo = pc_hi + cost;
        const int hi_ctas = ctas - p.lo_ctas;
        const int64_t alone = pf_div(axis + hi_ctas - 1, hi_ctas);
        if (pc_hi + alone <= pc_lo) {  // the CTAs with a prefix segment less take all of it
            p.cap_lo = 0;
            p.cap_hi = alone;
        } else {
            const int64_t share = pf_div(axis + p.lo_ctas * pc_lo + hi_ctas * pc_hi + ctas - 1, ctas);
            p.cap_lo = share - pc_lo;
            p.cap_hi = share - pc_hi;
        }
        if (lane == 0) *plan = p;
    } else {
        idle(warp);
    }
    __syncthreads();
}

// Starts K and V of the two tiles that CTA `blockIdx.x` is likely to be given first on their way into L2: those that it gets if
// the prefix is cut into as many runs as make one segment per CTA (16 requests over 32K 33.9 -> 33.0 us; four tiles 33.6). A
// wrong guess costs nothing but their early arrival.
template <int D>
__device__ __forceinline__ void pf_prefetch_first(const PrefixArgs &a, const PfDims &d, int64_t plen, int ctas) {
    const int lane = threadIdx.x & 31, units = a.Hkv * d.Rgp, tiles = pf_tiles(plen), runs = max(ctas / units, 1);
    const int k = (int)blockIdx.x / units, h = ((int)blockIdx.x - k * units) / d.Rgp, run = (tiles + runs - 1) / runs;
    const int p = 2 * k * run + (lane >> 1);
    if (lane >= 8 || lane >= 4 * run || p >= (plen + kChunk - 1) / kChunk) return;
    const int id = a.prefix_table[p];
    if (id < 0 || id >= a.num_pages) return;
    const uint16_t *src = (lane & 1 ? a.Vp : a.Kp) + ((int64_t)id * a.Hkv + h) * (kChunk * D);
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(kChunk * D * 2) : "memory");
}

// For the join: what this kernel's CTA 0 knows.
template <int NT>
__device__ void pf_publish(const PfDims &d, bool prefix, bool own, const PfPlan *plan, const int32_t *bcum, const PfWork &w) {
    if (blockIdx.x != 0) return;
    if (own)
        for (int k = threadIdx.x; k <= d.blocks; k += NT) w.bcum[k] = bcum[k];
    if (threadIdx.x == 0 && prefix) *w.planP = *plan;
    if (threadIdx.x == 0 && own) *w.planO = *plan;
}

__device__ __forceinline__ void pf_prefetch_tmap(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// A bounded wait of a whole warp, with one answer for all lanes: the warp is converged behind it, which the
// aligned tcgen05 loads and stores that follow need. All lanes wait: where one did it for the others the warp was not put to
// sleep, and twelve such warps took the issue slots of the softmax (every case 1.3 to 1.9 times slower).
// The limit is time, since a probe may take 88 ns or tens of microseconds. These waits are for work on a tile or two, which
// takes microseconds, but one: the warp that copies queries is done with its segment at once and waits for the next one's
// announcement, which comes when the last tile of this one is on its way, 512 tiles of up to 2.4 us later.
constexpr uint32_t kPfWaitNs = 2000000000;
__device__ __forceinline__ bool pf_wait(uint32_t mbar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc::mbar_wait_ns(mbar, parity & 1u, kPfWaitNs)) != 0;
}
__device__ __forceinline__ bool pf_wait_lane(uint32_t mbar, uint32_t parity) {
    return tc::mbar_wait_ns(mbar, parity & 1u, kPfWaitNs);
}
// One arrival for the warp, behind what all its lanes did.
__device__ __forceinline__ void pf_arrive(uint32_t mbar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(mbar);
}
__device__ __forceinline__ void pf_cp_async_arrive(uint32_t mbar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(mbar) : "memory");
}

// The kernels (prefix_few.cu, prefix_wide.cu). With d.wide the few-rows kernel is launched as the dependent of the wide
// one, whose results it does not need.
cudaError_t launch_prefix_few(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, cudaStream_t s);
cudaError_t launch_prefix_wide(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, cudaStream_t s);

}  // namespace hsa
