// prefix.cu -- softmax attention of a decode batch over a shared prefix and each request's own pages, on
// the 5th-generation tensor cores.
//
// For a query row q and its visible keys, out = sum_k exp(s_k - m) v_k / sum_k exp(s_k - m) with
// s = scale q.k. The keys are cut into tiles of 128 (two pages); over a run of tiles a row keeps its running
// maximum m, sum l and output O = sum exp(s - m) v, and runs are joined at the end by
// O = sum 2^(m_i - M) O_i, l likewise. All query rows of a key head read the same prefix keys, so the prefix
// is a matrix product with (requests x query heads x tokens) rows; a request's own keys are one with the
// few rows of its own. Both are the same SEGMENT here: up to 256 rows of one key head, a page list, a
// run of tiles, one partial (m, l, O) per row.
//
// Persistent, warp-specialised kernel, one CTA per SM:
//   warps 0-3, 4-7  two softmax warpgroups = two STREAMS, one thread per row. A segment of more than
//               128 rows gives each stream 128 of them and both read every tile; a smaller one gives both
//               streams the same rows and alternates the tiles between them (each keeps a partial of its own),
//               so that one stream's products run under the other's softmax either way;
//   warp 8      MMA issuer: S = Q K^T and O += P V of both streams, whichever is ready;
//   warp 9      K and V tiles by TMA, page by page (64 rows of one head are contiguous);
//   warps 10-11 Q rows by cp.async.
// P (bf16) is written over S in TMEM and is the A operand of P V. The accumulator in TMEM is rescaled only
// when a row's maximum grows by more than 2^8 (then P would leave a comfortable range; up to that the old
// maximum serves as well, since the final quotient cancels it).
#include <cuda.h>

#include "launch.h"
#include "profile.h"
#include "tc.cuh"

namespace hsa {

constexpr int kPfTile = 128;      // keys per tile = 2 pages, and rows per stream = MMA M
constexpr int kPfRows = 256;      // rows per segment at most
constexpr int kPfMmaWarp = 8, kPfTmaWarp = 9, kPfQWarp = 10, kPfQWarps = 2;
constexpr int kPfThreads = 32 * (kPfQWarp + kPfQWarps);
constexpr int kPfCtas = 148;      // at most: one per SM; the workspace is sized for it
constexpr int kPfItems = 4 * kPfCtas;  // prefix segments at most (or one per head and row group)
// What starting and ending a segment costs, in tiles, for dividing the work
constexpr int kPfPrefixCost = 2, kPfOwnCost = 1;

// How the work is divided; the same for every CTA, stored for the join kernel by CTA 0.
//   prefix: per key head and row group, `nsplit` runs of `run` tiles; segment i goes to CTA i % ctas, row
//   groups of one run next to each other (they read the same keys at the same time, through L2);
//   own: all (request, key head, row group) laid end to end on an axis, cost[b] + tiles each (cum), and
//   the axis cut into one interval per CTA such that prefix and own work add up evenly: the first `lo_ctas`
//   CTAs, which have one prefix segment more, get `cap_lo`, the others `cap_hi`.
struct PfPlan {
    int ctas, tiles, run, nsplit, items, lo_ctas;
    int64_t cap_lo, cap_hi, axis;
    int P;  // prefix tokens
    __device__ int64_t start(int i) const {
        const int64_t x = i <= lo_ctas ? i * cap_lo : lo_ctas * cap_lo + (i - lo_ctas) * cap_hi;
        return x < axis ? x : axis;
    }
    __device__ int cta_of(int64_t x) const {
        return x < lo_ctas * cap_lo ? (int)(x / cap_lo) : lo_ctas + (int)((x - lo_ctas * cap_lo) / cap_hi);
    }
};

// Sizes that follow from the call's arguments alone.
struct PfDims {
    int Rp, Rgp;       // prefix rows per key head, in groups of kPfRows
    int Ro, Rgo;       // own rows per request and key head
    int strideP, strideO;  // rows of one segment's partials
    int max_items, max_slots;
    __host__ __device__ PfDims(int B, int H, int Hkv, int Tq, int max_prefix_pages) {
        Ro = H / Hkv * Tq;
        Rp = B * Ro;
        Rgp = (Rp + kPfRows - 1) / kPfRows;
        Rgo = (Ro + kPfRows - 1) / kPfRows;
        strideP = Rp <= kPfTile ? 2 * Rp : kPfRows;
        strideO = Ro <= kPfTile ? 2 * Ro : kPfRows;
        const int units = Hkv * Rgp, tiles = (max_prefix_pages + 1) / 2;
        int ns = kPfItems / units;
        ns = ns < 1 ? 1 : ns;
        ns = ns < tiles ? ns : tiles;
        max_items = units * ns;
        max_slots = B * Hkv * Rgo + kPfCtas;
    }
};

struct PfWork {
    int32_t *err;
    PfPlan *plan;
    int32_t *status;   // [kPfCtas]
    int32_t *cum;      // [B + 1]
    float *Op, *mlp;   // prefix partials [max_items][strideP][D], [..][2]
    float *Oo, *mlo;   // own partials [max_slots][strideO][D], [..][2]
    size_t bytes;
};

static PfWork pf_work(void *ws, const PfDims &d, int B, int D) {
    PfWork w{};
    char *base = static_cast<char *>(ws);
    size_t used = 0;
    auto take = [&](size_t n) {
        char *p = base ? base + used : nullptr;
        used += (n + 255) / 256 * 256;
        return p;
    };
    w.err = reinterpret_cast<int32_t *>(take(sizeof(int32_t)));  // first: hsa_workspace_status reads it
    w.plan = reinterpret_cast<PfPlan *>(take(sizeof(PfPlan)));
    w.status = reinterpret_cast<int32_t *>(take(kPfCtas * sizeof(int32_t)));
    w.cum = reinterpret_cast<int32_t *>(take(((size_t)B + 1) * sizeof(int32_t)));
    w.mlp = reinterpret_cast<float *>(take((size_t)d.max_items * d.strideP * 2 * sizeof(float)));
    w.mlo = reinterpret_cast<float *>(take((size_t)d.max_slots * d.strideO * 2 * sizeof(float)));
    w.Op = reinterpret_cast<float *>(take((size_t)d.max_items * d.strideP * D * sizeof(float)));
    w.Oo = reinterpret_cast<float *>(take((size_t)d.max_slots * d.strideO * D * sizeof(float)));
    w.bytes = used;
    return w;
}

template <int D>
struct PfSmem {
    static constexpr int KH = D / 64;                       // 128-byte column blocks of D
    static constexpr uint32_t OP = KH * 16384;              // one operand tile [128][D]
    static constexpr int KS = D == 128 ? 2 : 4, VS = D == 128 ? 2 : 4;
    static constexpr uint32_t Q = 0, K = 2 * OP, V = K + KS * OP;
    static constexpr uint32_t BAR = V + VS * OP;
    // mbarriers
    static constexpr int kKFull = 0, kKEmpty = KS, kVFull = 2 * KS, kVEmpty = 2 * KS + VS, kQFull = 2 * KS + 2 * VS,
                         kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPFull = kSFull + 2, kODone = kPFull + 2,
                         kOEmpty = kODone + 2, NBAR = kOEmpty + 2;
    static constexpr uint32_t FLAG = BAR + 8 * NBAR;        // int[VS]: which of a V slot's two pages are good
    static constexpr uint32_t TMEM = FLAG + 4 * VS;
    static constexpr uint32_t BAD = TMEM + 4;
    static constexpr uint32_t PLAN = (BAD + 4 + 15) / 16 * 16;
    static constexpr uint32_t RED = PLAN + 128;             // scratch of the schedule's reductions: 2 x 64 words
    static constexpr uint32_t CUM = RED + 512;              // int[B + 1]
    static constexpr size_t dyn(int B) { return CUM + 4 * ((size_t)B + 1) + 1024; }  // slack for 1 KB alignment
    static constexpr uint32_t S_COL = 0, O_COL = 2 * kPfTile, TMEM_COLS = 512;
};
static_assert(PfSmem<128>::dyn(8192) <= 227 * 1024 && PfSmem<64>::dyn(8192) <= 227 * 1024, "shared memory budget");
static_assert(sizeof(PfPlan) <= 128, "plan slot");

__device__ __forceinline__ int64_t pf_clamp_len(int64_t n, int pages) { return min(n, (int64_t)pages * kChunk); }
__device__ __forceinline__ int pf_tiles(int64_t n) { return n > 0 ? (int)((n + kPfTile - 1) / kPfTile) : 0; }

// One segment, and the walk over a CTA's segments (every role walks them alike).
struct PfSeg {
    int h, b;            // key head; request (own segments; -1: prefix)
    int r0, nr;          // its rows among the key head's (prefix) or the request's (own)
    int tile0, nt;       // run of tiles
    int len;             // tokens of the sequence
    int part;            // index of its partials
    const int32_t *table;
    __device__ bool shared_tiles() const { return nr > kPfTile; }
    __device__ int count(int s) const { return nr > kPfTile ? nt : (nt + 1 - s) >> 1; }  // tiles of stream s
};

struct PfWalk {
    const PrefixArgs &a;
    const PfPlan &p;
    const int32_t *cum;
    const PfDims &d;
    int item;
    int64_t x, end;
    __device__ PfWalk(const PrefixArgs &a_, const PfPlan &p_, const int32_t *cum_, const PfDims &d_, int cta)
        : a(a_), p(p_), cum(cum_), d(d_), item(cta), x(p_.start(cta)), end(p_.start(cta + 1)) {}
    __device__ bool next(PfSeg &s) {
        if (item < p.items) {
            const int rg = item % d.Rgp, k = item / d.Rgp % p.nsplit;
            s.h = item / d.Rgp / p.nsplit;
            s.b = -1;
            s.r0 = rg * kPfRows;
            s.nr = min(kPfRows, d.Rp - s.r0);
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
            int lo = 0, hi = a.B;  // the request whose stretch of the axis holds x (empty ones have none)
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if ((int64_t)cum[m] * hr_n <= x) lo = m;
                else hi = m;
            }
            const int w = cum[lo + 1] - cum[lo];
            const int64_t rest = x - (int64_t)cum[lo] * hr_n;
            const int hr = (int)(rest / w), from = (int)(rest - (int64_t)hr * w);
            const int to = (int)min((int64_t)w, from + (end - x));
            x += to - from;
            const int t0 = max(from - kPfOwnCost, 0), t1 = max(to - kPfOwnCost, 0);
            if (t1 <= t0) continue;
            s.h = hr / d.Rgo;
            s.b = lo;
            s.r0 = hr % d.Rgo * kPfRows;
            s.nr = min(kPfRows, d.Ro - s.r0);
            s.tile0 = t0;
            s.nt = t1 - t0;
            s.len = (int)pf_clamp_len(a.own_len[lo], a.max_pages);
            s.part = lo * hr_n + hr + (int)blockIdx.x;
            s.table = a.block_table + (int64_t)lo * a.max_pages;
            return true;
        }
        return false;
    }
};

// Row rr of a segment: its row in q / out.
__device__ __forceinline__ int64_t pf_q_row(const PfSeg &s, const PfDims &d, int Hkv, int rr) {
    const int r = s.r0 + rr;
    return s.b < 0 ? (int64_t)(r / d.Ro * Hkv + s.h) * d.Ro + r % d.Ro : (int64_t)(s.b * Hkv + s.h) * d.Ro + r;
}

// A bounded wait of a whole warp, with one answer for all lanes: the warp is converged behind it, which the
// aligned tcgen05 loads and stores that follow need. A probe may suspend the thread for tens of microseconds, so
// 2^15 of them are seconds.
__device__ __forceinline__ bool pf_wait(uint32_t mbar, uint32_t parity) {
    return __all_sync(0xffffffffu, tc::mbar_wait_n(mbar, parity, 1u << 15)) != 0;
}
__device__ __forceinline__ bool pf_wait_lane(uint32_t mbar, uint32_t parity) {
    return tc::mbar_wait_n(mbar, parity, 1u << 15);
}

__device__ __forceinline__ void pf_cp_async_arrive(uint32_t mbar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(mbar) : "memory");
}

// The division of the work, by the whole block, into shared memory (cum and the plan).
__device__ void pf_schedule(const PrefixArgs &a, const PfDims &d, PfPlan *plan, int32_t *cum, int32_t *red) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ctas = gridDim.x;
    const int per = (a.B + kPfThreads - 1) / kPfThreads;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    int sum = 0;
    for (int b = lo; b < hi; ++b) {
        const int t = pf_tiles(pf_clamp_len(a.own_len[b], a.max_pages));
        const int w = t > 0 ? t + kPfOwnCost : 0;
        cum[b] = w;
        sum += w;
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kPfThreads / 32; ++w) {
        if (w < warp) before += red[w];
        total += red[w];
    }
    before += x - sum;
    for (int b = lo; b < hi; ++b) {
        const int w = cum[b];
        cum[b] = before;
        before += w;
    }
    if (tid == 0) cum[a.B] = total;
    const int64_t axis = (int64_t)total * a.Hkv * d.Rgo;
    const int64_t plen = a.max_prefix_pages > 0 ? pf_clamp_len(a.prefix_len[0], a.max_prefix_pages) : 0;
    const int P = plen > 0 ? (int)plen : 0, tiles = pf_tiles(P);
    // the number of runs per head and row group that ends the work soonest, both kinds of it counted
    const int units = a.Hkv * d.Rgp;
    const int ns_max = min(max(kPfItems / units, 1), tiles);
    int64_t best = INT64_MAX;
    for (int ns = 1 + tid; ns <= ns_max; ns += kPfThreads) {
        const int run = (tiles + ns - 1) / ns, items = units * ((tiles + run - 1) / run);
        const int64_t waves = (int64_t)((items + ctas - 1) / ctas) * (run + kPfPrefixCost);
        const int64_t even = ((int64_t)items * (run + kPfPrefixCost) + axis + ctas - 1) / ctas;
        const int64_t key = max(waves, even) * 4096 + ns;  // fewer runs win a tie
        best = min(best, key);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = min(best, (int64_t)__shfl_xor_sync(0xffffffffu, (long long)best, o));
    int64_t *red64 = reinterpret_cast<int64_t *>(red + 64);
    if (lane == 0) red64[warp] = best;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kPfThreads / 32; ++w) best = min(best, red64[w]);
        PfPlan p{};
        p.ctas = ctas;
        p.P = P;
        p.tiles = tiles;
        p.axis = axis;
        p.run = 1;
        p.nsplit = 1;
        if (tiles > 0) {
            const int ns = (int)(best % 4096);
            p.run = (tiles + ns - 1) / ns;
            p.nsplit = (tiles + p.run - 1) / p.run;
            p.items = units * p.nsplit;
        }
        const int64_t cost = p.run + kPfPrefixCost;
        p.lo_ctas = p.items % ctas;
        const int64_t pc_hi = p.items / ctas * cost, pc_lo = pc_hi + cost;
        const int hi_ctas = ctas - p.lo_ctas;
        const int64_t alone = (axis + hi_ctas - 1) / hi_ctas;
        if (pc_hi + alone <= pc_lo) {  // the CTAs with a prefix segment less take all of it
            p.cap_lo = 0;
            p.cap_hi = alone;
        } else {
            const int64_t share = (axis + p.lo_ctas * pc_lo + hi_ctas * pc_hi + ctas - 1) / ctas;
            p.cap_lo = share - pc_lo;
            p.cap_hi = share - pc_hi;
        }
        *plan = p;
    }
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) prefix_decode_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                      const __grid_constant__ CUtensorMap tmK,
                                                                      const __grid_constant__ CUtensorMap tmV) {
    using SM = PfSmem<D>;
    constexpr int KS = SM::KS, VS = SM::VS;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;  // 1 KB aligned (swizzle atoms)
    unsigned char *s = smem_raw + (sb - raw);
    volatile int *s_flag = reinterpret_cast<volatile int *>(s + SM::FLAG);
    int *s_bad = reinterpret_cast<int *>(s + SM::BAD);
    PfPlan *s_plan = reinterpret_cast<PfPlan *>(s + SM::PLAN);
    int32_t *s_cum = reinterpret_cast<int32_t *>(s + SM::CUM);
    auto bar = [&](int i) { return sb + SM::BAR + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kPfMmaWarp) tc::tmem_alloc(sb + SM::TMEM, SM::TMEM_COLS);
    if (tid == 0) {
        *s_bad = 0;
        for (int i = 0; i < KS; ++i) {
            tc::mbar_init(bar(SM::kKFull + i), 1);
            tc::mbar_init(bar(SM::kKEmpty + i), 2);  // each stream's S, or one stream's twice
        }
        for (int i = 0; i < VS; ++i) {
            tc::mbar_init(bar(SM::kVFull + i), 1);
            tc::mbar_init(bar(SM::kVEmpty + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(SM::kQFull + i), 32 * kPfQWarps);
            tc::mbar_init(bar(SM::kQEmpty + i), 2);
            tc::mbar_init(bar(SM::kSFull + i), 1);
            tc::mbar_init(bar(SM::kPFull + i), kPfTile);
            tc::mbar_init(bar(SM::kODone + i), 1);
            tc::mbar_init(bar(SM::kOEmpty + i), kPfTile);
        }
        tc::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t *>(s + SM::TMEM);
    pdl_wait();  // what precedes the call in its stream is visible from here on
    pf_schedule(a, d, s_plan, s_cum, reinterpret_cast<int32_t *>(s + SM::RED));
    const PfPlan &plan = *s_plan;
    if (blockIdx.x == 0) {  // for the join
        for (int b = tid; b <= a.B; b += kPfThreads) w.cum[b] = s_cum[b];
        if (tid == 0) *w.plan = plan;
    }
    bool ok = true;
    PfWalk walk(a, plan, s_cum, d, blockIdx.x);
    PfSeg seg;

    if (warp == kPfTmaWarp) {
        // ================= K and V tiles =================
        const int pages_all = a.num_pages;
        int n = 0;
        while (ok && walk.next(seg)) {
            const int npages = (seg.len + kChunk - 1) / kChunk;  // of the sequence; its table holds them
            auto fetch = [&](int from) {  // this lane's page id of the batch that starts at page `from`
                const int i = from + lane;
                return i < min(npages, 2 * (seg.tile0 + seg.nt)) ? seg.table[i] : -1;
            };
            int ids = fetch(2 * seg.tile0), ids_next = 0;
            for (int t = 0; t < seg.nt && ok; ++t, ++n) {
                if (t % 16 == 0) {
                    if (t > 0) ids = ids_next;
                    ids_next = fetch(2 * (seg.tile0 + t) + 32);
                }
                const int p0 = __shfl_sync(0xffffffffu, ids, 2 * (t & 15)), p1 = __shfl_sync(0xffffffffu, ids, 2 * (t & 15) + 1);
                if (lane == 0) {
                    const bool g0 = p0 >= 0 && p0 < pages_all, g1 = p1 >= 0 && p1 < pages_all;
                    // a page that is not there lies behind the pool's last row: it is filled with zeros
                    const int y0 = ((g0 ? p0 : pages_all) * a.Hkv + (g0 ? seg.h : 0)) * kChunk;
                    const int y1 = ((g1 ? p1 : pages_all) * a.Hkv + (g1 ? seg.h : 0)) * kChunk;
                    const int ks = n % KS, vs = n % VS;
                    ok = pf_wait_lane(bar(SM::kKEmpty + ks), ((uint32_t)(n / KS) & 1u) ^ 1u);
                    if (ok) {
                        const uint32_t dst = sb + SM::K + ks * SM::OP;
                        tc::mbar_arrive_expect_tx(bar(SM::kKFull + ks), SM::OP);
#pragma unroll
                        for (int h = 0; h < SM::KH; ++h) {
                            tc::tma_load_2d(dst + h * 16384, &tmK, h * 64, y0, bar(SM::kKFull + ks));
                            tc::tma_load_2d(dst + h * 16384 + 8192, &tmK, h * 64, y1, bar(SM::kKFull + ks));
                        }
                        ok = pf_wait_lane(bar(SM::kVEmpty + vs), ((uint32_t)(n / VS) & 1u) ^ 1u);
                        if (!ok) pf_wait_lane(bar(SM::kKFull + ks), (uint32_t)(n / KS) & 1u);
                    }
                    if (ok) {
                        const uint32_t dst = sb + SM::V + vs * SM::OP;
                        s_flag[vs] = (g0 ? 1 : 0) | (g1 ? 2 : 0);
                        tc::mbar_arrive_expect_tx(bar(SM::kVFull + vs), SM::OP);
#pragma unroll
                        for (int h = 0; h < SM::KH; ++h) {
                            tc::tma_load_2d(dst + h * 16384, &tmV, h * 64, y0, bar(SM::kVFull + vs));
                            tc::tma_load_2d(dst + h * 16384 + 8192, &tmV, h * 64, y1, bar(SM::kVFull + vs));
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                if (!ok) break;
            }
        }
        // every copy has landed before the CTA may exit, however the walk ended
        for (int i = max(0, n - KS); i < n; ++i) pf_wait(bar(SM::kKFull + i % KS), (uint32_t)(i / KS) & 1u);
        for (int i = max(0, n - VS); i < n; ++i) pf_wait(bar(SM::kVFull + i % VS), (uint32_t)(i / VS) & 1u);
    } else if (warp >= kPfQWarp) {
        // ================= Q rows =================
        constexpr int CPR = D / 8, RPW = 32 / CPR;  // 16-byte chunks per row, rows per warp-wide copy
        const int qw = warp - kPfQWarp, rsub = lane / CPR, ch = lane % CPR;
        uint32_t uses[2] = {0, 0};
        int turn = 0;
        while (ok && walk.next(seg)) {
            const bool both = seg.shared_tiles();
            for (int k = 0; k < (both ? 2 : 1) && ok; ++k) {
                const int q = both ? k : turn;
                ok = pf_wait(bar(SM::kQEmpty + q), (uses[q] & 1u) ^ 1u);
                if (!ok) break;
                ++uses[q];
                const int rows = min(kPfTile, seg.nr - k * kPfTile);
                const uint32_t dst = sb + SM::Q + q * SM::OP;
                for (int r = qw * RPW + rsub; r < rows; r += kPfQWarps * RPW)  // the other rows are nobody's
                    cp_async16_u32(dst + (ch >> 3) * 16384 + tc::sw128(r, ch & 7),
                                   a.q + pf_q_row(seg, d, a.Hkv, k * kPfTile + r) * D + ch * 8, 16);
                pf_cp_async_arrive(bar(SM::kQFull + q));  // fires when this thread's copies have landed
            }
            if (!both) turn ^= 1;
        }
        cp_async_commit();
        cp_async_wait<0>();  // nothing in flight when the CTA exits
    } else if (warp == kPfMmaWarp) {
        // ================= MMA issuer: the whole warp runs the loop, one elected lane issues =================
        constexpr uint32_t idesc_s = tc::idesc_bf16(kPfTile, kPfTile, 0, 0);
        constexpr uint32_t idesc_o = tc::idesc_bf16(kPfTile, D, 0, 1);
        struct Stream {
            PfSeg seg;
            int item;
            int64_t x;
            bool live, want_pv;
            int j, cnt, n0, q, turn;
            uint32_t uses0, uses1, qphase, tiles, segs;
        } st[2];
        auto advance = [&](Stream &c, int sid) {  // to the next segment with tiles of this stream
            walk.item = c.item;
            walk.x = c.x;
            c.live = false;
            while (walk.next(c.seg)) {
                const bool both = c.seg.shared_tiles();
                if (both) {
                    c.q = sid;
                    c.qphase = sid ? c.uses1 : c.uses0;
                    ++c.uses0;
                    ++c.uses1;
                } else {
                    c.q = c.turn;
                    c.qphase = c.turn ? c.uses1 : c.uses0;
                    if (c.turn) ++c.uses1;
                    else ++c.uses0;
                    c.turn ^= 1;
                }
                c.j = 0;
                c.cnt = c.seg.count(sid);
                if (c.cnt > 0) {
                    c.live = true;
                    break;
                }
                c.n0 += c.seg.nt;
            }
            c.item = walk.item;
            c.x = walk.x;
        };
#pragma unroll
        for (int sid = 0; sid < 2; ++sid) {
            st[sid].item = walk.item;
            st[sid].x = walk.x;
            st[sid].want_pv = false;
            st[sid].n0 = st[sid].turn = 0;
            st[sid].uses0 = st[sid].uses1 = st[sid].tiles = st[sid].segs = 0;
        }
        advance(st[0], 0);
        advance(st[1], 1);
        // one answer for the whole warp, so that it stays converged
        auto done = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, tc::mbar_test(bar(i), parity)) != 0; };
        // A slot's fillings are used by either stream, and a stream that skips some cannot tell a filling from the
        // one two before it by its parity. So the warp observes every filling of every slot in order (none can be
        // replaced before a stream has used it), and the streams ask the counts.
        int k_seen = 0, v_seen = 0, k_slot = 0, v_slot = 0;
        uint32_t q_seen0 = 0, q_seen1 = 0, k_par = 0, v_par = 0;
        uint32_t idle = 0;
        while (st[0].live || st[1].live) {
            bool progress = false;
            if (done(SM::kKFull + k_slot, k_par)) {
                ++k_seen;
                if (++k_slot == KS) k_slot = 0, k_par ^= 1u;
            }
            if (done(SM::kVFull + v_slot, v_par)) {
                ++v_seen;
                if (++v_slot == VS) v_slot = 0, v_par ^= 1u;
            }
            if (done(SM::kQFull, q_seen0 & 1u)) ++q_seen0;
            if (done(SM::kQFull + 1, q_seen1 & 1u)) ++q_seen1;
#pragma unroll
            for (int sid = 0; sid < 2; ++sid) {
                Stream &c = st[sid];
                if (!c.live) continue;
                const bool both = c.seg.shared_tiles();
                const int n = c.n0 + (both ? c.j : 2 * c.j + sid);
                const int ks = n % KS, vs = n % VS;
                if (!c.want_pv) {
                    // the V filling before this tile's in its slot has landed, too: the softmax's wait on the slot's
                    // parity, which follows S, is then exact
                    if (n >= k_seen || n - VS >= v_seen) continue;
                    if (c.j == 0 && c.qphase >= (c.q ? q_seen1 : q_seen0)) continue;
                    // S and P share columns: P of the stream's tile before must have been read
                    if (c.tiles > 0 && !done(SM::kODone + sid, (c.tiles - 1) & 1u)) continue;
                    tc::fence_after();
                    tc::fence_proxy_async_smem();  // the Q rows came by cp.async (generic proxy)
                    const uint32_t sq = sb + SM::Q + c.q * SM::OP, sk = sb + SM::K + ks * SM::OP;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (uint32_t)((k >> 2) * 16384 + (k & 3) * 32);
                        tc::mma_bf16_ss_w(tmem + SM::S_COL + sid * kPfTile, tc::desc_kmajor(sq + off),
                                          tc::desc_kmajor(sk + off), idesc_s, k > 0 ? 1u : 0u);
                    }
                    tc::commit_w(bar(SM::kSFull + sid));
                    tc::commit_w(bar(SM::kKEmpty + ks));
                    if (!both) tc::commit_w(bar(SM::kKEmpty + ks));
                    if (c.j == c.cnt - 1) {
                        tc::commit_w(bar(SM::kQEmpty + c.q));
                        if (both || c.seg.count(sid ^ 1) == 0) tc::commit_w(bar(SM::kQEmpty + c.q));
                    }
                    c.want_pv = true;
                } else {
                    if (!done(SM::kPFull + sid, c.tiles & 1u)) continue;
                    if (n >= v_seen) continue;
                    if (c.j == 0 && c.segs > 0 && !done(SM::kOEmpty + sid, (c.segs - 1) & 1u)) continue;
                    tc::fence_after();
                    const uint32_t sv = sb + SM::V + vs * SM::OP;
#pragma unroll
                    for (int k = 0; k < kPfTile / 16; ++k)
                        tc::mma_bf16_ts_w(tmem + SM::O_COL + sid * D, tmem + SM::S_COL + sid * kPfTile + k * 8,
                                          tc::desc_mnmajor(sv + k * 2048, 16384), idesc_o, c.j > 0 || k > 0 ? 1u : 0u);
                    tc::commit_w(bar(SM::kODone + sid));
                    tc::commit_w(bar(SM::kVEmpty + vs));
                    if (!both) tc::commit_w(bar(SM::kVEmpty + vs));
                    c.want_pv = false;
                    ++c.tiles;
                    if (++c.j == c.cnt) {
                        ++c.segs;
                        c.n0 += c.seg.nt;
                        advance(c, sid);
                    }
                }
                progress = true;
            }
            if (progress) {
                idle = 0;
            } else if (++idle > (1u << 26)) {
                ok = false;
                break;
            }
        }
        __syncwarp();
    } else {
        // ================= softmax: stream sid, thread = row =================
        const int sid = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + SM::S_COL + sid * kPfTile;
        const uint32_t tO = tmem + lane_off + SM::O_COL + sid * D;
        const float sl2 = a.scale * 1.4426950408889634f;
        uint32_t tiles = 0;
        int n0 = 0;
        for (; ok && walk.next(seg); n0 += seg.nt) {
            const int cnt = seg.count(sid);
            if (cnt == 0) continue;
            const bool both = seg.shared_tiles();
            const int rr = both ? sid * kPfTile + r : r;
            const bool mine = rr < seg.nr;
            const bool active = rr - lane < seg.nr;  // does this warp hold any row?
            // tokens of the sequence that the row sees; rows that are nobody's, and those of the empty rows of a
            // padded batch, compute something that is never read
            int lim = INT32_MAX;
            if (mine) {
                const int rw = seg.r0 + rr;
                const int b = seg.b < 0 ? rw / d.Ro : seg.b;
                const int64_t own = pf_clamp_len(a.own_len[b], a.max_pages);
                const int last = (int)own - a.Tq + (rw % d.Ro) % a.Tq + 1;  // own tokens seen; below 0: prefix tokens not seen
                if (own >= 0) lim = max(0, seg.b < 0 ? seg.len + min(last, 0) : last);
            }
            float m = -INFINITY, l = 0.0f;
            for (int j = 0; j < cnt; ++j, ++tiles) {
                const int t = both ? j : 2 * j + sid, n = n0 + t, vs = n % VS;
                const int base = (seg.tile0 + t) * kPfTile;
                // v_full also publishes the tile's page flags; its slot is not filled again before this
                // stream's P V has read it, and S says that the filling before this one is over
                ok = pf_wait(bar(SM::kSFull + sid), tiles & 1u) && pf_wait(bar(SM::kVFull + vs), (uint32_t)(n / VS) & 1u);
                if (!ok) break;
                tc::fence_after();
                const int flags = s_flag[vs];
                if (active) {
                    __syncwarp();
                    float x[2][64];
                    tc::tmem_ld64(tS, x[0]);
                    tc::tmem_ld64(tS + 64, x[1]);
                    if (__any_sync(0xffffffffu, flags != 3 || base + kPfTile > lim)) {
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const int vis = (flags >> p) & 1 ? lim - base - 64 * p : 0;
#pragma unroll
                            for (int i = 0; i < 64; ++i) x[p][i] = i < vis ? x[p][i] : -INFINITY;
                        }
                    }
                    float m8[8];  // row maximum as a tree
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        m8[i] = fmaxf(x[0][i], x[1][i]);
#pragma unroll
                        for (int k = 8; k < 64; k += 8) m8[i] = fmaxf(m8[i], fmaxf(x[0][i + k], x[1][i + k]));
                    }
                    const float mx = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                                           fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                    const bool grow = (mx - m) * sl2 > 8.0f;  // from -inf, too; false while nothing is visible
                    if (j == 0) {
                        m = mx;
                    } else if (__any_sync(0xffffffffu, grow)) {
                        ok = pf_wait(bar(SM::kODone + sid), (tiles - 1) & 1u);
                        if (!ok) break;
                        tc::fence_after();
                        const float f = grow ? ex2_approx((m - mx) * sl2) : 1.0f;
                        if (grow) m = mx;
                        l *= f;
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tc::tmem_ld32(tO + c, o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= f;
                            tc::tmem_st32f(tO + c, o);
                        }
                    }
                    const float ms = m > -INFINITY ? m * sl2 : 0.0f;
                    float l4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint32_t pk[32];  // P row as bf16 pairs, over S
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float p0 = ex2_approx(fmaf(x[p][2 * i], sl2, -ms));
                            const float p1 = ex2_approx(fmaf(x[p][2 * i + 1], sl2, -ms));
                            l4[i & 3] += p0 + p1;
                            pk[i] = pack_bf16x2(p0, p1);
                        }
                        tc::tmem_st32(tS + 32 * p, pk);
                    }
                    l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                }
                // keys behind the sequence's end weigh nothing, but 0 x NaN is NaN: their V rows become zero
                if (base + kPfTile > seg.len) {
                    if (r >= seg.len - base) {
#pragma unroll
                        for (int h = 0; h < SM::KH; ++h) {
                            uint4 *row = reinterpret_cast<uint4 *>(s + SM::V + vs * SM::OP + h * 16384 + r * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) row[i] = make_uint4(0, 0, 0, 0);
                        }
                    }
                    tc::fence_proxy_async_smem();
                }
                tc::fence_before();
                tc::mbar_arrive(bar(SM::kPFull + sid));
            }
            if (!ok) break;
            ok = pf_wait(bar(SM::kODone + sid), (tiles - 1) & 1u);
            if (!ok) break;
            tc::fence_after();
            if (active) {
                const int64_t at = (int64_t)seg.part * (seg.b < 0 ? d.strideP : d.strideO) + (both ? rr : sid * seg.nr + rr);
                float *O = (seg.b < 0 ? w.Op : w.Oo) + at * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    __syncwarp();  // the lanes without a row skip the stores
                    tc::tmem_ld32(tO + c, o);
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<float4 *>(O + c)[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (mine) reinterpret_cast<float2 *>(seg.b < 0 ? w.mlp : w.mlo)[at] = make_float2(m, l);
            }
            tc::fence_before();
            tc::mbar_arrive(bar(SM::kOEmpty + sid));
        }
    }
    if (!ok) *s_bad = 1;
    tc::fence_before();
    __syncthreads();
    pdl_launch_dependents();
    if (tid == 0) w.status[blockIdx.x] = *s_bad;
    if (warp == kPfMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, SM::TMEM_COLS);
    }
}

// Joins a row's partials, one warp per row: M = max m_i, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
constexpr int kPfJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPfJoinThreads) prefix_join_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                     int ctas) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x < 32) {
        int bad = 0;
        for (int i = lane; i < ctas; i += 32) bad |= w.status[i];
        bad = __any_sync(0xffffffffu, bad != 0);
        if (lane == 0) *w.err = bad;
    }
    const int64_t row = (int64_t)blockIdx.x * (kPfJoinThreads / 32) + (threadIdx.x >> 5);
    if (row >= (int64_t)a.B * a.H * a.Tq) return;
    const PfPlan p = *w.plan;
    const int b = (int)(row / ((int64_t)a.H * a.Tq)), hr_n = a.Hkv * d.Rgo;
    const int rem = (int)(row % ((int64_t)a.H * a.Tq)), h = rem / d.Ro, ro = rem % d.Ro;
    int np = 0, per = 1, nr = 0, rr = 0, rg = 0;      // prefix partials: np runs of `per` streams
    int i0 = 0, no = 0, orr = 0, onr = 0, obase = 0;  // own partials: CTAs i0 .. i0 + no - 1, two streams each
    int64_t x0 = 0;
    int wt = 0;
    if (a.own_len[b] >= 0) {
        const int rp = b * d.Ro + ro;
        rg = rp / kPfRows;
        rr = rp % kPfRows;
        nr = min(kPfRows, d.Rp - rg * kPfRows);
        per = nr > kPfTile ? 1 : 2;
        np = p.items > 0 ? p.nsplit : 0;
        wt = w.cum[b + 1] - w.cum[b];
        if (wt > 0) {
            const int hr = h * d.Rgo + ro / kPfRows;
            x0 = (int64_t)w.cum[b] * hr_n + (int64_t)hr * wt;
            i0 = p.cta_of(x0);
            no = p.cta_of(x0 + wt - 1) - i0 + 1;
            obase = b * hr_n + hr;
            orr = ro % kPfRows;
            onr = min(kPfRows, d.Ro - ro / kPfRows * kPfRows);
        }
    }
    const int total = np * per + 2 * no;
    // partial idx: its place (rows of D), or -1
    auto place = [&](int idx) -> int64_t {
        if (idx < np * per) {
            const int k = idx / per, st = idx - k * per;
            const int nt = min(p.run, p.tiles - k * p.run);
            if (st >= nt) return -1;
            return (int64_t)((h * p.nsplit + k) * d.Rgp + rg) * d.strideP + st * nr + rr;
        }
        const int i = i0 + (idx - np * per) / 2, st = (idx - np * per) & 1;
        const int64_t from = max(p.start(i), x0) - x0, to = min(p.start(i + 1), x0 + wt) - x0;
        const int nt = (int)(max(to - kPfOwnCost, (int64_t)0) - max(from - kPfOwnCost, (int64_t)0));
        if (onr > kPfTile) {
            if (nt <= 0 || st > 0) return -1;
            return (int64_t)(obase + i) * d.strideO + orr;
        }
        if (st >= nt) return -1;
        return (int64_t)(obase + i) * d.strideO + st * onr + orr;
    };
    const float sl2 = a.scale * 1.4426950408889634f;
    const float2 *mlp = reinterpret_cast<const float2 *>(w.mlp), *mlo = reinterpret_cast<const float2 *>(w.mlo);
    float M = -INFINITY;
    for (int idx = lane; idx < total; idx += 32) {
        const int64_t at = place(idx);
        if (at >= 0) M = fmaxf(M, (idx < np * per ? mlp : mlo)[at].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    constexpr int V = D / 32;  // columns per lane
    float acc[V] = {}, L = 0.0f;
    if (M > -INFINITY) {
        for (int base = 0; base < total; base += 32) {
            const int idx = base + lane;
            int64_t at = idx < total ? place(idx) : -1;
            float f = 0.0f;
            if (at >= 0) {
                const float2 ml = (idx < np * per ? mlp : mlo)[at];
                f = ml.x > -INFINITY ? ex2_approx((ml.x - M) * sl2) : 0.0f;
                L = fmaf(ml.y, f, L);
            }
            const int cnt = min(32, total - base);
#pragma unroll 4
            for (int k = 0; k < cnt; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                const int64_t ak = __shfl_sync(0xffffffffu, (long long)at, k);
                if (ak < 0) continue;
                const float *O = (base + k < np * per ? w.Op : w.Oo) + ak * D + lane * V;
                if constexpr (V == 4) {
                    const float4 o = *reinterpret_cast<const float4 *>(O);
                    acc[0] = fmaf(fk, o.x, acc[0]);
                    acc[1] = fmaf(fk, o.y, acc[1]);
                    acc[2] = fmaf(fk, o.z, acc[2]);
                    acc[3] = fmaf(fk, o.w, acc[3]);
                } else {
                    const float2 o = *reinterpret_cast<const float2 *>(O);
                    acc[0] = fmaf(fk, o.x, acc[0]);
                    acc[1] = fmaf(fk, o.y, acc[1]);
                }
            }
        }
        L = warp_sum(L);
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + row * D + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) out[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0 && a.lse) a.lse[row] = L > 0.0f ? fmaf(M, a.scale, logf(L)) : -INFINITY;
}

size_t prefix_workspace(int B, int H, int Hkv, int Tq, int D, int max_prefix_pages, int max_pages) {
    (void)max_pages;
    return pf_work(nullptr, PfDims(B, H, Hkv, Tq, max_prefix_pages), B, D).bytes;
}

template <int D>
static cudaError_t launch_prefix_d(const PrefixArgs &a, cudaStream_t s) {
    const PfDims d(a.B, a.H, a.Hkv, a.Tq, a.max_prefix_pages);
    const PfWork w = pf_work(a.workspace, d, a.B, D);
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * kChunk;
    if (!make_tmap_bf16(&tk, a.Kp, rows, D, kChunk) || !make_tmap_bf16(&tv, a.Vp, rows, D, kChunk))
        return cudaErrorInvalidValue;
    const size_t smem = PfSmem<D>::dyn(a.B);
    cudaError_t e = cudaFuncSetAttribute(prefix_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = kPfCtas;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int ctas = sms < kPfCtas ? sms : kPfCtas;
    {
        HSA_PROF("prefix_decode", s);
        e = launch_pdl(prefix_decode_kernel<D>, dim3(ctas), dim3(kPfThreads), smem, s, a, d, w, tk, tv);
    }
    if (e != cudaSuccess) return e;
    const int64_t out_rows = (int64_t)a.B * a.H * a.Tq;
    HSA_PROF("prefix_join", s);
    return launch_pdl(prefix_join_kernel<D>, dim3((unsigned)((out_rows + kPfJoinThreads / 32 - 1) / (kPfJoinThreads / 32))),
                      dim3(kPfJoinThreads), 0, s, a, d, w, ctas);
}

cudaError_t launch_prefix_decode(const PrefixArgs &a, cudaStream_t s) {
    return a.D == 128 ? launch_prefix_d<128>(a, s) : launch_prefix_d<64>(a, s);
}

}  // namespace hsa
