// prefix_wide.cu -- segments of more than 64 query rows of the shared-prefix decode: the prefix of large batches,
// a matrix product with (requests x query heads x tokens) rows, bound by the tensor cores and the exponentials.
//
// S = Q K^T (128 rows x 128 keys, fp32 in TMEM), P = exp2(S scale' - m) as bf16 over S in TMEM, which is the A operand
// of O += P V (128 x D, fp32 in TMEM). The reference m of a row need not be its maximum (see prefix_few.cu): it is the
// logit of the first key that the row sees in the segment, so no maximum is taken at all; a tile whose row sum exceeds
// 2^70 moves it (rarely): the pair of warps then reduces the maximum, rescales O in TMEM and does the tile again. (Half a tile, 64
// keys, adds up to 2^70 at most, so a sum over 2^31 keys, times V below 2^28, stays below 2^123.)
//
// Measured, per tile of 128 keys and 256 rows on an SM: D = 128 1.89 us out of L2 (1.32 PFLOP/s over 148 SMs), 2.43 us out of
// HBM; D = 64 1.50 and 1.56. Tensor cores and exponentials are busy half of that time each: a stream's chain bounds it,
// its products S and O wait for one another through four barriers, since P stands in the columns of S. (A third stream
// would need 256 more columns of TMEM, P in shared memory 64 KB that the operands hold.) Start 7 us (schedule 2.4, 128 query rows 2.5 each), end 5 us.
//
// Persistent, warp-specialised kernel, one CTA per SM:
//   warps 0-7, 8-15 softmax of two STREAMS: two threads per row, one for each page of the tile (a thread's 64
//               logits stay in registers). The work is a sequence of items that go to the streams in turn: a
//               segment of more than 128 rows has two items per tile, one for each 128 rows; a smaller one has one
//               (and each stream keeps a partial of its own). So one stream's products run under the other's softmax;
//   warp 16     issues the products S of the items, in order;
//   warp 17     issues the products O, in order (one warp for both spent 2300 cycles on an item, half of them in waits
//               for what was there already and in its own bookkeeping);
//   warp 18     walks the segments and copies K and V tiles by TMA, page by page (64 rows of one head are contiguous);
//   warp 19     Q rows by cp.async, padded with zero rows.
#include <cuda.h>

#include <type_traits>

#include "prefix.cuh"
#include "profile.h"

namespace hsa {

constexpr int kPfStreamWarps = 8;
constexpr int kPfSWarp = 2 * kPfStreamWarps, kPfOWarp = kPfSWarp + 1, kPfTmaWarp = kPfSWarp + 2, kPfQWarp = kPfSWarp + 3;
constexpr int kPfThreads = 32 * (kPfQWarp + 1);
constexpr float kPfGrow = 64.0f, kPfSumMax = 0x1p70f;  // a sum of 64 terms of at most 2^64

template <int D>
struct PfSmem {
    static constexpr int KH = D / 64;                       // 128-byte column blocks of D
    static constexpr uint32_t OP = KH * 16384;              // one operand tile [128][D]
    static constexpr int KS = D == 128 ? 2 : 4, VS = D == 128 ? 2 : 4;
    static constexpr uint32_t Q = 0, K = 2 * OP, V = K + KS * OP;
    static constexpr uint32_t BAR = V + VS * OP;
    // mbarriers
    static constexpr int kKFull = 0, kKEmpty = KS, kVFull = 2 * KS, kVEmpty = 2 * KS + VS, kQFull = 2 * KS + 2 * VS,
                         kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPFull = kSFull + 2,
                         kODone = kPFull + 2, kOEmpty = kODone + 2, kSegFull = kOEmpty + 2, kSegEmpty = kSegFull + kPfRing,
                         NBAR = kSegEmpty + kPfRing;
    static constexpr uint32_t RING = (BAR + 8 * NBAR + 15) / 16 * 16;  // PfNote[kPfRing]
    static constexpr uint32_t ROW = RING + kPfRing * sizeof(PfNote);   // float[2 streams][2 halves][128]: exchanged by a row's threads
    static constexpr uint32_t BADP = ROW + 2 * 2 * 128 * 4;  // int[8]: a wait of the pair of warps ran out
    static constexpr uint32_t TMEM = BADP + 32;
    static constexpr uint32_t BAD = TMEM + 4;
    static constexpr uint32_t PLAN = (BAD + 4 + 15) / 16 * 16;
    static constexpr uint32_t BCUM = PLAN + (sizeof(PfPlan) + 15) / 16 * 16;  // int[blocks + 1]
    static constexpr size_t dyn(int blocks) { return BCUM + 4 * ((size_t)blocks + 1) + 1024; }  // slack: 1 KB alignment
    static constexpr uint32_t S_COL = 0, O_COL = 2 * kPfTile, TMEM_COLS = 512;
};
static_assert(PfSmem<128>::dyn(kPagedMaxBatch / 32) <= 227 * 1024 && PfSmem<64>::dyn(kPagedMaxBatch / 32) <= 227 * 1024, "shared memory budget");

// 2^y for two numbers, by the pipe of the fused multiply-adds: 2^n 2^f with n = round(y), by which a sum with 1.5 2^23 leaves
// the integer in its last bits, and |f| <= 1/2. The polynomial interpolates 2^f at the six Chebyshev nodes of the
// interval; evaluated in fp32 it is off by 2^-22, as the hardware's exponential is. Outside -126 .. 127 it is 2^-126
// (which weighs nothing) and 2^127 (which is out of range for the caller, as the true value is).
__device__ __forceinline__ float2 pf_exp2_fma(float2 y) {
    y = {fminf(fmaxf(y.x, -126.0f), 127.0f), fminf(fmaxf(y.y, -126.0f), 127.0f)};
    const float2 t = add2(y, {12582912.0f, 12582912.0f}), n = add2(t, {-12582912.0f, -12582912.0f});
    const float2 f = fma2(n, {-1.0f, -1.0f}, y);
    float2 p = {0x1.5f089p-10f, 0x1.5f089p-10f};
    p = fma2(p, f, {0x1.3d107p-7f, 0x1.3d107p-7f});
    p = fma2(p, f, {0x1.c6af6cp-5f, 0x1.c6af6cp-5f});
    p = fma2(p, f, {0x1.ebf906p-3f, 0x1.ebf906p-3f});
    p = fma2(p, f, {0x1.62e43p-1f, 0x1.62e43p-1f});
    p = fma2(p, f, {0x1.000002p+0f, 0x1.000002p+0f});
    return {__int_as_float(__float_as_int(p.x) + (__float_as_int(t.x) << 23)), __int_as_float(__float_as_int(p.y) + (__float_as_int(t.y) << 23))};
}

// Do both streams read every tile of the segment, each for rows of its own?
__device__ __forceinline__ bool pf_both(const PfSeg &s) { return s.nr > kPfTile; }

// Named barriers of the two warps (64 threads) that share 32 rows.
__device__ __forceinline__ void pf_pair_bar(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pf_pair_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0u;
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) prefix_wide_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                      const __grid_constant__ CUtensorMap tmK,
                                                                      const __grid_constant__ CUtensorMap tmV) {
    using SM = PfSmem<D>;
    constexpr int KS = SM::KS, VS = SM::VS;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;  // 1 KB aligned (swizzle atoms)
    unsigned char *s = smem_raw + (sb - raw);
    PfNote *s_ring = reinterpret_cast<PfNote *>(s + SM::RING);
    volatile int *s_badp = reinterpret_cast<volatile int *>(s + SM::BADP), *s_bad = reinterpret_cast<volatile int *>(s + SM::BAD);
    PfPlan *s_plan = reinterpret_cast<PfPlan *>(s + SM::PLAN);
    int32_t *s_bcum = reinterpret_cast<int32_t *>(s + SM::BCUM);
    auto bar = [&](int i) { return sb + SM::BAR + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kPfSWarp) tc::tmem_alloc(sb + SM::TMEM, SM::TMEM_COLS);
    if (warp == kPfTmaWarp && lane == 0) {
        pf_prefetch_tmap(&tmK);
        pf_prefetch_tmap(&tmV);
    }
    if (tid == 0) {
        *s_bad = 0;
        for (int i = 0; i < 8; ++i) s_badp[i] = 0;
        for (int i = 0; i < KS; ++i) {
            tc::mbar_init(bar(SM::kKFull + i), 1);
            tc::mbar_init(bar(SM::kKEmpty + i), 1);
        }
        for (int i = 0; i < VS; ++i) {
            tc::mbar_init(bar(SM::kVFull + i), 1);
            tc::mbar_init(bar(SM::kVEmpty + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(bar(SM::kQFull + i), 32);
            tc::mbar_init(bar(SM::kQEmpty + i), 1);
            tc::mbar_init(bar(SM::kSFull + i), 1);
            tc::mbar_init(bar(SM::kPFull + i), kPfStreamWarps);
            tc::mbar_init(bar(SM::kODone + i), 1);
            tc::mbar_init(bar(SM::kOEmpty + i), kPfStreamWarps);
        }
        for (int i = 0; i < kPfRing; ++i) {
            tc::mbar_init(bar(SM::kSegFull + i), 1);
            tc::mbar_init(bar(SM::kSegEmpty + i), kPfThreads / 32 - 1);  // the warps but this ring's writer
        }
        tc::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t *>(s + SM::TMEM);
    pdl_wait();  // what precedes the call in its stream is visible from here on
    pdl_launch_dependents();  // the few-rows kernel may come in as SMs fall free; the join waits for this grid's end
    pf_schedule<kPfThreads>(a, d, true, false, s_plan, s_bcum, [](int) {});
    pf_publish<kPfThreads>(d, true, false, s_plan, s_bcum, w);
    bool ok = true;

    int seg_no = 0;  // the next announced segment
    auto take = [&](PfNote &g) {
        const int slot = seg_no % kPfRing;
        if (!pf_wait(bar(SM::kSegFull + slot), (uint32_t)(seg_no / kPfRing) & 1u)) return false;
        g = s_ring[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(SM::kSegEmpty + slot));
        ++seg_no;
        return true;
    };

    if (warp == kPfTmaWarp) {
        // ================= the walk, K and V tiles =================
        PfWalk walk(a, *s_plan, s_bcum, d);
        const int pages_all = a.num_pages;
        int n = 0, items = 0;
        bool more = true;
        PfNote g;
        while (ok && more) {
            more = walk.next(g.s);
            if (!more) g.s.nr = 0;
            g.n0 = n;
            g.i0 = items;
            if (more) items += pf_both(g.s) ? 2 * g.s.nt : g.s.nt;
            const int slot = seg_no % kPfRing;
            ok = pf_wait(bar(SM::kSegEmpty + slot), ((uint32_t)(seg_no / kPfRing) & 1u) ^ 1u);
            if (!ok) break;
            if (lane == 0) {
                s_ring[slot] = g;
                tc::mbar_arrive(bar(SM::kSegFull + slot));
            }
            ++seg_no;
            if (!more) break;
            const PfSeg &seg = g.s;
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
    } else if (warp == kPfQWarp) {
        // ================= Q rows =================
        uint32_t uses[2] = {0, 0};
        int turn = 0;
        PfNote g;
        while (true) {
            ok = take(g);
            if (!ok || g.s.nr == 0) break;
            const PfSeg &seg = g.s;
            const bool both = pf_both(seg);
            for (int k = 0; k < (both ? 2 : 1) && ok; ++k) {
                const int q = both ? k : turn;
                ok = pf_wait(bar(SM::kQEmpty + q), (uses[q] & 1u) ^ 1u);
                if (!ok) break;
                ++uses[q];
                const int rows = min(kPfTile, seg.nr - k * kPfTile);
                const uint32_t dst = sb + SM::Q + q * SM::OP;
                pf_copy_q<D>(a, d, seg, k * kPfTile, rows, kPfTile,
                             [&](int r, int ch) { return dst + (ch >> 3) * 16384 + tc::sw128(r, ch & 7); });
                pf_cp_async_arrive(bar(SM::kQFull + q));  // fires when this thread's copies have landed
            }
            if (!ok) break;
            if (!both) turn ^= 1;
        }
        cp_async_commit();
        cp_async_wait<0>();  // nothing in flight when the CTA exits
    } else if (warp == kPfSWarp) {
        // ================= S products: the whole warp runs the loop, one elected lane issues =================
        // Item i is item i / 2 of stream i % 2. Every filling of every slot is waited for, in order (here and below).
        constexpr uint32_t idesc = tc::idesc_bf16(kPfTile, kPfTile, 0, 0);
        PfNote g;
        uint32_t uses0 = 0, uses1 = 0;  // fillings of the Q buffers before this segment's
        int turn = 0;
        while (true) {
            ok = take(g);
            if (!ok || g.s.nr == 0) break;
            const bool both = pf_both(g.s);
            const int q0 = both ? 0 : turn;
            if (!both) turn ^= 1;
            int i = g.i0;
            for (int t = 0; t < g.s.nt && ok; ++t) {
                const int n = g.n0 + t, ks = n % KS;
                ok = pf_wait(bar(SM::kKFull + ks), (uint32_t)(n / KS));
                for (int q = q0; ok && q < q0 + (both ? 2 : 1); ++q, ++i) {
                    const int sid = i & 1;
                    if (t == 0) ok = pf_wait(bar(SM::kQFull + q), q ? uses1 : uses0);
                    // S and P share columns: P of the stream's item before must have been read
                    if (ok && i >= 2) ok = pf_wait(bar(SM::kODone + sid), (uint32_t)(i / 2 - 1));
                    if (!ok) break;
                    tc::fence_after();
                    if (t == 0) tc::fence_proxy_async_smem();  // the Q rows came by cp.async (generic proxy)
                    const uint64_t dq = tc::desc_kmajor(sb + SM::Q + q * SM::OP), dk = tc::desc_kmajor(sb + SM::K + ks * SM::OP);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {  // (a descriptor's low bits are its address / 16)
                        const uint64_t off = (uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                        tc::mma_bf16_ss_w(tmem + SM::S_COL + sid * kPfTile, dq + off, dk + off, idesc, k > 0 ? 1u : 0u);
                    }
                    tc::commit_w(bar(SM::kSFull + sid));
                    if (t == g.s.nt - 1) tc::commit_w(bar(SM::kQEmpty + q));
                }
                if (ok) tc::commit_w(bar(SM::kKEmpty + ks));
            }
            if (!ok) break;
            uses0 += both || q0 == 0;
            uses1 += both || q0 == 1;
        }
        __syncwarp();
    } else if (warp == kPfOWarp) {
        // ================= O products =================
        constexpr uint32_t idesc = tc::idesc_bf16(kPfTile, D, 0, 1);
        PfNote g;
        uint32_t runs0 = 0, runs1 = 0;  // of a stream: sums begun in O, one per segment in which it has an item
        while (true) {
            ok = take(g);
            if (!ok || g.s.nr == 0) break;
            const int per = pf_both(g.s) ? 2 : 1, items = per * g.s.nt;
            for (int u = 0; u < items; ++u) {
                const int i = g.i0 + u, sid = i & 1, n = g.n0 + (per == 2 ? u >> 1 : u), vs = n % VS;
                if (per == 1 || !(u & 1)) ok = pf_wait(bar(SM::kVFull + vs), (uint32_t)(n / VS));  // (once for a tile)
                if (u < 2) {  // the stream's first: O of its segment before has been read out
                    const uint32_t run = sid ? runs1++ : runs0++;
                    if (ok && run > 0) ok = pf_wait(bar(SM::kOEmpty + sid), run - 1);
                }
                if (ok) ok = pf_wait(bar(SM::kPFull + sid), (uint32_t)(i / 2));
                if (!ok) break;
                tc::fence_after();
                const uint64_t dv = tc::desc_mnmajor(sb + SM::V + vs * SM::OP, 16384);
#pragma unroll
                for (int k = 0; k < kPfTile / 16; ++k)  // a page's P stands where its S began
                    tc::mma_bf16_ts_w(tmem + SM::O_COL + sid * D, tmem + SM::S_COL + sid * kPfTile + (k >> 2) * 64 + (k & 3) * 8,
                                      dv + (uint64_t)k * (2048 >> 4), idesc, u >= 2 || k > 0 ? 1u : 0u);
                tc::commit_w(bar(SM::kODone + sid));
                if (per == 1 || (u & 1)) tc::commit_w(bar(SM::kVEmpty + vs));
            }
            if (!ok) break;
        }
        __syncwarp();
    } else {
        // ================= softmax: stream sid, two threads per row (half = page of the tile) =================
        // A warp whose wait ran out says so and still comes to the pair's next barrier, and the pair leaves together
        const int sid = warp / kPfStreamWarps, half = (warp >> 2) & 1, quad = warp & 3, r = quad * 32 + lane;
        const int pid = 1 + sid * 4 + quad;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + lane_off + SM::S_COL + sid * kPfTile;
        const uint32_t tO = tmem + lane_off + SM::O_COL + sid * D + half * (D / 2);
        float *s_row = reinterpret_cast<float *>(s + SM::ROW) + sid * 256 + r;  // [0]: half 0, [128]: half 1
        const float sl2 = a.scale * 1.4426950408889634f;
        uint32_t tiles = 0;
        PfNote g;
        while (ok) {
            if (!take(g)) s_badp[pid - 1] = 1;
            pf_pair_bar(pid);
            if (s_badp[pid - 1]) ok = false;
            if (!ok || g.s.nr == 0) break;
            const PfSeg &seg = g.s;
            const bool both = pf_both(seg);
            const int turn = (sid ^ g.i0) & 1;  // which of the segment's items go to this stream: the even or the odd ones
            if (!both && turn >= seg.nt) continue;
            const int rr = both ? turn * kPfTile + r : r, t0 = both ? 0 : turn, dt = both ? 1 : 2;
            const bool mine = rr < seg.nr;
            const bool active = rr - lane < seg.nr;  // do this pair's warps hold any row?
            const int lim = mine ? pf_limit(a, seg, d, rr) : INT32_MAX;
            float ms = 0.0f, l = 0.0f, x[32];
            uint32_t pk[32];  // P of this half as bf16 pairs
            // 32 keys at a time: the logits of 64 beside their P would not fit a thread's 96 registers
            auto probs = [&](const int c, auto with_edge, const int vis) {
                const float2 scale2 = {sl2, sl2}, off2 = {-ms, -ms};
                float2 s2[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                tc::tmem_ld32(tS + 64 * half + 32 * c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 y = fma2({x[2 * i], x[2 * i + 1]}, scale2, off2);
                    float2 p;
                    // (one in four by the other pipe: 94.8 -> 92.7 us for 64 x 16:1 heads over 64K; three in eight 93.5, half 101.8)
                    if (!decltype(with_edge)::value && i % 4 == 3) p = pf_exp2_fma(y);
                    else p = {ex2_approx(y.x), ex2_approx(y.y)};
                    if constexpr (decltype(with_edge)::value) {
                        const int k = 32 * c + 2 * i;
                        p = {k < vis ? p.x : 0.0f, k + 1 < vis ? p.y : 0.0f};
                    }
                    s2[i & 1] = add2(s2[i & 1], p);
                    pk[16 * c + i] = pack_bf16x2(p.x, p.y);
                }
                return (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
            };
            const PfPages pages(seg, a.num_pages);
            int id_next = pages.fetch(seg.tile0), block_end = 0;  // of the 16 tiles whose pages `there_all` tells of
            uint32_t there_all = 0;
            // the tiles before this one lie before the sequence's end, for each of the pair's rows, too
            const int whole = min((int)__reduce_min_sync(0xffffffffu, (uint32_t)lim), seg.len) / kPfTile - seg.tile0;
            bool redo = false;
            for (int t = t0; t < seg.nt;) {
                if (t >= block_end) {
                    there_all = pages.there(id_next);
                    id_next = pages.fetch(seg.tile0 + block_end + 16);
                    block_end += 16;
                }
                // Tiles that every row sees all of, in a loop of their own (see prefix_few.cu)
                const uint32_t gaps = ~(there_all & there_all >> 1) & 0x55555555u & ~0u << 2 * (t & 15);
                const int stop = min(min(seg.nt, whole), gaps ? block_end - 16 + (__ffs(gaps) - 1) / 2 : block_end);
                if (t > t0 && active && !redo) {
                    for (; t < stop; t += dt, ++tiles) {
                        const bool good = pf_wait(bar(SM::kSFull + sid), tiles);
                        tc::fence_after();
                        float sum = probs(0, std::false_type{}, 64);
                        sum += probs(1, std::false_type{}, 64);
                        redo = pf_pair_or(pid, !good || sum > kPfSumMax);
                        if (redo) break;
                        tc::tmem_st32(tS + 64 * half, pk);
                        l += sum;
                        tc::fence_before();
                        pf_arrive(bar(SM::kPFull + sid));
                    }
                    if (t >= seg.nt) break;
                    if (t >= block_end) continue;
                }
                redo = false;
                // Any tile: the first, the ones with an edge, and those where a term left the range
                const int flags = there_all >> 2 * (t & 15) & 3u, n = g.n0 + t, vs = n % VS;
                const int base = (seg.tile0 + t) * kPfTile;
                const int vis = flags >> half & 1 ? lim - base - 64 * half : 0;  // keys of this half that the row sees
                bool good = pf_wait(bar(SM::kSFull + sid), tiles);
                tc::fence_after();
                if (!good) s_badp[pid - 1] = 1;
                if (active) {
                    if (t == t0) {  // the row's reference: its first key, or the second page's where the first is bad
                        if (half == (flags & 1 ? 0 : 1)) {
                            tc::tmem_ld32(tS + 64 * half, x);
                            s_row[0] = vis > 0 ? x[0] * sl2 : -INFINITY;
                        }
                        pf_pair_bar(pid);
                        ms = s_row[0];
                    }
                    float sum;
#pragma unroll 1
                    for (bool again = false;; again = true) {
                        sum = probs(0, std::true_type{}, vis);
                        sum += probs(1, std::true_type{}, vis);
                        if (again || !pf_pair_or(pid, sum > kPfSumMax)) break;
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            tc::tmem_ld32(tS + 64 * half + 32 * c, x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, 32 * c + i < vis ? x[i] * sl2 : -INFINITY);
                        }
                        s_row[128 * half] = mx;
                        if (tiles > 0) good = pf_wait(bar(SM::kODone + sid), (tiles - 1) & 1u);  // O is at rest
                        if (!good) s_badp[pid - 1] = 1;
                        pf_pair_bar(pid);
                        mx = fmaxf(s_row[0], s_row[128]);
                        const bool grow = mx - ms > kPfGrow;  // from -inf, too; not where nothing is visible yet
                        const float f = grow ? ex2_approx(ms - mx) : 1.0f;
                        if (grow) ms = mx;
                        l *= f;
                        if (t > t0) {
                            tc::fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 2; c += 32) {
                                tc::tmem_ld32(tO + c, x);
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] *= f;
                                tc::tmem_st32f(tO + c, x);
                            }
                        }
                    }
                    if (s_badp[pid - 1]) {
                        ok = false;
                        break;
                    }
                    tc::tmem_st32(tS + 64 * half, pk);
                    l += sum;
                } else if (!good) {
                    break;
                }
                // keys behind the sequence's end weigh nothing, but 0 x NaN is NaN: their V rows become zero
                if (base + kPfTile > seg.len) {
                    if (!pf_wait(bar(SM::kVFull + vs), (uint32_t)(n / VS) & 1u)) s_badp[pid - 1] = 1;
                    if (half == 0 && r >= seg.len - base) {
#pragma unroll
                        for (int h = 0; h < SM::KH; ++h) {
                            uint4 *row = reinterpret_cast<uint4 *>(s + SM::V + vs * SM::OP + h * 16384 + r * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) row[i ^ (r & 7)] = make_uint4(0, 0, 0, 0);  // (eight lanes, all banks)
                        }
                    }
                    tc::fence_proxy_async_smem();
                }
                tc::fence_before();
                pf_arrive(bar(SM::kPFull + sid));
                t += dt;
                ++tiles;
            }
            if (!ok) break;
            // (warps without a row wait as well: they must not come to the next segment's end before this one's)
            const bool rest = pf_wait(bar(SM::kODone + sid), (tiles - 1) & 1u);
            if (!rest) s_badp[pid - 1] = 1;
            if (!active && !rest) continue;
            if (active) {
                const int64_t at = (int64_t)seg.place() * d.strideP + (both ? rr : turn * seg.nr + rr);
                float2 *ml = reinterpret_cast<float2 *>(w.mlp) + at;
                float2 old = {-INFINITY, 0.0f};
                if (seg.added() && mine) old = *ml;
                s_row[128 * half] = l;
                pf_pair_bar(pid);
                if (s_badp[pid - 1]) {
                    ok = false;
                    break;
                }
                tc::fence_after();
                float *O = w.Op + at * D + half * (D / 2);
                if (seg.added()) {
                    const PfSum sum(old.x, ms);
                    if (mine && half == 0) *ml = make_float2(sum.m, pf_add(old.y, sum.f0, s_row[0] + s_row[128], sum.f1));
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 8) {
                        float o[8];
                        __syncwarp();
                        tc::tmem_ld8(tO + c, o);
                        if (mine) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = pf_add(O[c + i], sum.f0, o[i], sum.f1);
                            pf_store8(O + c, o);
                        }
                    }
                } else if (mine && half == 0) {
                    *ml = make_float2(ms, s_row[0] + s_row[128]);
                }
#pragma unroll 1
                for (int c = 0; !seg.added() && c < D / 2; c += 32) {
                    float o[32];
                    __syncwarp();  // the lanes without a row skip the stores
                    tc::tmem_ld32(tO + c, o);
                    if (mine) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) pf_store8(O + c + i, o + i);
                    }
                }
                pf_pair_bar(pid);  // s_row is written again by the next segment
            }
            tc::fence_before();
            pf_arrive(bar(SM::kOEmpty + sid));
        }
    }
    if (!ok) *s_bad = 1;  // (any thread's)
    tc::fence_before();
    __syncthreads();
    if (tid == 0) w.status[blockIdx.x] = *s_bad;
    if (warp == kPfSWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, SM::TMEM_COLS);
    }
}

template <int D>
static cudaError_t launch_wide(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, cudaStream_t s) {
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * kChunk;
    if (!make_tmap_bf16(&tk, a.Kp, rows, D, kChunk) || !make_tmap_bf16(&tv, a.Vp, rows, D, kChunk))
        return cudaErrorInvalidValue;
    const size_t smem = PfSmem<D>::dyn(d.blocks);
    cudaError_t e = allow_smem<prefix_wide_kernel<D>>(PfSmem<D>::dyn(kPagedMaxBatch / 32));
    if (e != cudaSuccess) return e;
    HSA_PROF("prefix_wide", s);
    return launch_pdl(prefix_wide_kernel<D>, dim3(ctas), dim3(kPfThreads), smem, s, a, d, w, tk, tv);
}

cudaError_t launch_prefix_wide(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, cudaStream_t s) {
    return a.D == 128 ? launch_wide<128>(a, d, w, ctas, s) : launch_wide<64>(a, d, w, ctas, s);
}

}  // namespace hsa
