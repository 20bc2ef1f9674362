// prefix_few.cu -- segments of up to 64 query rows of the shared-prefix decode: the requests' own pages, and the
// prefix of small batches. Bound by the bytes of K and V, so everything is laid out to keep copies in flight.
//
// Transposed products, keys on the tensor core's 128 rows and the few query rows on its N side, so that no
// part of an MMA or of the softmax is spent on padding rows:
//   S^T = K Q^T    (128 keys x N, fp32 in TMEM; thread = key)       P^T = exp2(S^T scale' - m) (bf16, to shared memory)
//   O^T += V^T P^T (D x N, fp32 in TMEM; thread = dim)
// P is rounded to bf16, here and in the wide kernel, because both operands of a product have one type and V's is bf16: a term is off
// by up to 2^-8, which averages out over the keys (the result's error against 64 bits is 1.4 times that of its own rounding). P in
// two parts would double the products and P's way through shared memory. The row sums add the terms before their rounding.
// The reference m of a row need not be its maximum: the final quotient cancels it, and P (bf16) and the fp32 sums keep
// their relative precision as long as nothing leaves their range. So m is the logit of the first key that the row sees
// in the segment, and moves only when a later one exceeds it by more than 2^59 (a term stays below 2^64, its sum over the 2^31
// keys of a prefix and a request, times V below 2^28, below 2^123; what is 2^126 below m is less than 2^-126 of the sum, which is at
// least 1). Then the warpgroup reduces the maxima over the keys, rescales O^T in TMEM and does the tile again; every other tile
// costs a thread one exponential per row and one barrier with a vote. Row sums stay per thread until the segment ends.
//
// Measured, per tile of 128 keys and SM: D = 128, 16 rows 1.39 us = 64 KB at 7.0 TB/s over 148 SMs, out of L2 0.60 us; 64 rows
// 1.43 us, out of L2 0.77; D = 64, 16 rows 0.64 us, 64 rows 0.76, out of L2 0.75: there the softmax bounds it (1400
// cycles: exponentials of 64 rows 512, waits, vote and hand-over the rest). The start (schedule 4400 cycles, first tile 5000)
// and the end of a kernel are 5 us of a small call.
//
// Persistent, warp-specialised, one CTA per SM; the CTA's tiles are numbered through all its segments:
//   warps 0-3, 4-7  softmax of the lower and the upper half of the rows, both on every tile (in turn on the tiles, 64 rows
//               a thread, they took longer for a tile and kept two partials);
//               S^T and P^T of two or four tiles, so that the products of one run under the softmax of another;
//   warp 8      issues S^T(n), in order, when its operands are there and its S^T and P^T buffers have been read;
//   warp 9      issues O^T(n), in order, when P^T(n) and V are there. (Two warps that sleep in their waits: one that polled
//               for both took issue slots from the softmax warps beside it.) O^T of two segments, so that one is
//               read out under the next one's products;
//   warp 10     walks the segments, announces them to the other warps and copies K and V tiles by TMA, page by
//               page (64 rows of one head are contiguous);
//   warp 11     Q rows by cp.async, padded with zero rows to N.
#include <cuda.h>

#include <type_traits>

#include "prefix.cuh"
#include "profile.h"

namespace hsa {

constexpr int kFwSWarp = 8, kFwOWarp = 9, kFwTmaWarp = 10, kFwQWarp = 11;
constexpr int kFwThreads = 32 * (kFwQWarp + 1);
constexpr float kFwGrow = 59.0f, kFwSumMax = 0x1p64f;  // a sum of 32 terms of at most 2^59

template <int D, int NR>  // NR: rows per segment at most
struct FwSmem {
    static constexpr int KH = D / 64;                     // 128-byte column blocks of D
    static constexpr uint32_t OP = KH * 16384;            // one K or V tile [128][D]
    static constexpr uint32_t QB = KH * NR * 128;         // Q rows [NR][D]
    static constexpr uint32_t PB = 16384;                 // P^T [128 keys][64 rows]
    static constexpr int KS = D == 64 ? 4 : 2, VS = D == 64 ? 4 : NR == 64 ? 2 : 3;
    // S^T and P^T buffers. A tile goes through its products and its softmax in some 2500 cycles; its bytes take half
    // as long with D = 64, so four tiles are on their way there, two with D = 128.
    static constexpr int NB = D == 64 ? 4 : 2;
    static_assert(VS >= NB, "the softmax's waits for V");
    static constexpr uint32_t K = 0, V = K + KS * OP, P = V + VS * OP, Q = P + NB * PB;
    static constexpr uint32_t BAR = Q + 2 * QB;
    static constexpr int kKFull = 0, kKEmpty = KS, kVFull = 2 * KS, kVEmpty = 2 * KS + VS, kQFull = 2 * KS + 2 * VS,
                         kQEmpty = kQFull + 2, kSFull = kQEmpty + 2, kPFull = kSFull + NB,
                         kODone = kPFull + NB, kOEmpty = kODone + NB, kSegFull = kOEmpty + 2, kSegEmpty = kSegFull + kPfRing,
                         NBAR = kSegEmpty + kPfRing;
    static constexpr uint32_t RING = (BAR + 8 * NBAR + 15) / 16 * 16;
    static constexpr uint32_t MS = RING + kPfRing * sizeof(PfNote);       // float[NR]: -m * scale * log2(e), inf while a row sees nothing
    static constexpr uint32_t LIM = MS + NR * 4;                          // int[NR]: keys that the row sees
    static constexpr uint32_t RED = LIM + NR * 4;                         // float[4][NR]: of a row and a warp's keys (maxima, sums)
    static constexpr uint32_t FAC = RED + 4 * NR * 4;                     // float[NR]: rescaling
    static constexpr uint32_t MISC = FAC + NR * 4;                        // TMEM base, bad[3]
    static constexpr uint32_t PLAN = (MISC + 16 + 15) / 16 * 16;
    static constexpr uint32_t BCUM = PLAN + (sizeof(PfPlan) + 15) / 16 * 16;  // int[blocks + 1]
    static constexpr size_t dyn(int blocks) { return BCUM + 4 * ((size_t)blocks + 1) + 1024; }  // slack: 1 KB alignment
    static constexpr uint32_t S_COL = 0, O_COL = NB * 64, TMEM_COLS = NB == 4 ? 512 : 256;
};
static_assert(FwSmem<128, 64>::dyn(kPagedMaxBatch / 32) <= 227 * 1024 && FwSmem<128, 32>::dyn(kPagedMaxBatch / 32) <= 227 * 1024 &&
                  FwSmem<64, 64>::dyn(kPagedMaxBatch / 32) <= 227 * 1024,
              "shared memory budget");

// Named barrier of a warpgroup that also ORs a predicate.
__device__ __forceinline__ bool fw_bar_or(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id)
        : "memory");
    return r != 0u;
}
__device__ __forceinline__ void fw_bar(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

template <int NR>
__device__ __forceinline__ void fw_ld(uint32_t taddr, float (&v)[NR]) {  // NR consecutive columns of this thread's TMEM lane
    if constexpr (NR == 8) tc::tmem_ld8(taddr, v);
    else if constexpr (NR == 16) tc::tmem_ld16(taddr, v);
    else tc::tmem_ld32(taddr, v);
}
template <int D, int NR>
__global__ void __launch_bounds__(kFwThreads, 1) prefix_few_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                   const __grid_constant__ CUtensorMap tmK,
                                                                   const __grid_constant__ CUtensorMap tmV) {
    using SM = FwSmem<D, NR>;
    constexpr int KS = SM::KS, VS = SM::VS, NB = SM::NB;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;  // 1 KB aligned (swizzle atoms)
    unsigned char *s = smem_raw + (sb - raw);
    PfNote *s_ring = reinterpret_cast<PfNote *>(s + SM::RING);
    volatile int *s_bad = reinterpret_cast<volatile int *>(s + SM::MISC) + 1;  // [2] per warpgroup, [1] any other warp's, too
    PfPlan *s_plan = reinterpret_cast<PfPlan *>(s + SM::PLAN);
    int32_t *s_bcum = reinterpret_cast<int32_t *>(s + SM::BCUM);
    auto bar = [&](int i) { return sb + SM::BAR + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kFwSWarp) tc::tmem_alloc(sb + SM::MISC, SM::TMEM_COLS);
    if (warp == kFwTmaWarp && lane == 0) {
        pf_prefetch_tmap(&tmK);
        pf_prefetch_tmap(&tmV);
    }
    if (tid == 0) {
        s_bad[0] = s_bad[1] = s_bad[2] = 0;
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
            tc::mbar_init(bar(SM::kOEmpty + i), 8);
        }
        for (int i = 0; i < NB; ++i) {
            tc::mbar_init(bar(SM::kSFull + i), 1);
            tc::mbar_init(bar(SM::kPFull + i), 8);  // a softmax warp each
            tc::mbar_init(bar(SM::kODone + i), 1);
        }
        for (int i = 0; i < kPfRing; ++i) {
            tc::mbar_init(bar(SM::kSegFull + i), 1);
            tc::mbar_init(bar(SM::kSegEmpty + i), kFwThreads / 32 - 1);  // the warps but this ring's writer
        }
        tc::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t *>(s + SM::MISC);
    if (!d.wide) pdl_wait();  // what precedes the call in its stream is visible from here on
    int64_t plen = 0;
    if (warp == kFwQWarp && !d.wide && a.max_prefix_pages > 0) plen = pf_clamp_len(a.prefix_len[0], a.max_prefix_pages);
    pf_schedule<kFwThreads>(a, d, !d.wide, true, s_plan, s_bcum, [&](int wp) {
        if (wp == kFwQWarp && plen > 0) pf_prefetch_first<D>(a, d, plen, (int)gridDim.x);
    });
    pf_publish<kFwThreads>(d, !d.wide, true, s_plan, s_bcum, w);
    bool ok = true;

    // the next announced segment; nr = 0 ends the walk
    int seg_no = 0;
    auto take = [&](PfNote &g) {
        const int slot = seg_no % kPfRing;
        if (!pf_wait(bar(SM::kSegFull + slot), (uint32_t)(seg_no / kPfRing) & 1u)) return false;
        g = s_ring[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar(SM::kSegEmpty + slot));
        ++seg_no;
        return true;
    };

    if (warp == kFwTmaWarp) {
        // ================= the walk, K and V tiles =================
        PfWalk walk(a, *s_plan, s_bcum, d);
        const int pages_all = a.num_pages;
        int n = 0;
        PfNote g;
        bool more = walk.next(g.s);
        int ids_first = 0;
        while (ok) {
            if (!more) g.s.nr = 0;
            g.n0 = n;
            const int slot = seg_no % kPfRing;
            ok = pf_wait(bar(SM::kSegEmpty + slot), ((uint32_t)(seg_no / kPfRing) & 1u) ^ 1u);
            if (!ok) break;
            if (lane == 0) {
                s_ring[slot] = g;
                tc::mbar_arrive(bar(SM::kSegFull + slot));
            }
            ++seg_no;
            if (!more) break;
            const PfSeg seg = g.s;
            const PfPages pages(seg, pages_all);
            int ids = n == 0 ? pages.fetch(seg.tile0) : ids_first, ids_next = 0;
            for (int t = 0; t < seg.nt; ++t, ++n) {
                if (t % 16 == 0) {
                    if (t > 0) ids = ids_next;
                    ids_next = pages.fetch(seg.tile0 + t + 16);
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
                if (t == min(seg.nt - 1, 1)) {  // the next segment and its first pages, while this one's copies run
                    more = walk.next(g.s);
                    if (more) ids_first = PfPages(g.s, pages_all).fetch(g.s.tile0);
                }
            }
        }
        // every copy has landed before the CTA may exit, however the walk ended
        for (int i = max(0, n - KS); i < n; ++i) pf_wait(bar(SM::kKFull + i % KS), (uint32_t)(i / KS) & 1u);
        for (int i = max(0, n - VS); i < n; ++i) pf_wait(bar(SM::kVFull + i % VS), (uint32_t)(i / VS) & 1u);
    } else if (warp == kFwQWarp) {
        // ================= Q rows =================
        PfNote g;
        while (true) {
            const int q = seg_no & 1;
            const uint32_t use = (uint32_t)(seg_no >> 1);
            ok = take(g);
            if (!ok || g.s.nr == 0) break;
            ok = pf_wait(bar(SM::kQEmpty + q), (use & 1u) ^ 1u);
            if (!ok) break;
            const uint32_t dst = sb + SM::Q + q * SM::QB;
            pf_copy_q<D>(a, d, g.s, 0, g.s.nr, (g.s.nr + 15) / 16 * 16,
                         [&](int r, int ch) { return dst + (ch >> 3) * (NR * 128) + tc::sw128(r, ch & 7); });
            pf_cp_async_arrive(bar(SM::kQFull + q));  // fires when this thread's copies have landed
        }
        cp_async_commit();
        cp_async_wait<0>();  // nothing in flight when the CTA exits
    } else if (warp == kFwSWarp) {
        // ================= S^T products: the whole warp runs the loop, one elected lane issues =================
        PfNote g;
        int n = 0;
        while (true) {
            const int q = seg_no & 1;
            const uint32_t use = (uint32_t)(seg_no >> 1);
            ok = take(g);
            if (!ok || g.s.nr == 0) break;
            const uint32_t id = tc::idesc_bf16(128, (g.s.nr + 15) / 16 * 16, 0, 0);
            const uint64_t dq = tc::desc_kmajor(sb + SM::Q + q * SM::QB);
            for (int t = 0; t < g.s.nt; ++t, ++n) {
                const int buf = n % NB, ks = n % KS;
                ok = pf_wait(bar(SM::kKFull + ks), (uint32_t)(n / KS)) && (t > 0 || pf_wait(bar(SM::kQFull + q), use));
                // S^T and P^T of the tile that had their buffers before have been read
                if (ok && n >= NB) ok = pf_wait(bar(SM::kODone + buf), (uint32_t)(n / NB - 1));
                if (!ok) break;
                tc::fence_after();
                if (t == 0) tc::fence_proxy_async_smem();  // the Q rows came by cp.async (generic proxy)
                const uint64_t dk = tc::desc_kmajor(sb + SM::K + ks * SM::OP);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)  // (a descriptor's low bits are its address / 16)
                    tc::mma_bf16_ss_w(tmem + SM::S_COL + buf * 64, dk + ((uint64_t)((k >> 2) * 16384 + (k & 3) * 32) >> 4),
                                      dq + ((uint64_t)((k >> 2) * (NR * 128) + (k & 3) * 32) >> 4), id, k > 0 ? 1u : 0u);
                tc::commit_w(bar(SM::kSFull + buf));
                tc::commit_w(bar(SM::kKEmpty + ks));
                if (t == g.s.nt - 1) tc::commit_w(bar(SM::kQEmpty + q));
            }
            if (!ok) break;
        }
        __syncwarp();
    } else if (warp == kFwOWarp) {
        // ================= O^T products =================
        PfNote g;
        int n = 0;
        while (true) {
            const int ob = seg_no & 1;
            const uint32_t use = (uint32_t)(seg_no >> 1);
            ok = take(g);
            if (!ok || g.s.nr == 0) break;
            // A and B MN-major. The second 64 rows of A: dims 64 .. 127, or, with D = 64, whatever follows the tile (lanes
            // that are not read)
            const uint32_t id = tc::idesc_bf16(128, (g.s.nr + 15) / 16 * 16, 1, 1);
            for (int t = 0; t < g.s.nt; ++t, ++n) {
                const int buf = n % NB, vs = n % VS;
                ok = pf_wait(bar(SM::kVFull + vs), (uint32_t)(n / VS));
                // O^T of the segment two before has been read out
                if (ok && t == 0) ok = pf_wait(bar(SM::kOEmpty + ob), use ^ 1u);
                if (ok) ok = pf_wait(bar(SM::kPFull + buf), (uint32_t)(n / NB));
                if (!ok) break;
                tc::fence_after();
                const uint64_t dv = tc::desc_mnmajor(sb + SM::V + vs * SM::OP, 16384);
                const uint64_t dp = tc::desc_mnmajor(sb + SM::P + buf * SM::PB, 16384);
#pragma unroll
                for (int k = 0; k < kPfTile / 16; ++k)
                    tc::mma_bf16_ss_w(tmem + SM::O_COL + ob * 64, dv + (uint64_t)k * (2048 >> 4), dp + (uint64_t)k * (2048 >> 4), id,
                                      t > 0 || k > 0 ? 1u : 0u);
                tc::commit_w(bar(SM::kODone + buf));
                tc::commit_w(bar(SM::kVEmpty + vs));
            }
            if (!ok) break;
        }
        __syncwarp();
    } else {
        // ================= softmax of half of the rows; thread = key, then thread = dim =================
        constexpr int H = NR / 2;
        const int half = warp >> 2, r = tid & 127, wq = warp & 3, bid = 1 + half;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        float *nms = reinterpret_cast<float *>(s + SM::MS) + half * H, *s_fac = reinterpret_cast<float *>(s + SM::FAC) + half * H;
        float *s_red = reinterpret_cast<float *>(s + SM::RED) + half * 4 * H;
        int *lims = reinterpret_cast<int *>(s + SM::LIM) + half * H;
        const float sl2 = a.scale * 1.4426950408889634f;
        PfNote g;
        // A warp whose wait ran out says so and still comes to the barriers, and the warpgroup leaves together
        while (true) {
            const int ob = seg_no & 1;
            if (!take(g)) s_bad[half] = 1;
            fw_bar(bid);
            if (s_bad[half]) {
                ok = false;
                break;
            }
            if (g.s.nr == 0) break;
            const PfSeg &seg = g.s;
            // this warpgroup's rows, by eights (none: it keeps step)
            const int split = (seg.nr + 15) / 16 * 8, row0 = half ? split : 0, rows = half ? seg.nr - split : min(seg.nr, split);
            const uint32_t tO = tmem + lane_off + SM::O_COL + ob * 64 + row0;
            const int min_lim = pf_min_limit(a, seg);
            if (r < H) {  // rows that are nobody's: -1 (they see nothing, where it is asked: in tiles with an edge)
                const int lim = r < rows ? pf_limit(a, seg, d, row0 + r) : -1;
                lims[r] = lim == INT32_MAX ? -1 : lim;
            }
            fw_bar(bid);
            float l[H], off[H];  // sums over this thread's keys; the references (nms) at hand
#pragma unroll
            for (int i = 0; i < H; ++i) l[i] = off[i] = 0.0f;
            auto load_off = [&]() {
#pragma unroll
                for (int i = 0; i < H; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(nms + i);
                    off[i] = v.x, off[i + 1] = v.y, off[i + 2] = v.z, off[i + 3] = v.w;
                }
            };
            float p[H];
            // P^T of tile t's key to shared memory, kept in p for the row sums; false if a term leaves the range
            auto probs = [&](int t, uint32_t tS, auto with_edge, uint32_t flags) {
                const int buf = (g.n0 + t) % NB;
                unsigned char *s_p = s + SM::P + buf * SM::PB;
                float2 sum = {0.0f, 0.0f};
                fw_ld<H>(tS, p);
#pragma unroll
                for (int c = 0; c < H / 8; ++c) {
                    if (8 * c >= rows) break;
                    uint32_t pk[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const int e = 8 * c + i;
                        float2 a0 = fma2({p[e], p[e + 1]}, {sl2, sl2}, {off[e], off[e + 1]});
                        float2 a1 = fma2({p[e + 2], p[e + 3]}, {sl2, sl2}, {off[e + 2], off[e + 3]});
                        a0 = {ex2_approx(a0.x), ex2_approx(a0.y)};
                        a1 = {ex2_approx(a1.x), ex2_approx(a1.y)};
                        if constexpr (decltype(with_edge)::value) {
                            const int key = (seg.tile0 + t) * kPfTile + r;
                            const bool page_ok = flags >> (r >> 6) & 1u;
                            const int4 lim = *reinterpret_cast<const int4 *>(lims + e);
                            a0 = {page_ok && key < lim.x ? a0.x : 0.0f, page_ok && key < lim.y ? a0.y : 0.0f};
                            a1 = {page_ok && key < lim.z ? a1.x : 0.0f, page_ok && key < lim.w ? a1.y : 0.0f};
                        }
                        sum = add2(sum, add2(a0, a1));
                        p[e] = a0.x;
                        p[e + 1] = a0.y;
                        p[e + 2] = a1.x;
                        p[e + 3] = a1.y;
                        pk[i / 2] = pack_bf16x2(a0.x, a0.y);
                        pk[i / 2 + 1] = pack_bf16x2(a1.x, a1.y);
                    }
                    *reinterpret_cast<uint4 *>(s_p + tc::sw128(r, row0 / 8 + c)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                return sum.x + sum.y <= kFwSumMax;  // (not of an infinity or NaN)
            };
            auto deliver = [&](int buf) {  // P^T (and V rows made zero) to the products; p to the row sums
                tc::fence_proxy_async_smem();
                tc::fence_before();
                pf_arrive(bar(SM::kPFull + buf));
#pragma unroll
                for (int c = 0; c < H; c += 8) {
                    if (c >= rows) break;
#pragma unroll
                    for (int i = c; i < c + 8; i += 2) {
                        const float2 sum = add2({l[i], l[i + 1]}, {p[i], p[i + 1]});
                        l[i] = sum.x;
                        l[i + 1] = sum.y;
                    }
                }
            };
            const PfPages pages(seg, a.num_pages);
            int id_next = pages.fetch(seg.tile0), block_end = 0;  // of the 16 tiles whose pages `there` tells of
            uint32_t there = 0;
            const int whole = min_lim / kPfTile - seg.tile0;  // the tiles before this one lie before every row's end
            bool redo = false;
            for (int t = 0; t < seg.nt;) {
                if (t == block_end) {
                    there = pages.there(id_next);
                    id_next = pages.fetch(seg.tile0 + t + 16);
                    block_end += 16;
                }
                // Tiles that every row sees all of, in a loop of their own: with the rare things in the same loop, what
                // the compiler did to keep the paths apart took 40% of a tile's time (2470 cycles for 64 rows, here 1460)
                const uint32_t gaps = ~(there & there >> 1) & 0x55555555u & ~0u << 2 * (t & 15);
                const int stop = min(min(seg.nt, whole), gaps ? block_end - 16 + (__ffs(gaps) - 1) / 2 : block_end);
                if (t > 0 && !redo) {
                    for (; t < stop; ++t) {
                        const int n = g.n0 + t, buf = n % NB;
                        const uint32_t tS = tmem + lane_off + SM::S_COL + buf * 64 + row0;
                        const bool good = pf_wait(bar(SM::kSFull + buf), (uint32_t)(n / NB));
                        tc::fence_after();
                        bool high = !good;
                        if (rows > 0) high |= !probs(t, tS, std::false_type{}, 3u);
                        redo = fw_bar_or(bid, high);
                        if (redo) break;
                        deliver(buf);
                    }
                    if (t >= seg.nt) break;
                    if (t == block_end && !redo) continue;
                }
                redo = false;
                // Any tile: the first, the ones with an edge, and those where a term left the range
                const uint32_t flags = there >> 2 * (t & 15) & 3u;  // of this tile's two pages
                const int n = g.n0 + t, buf = n % NB, vs = n % VS, base = (seg.tile0 + t) * kPfTile;
                const uint32_t tS = tmem + lane_off + SM::S_COL + buf * 64 + row0;
                // S^T is there, and P^T's buffer has been read (so every V filling before this
                // tile's in its slot is over, too, which makes the wait for it by its parity exact)
                const bool good = pf_wait(bar(SM::kSFull + buf), (uint32_t)(n / NB));
                tc::fence_after();
                if (!good) s_bad[half] = 1;
                const bool page_ok = flags >> (r >> 6) & 1u;
                if (t == 0) {  // the references: the first key, or the 65th where the first page is bad
                    const int lead = flags & 1u ? 0 : 64;
                    if (r >> 5 == lead >> 5 && good && rows > 0) {
                        fw_ld<H>(tS, p);
                        if (lane == 0) {
#pragma unroll
                            for (int i = 0; i < H; i += 4) *reinterpret_cast<float4 *>(s_fac + i) = make_float4(p[i], p[i + 1], p[i + 2], p[i + 3]);
                        }
                        __syncwarp();
                        if (lane < H) {
                            const int lim = lims[lane];
                            nms[lane] = lim < 0 ? 0.0f : page_ok && base + lead < lim ? -s_fac[lane] * sl2 : INFINITY;
                        }
                    }
                    fw_bar(bid);
                    load_off();
                }
                bool high = false;
                if (good && rows > 0) high = !probs(t, tS, std::true_type{}, flags);
                const bool any = fw_bar_or(bid, high);
                if (s_bad[half]) {
                    ok = false;
                    break;
                }
                if (any) {
                    // O^T is at rest once the tile before is in it
                    if (n >= 1 && !pf_wait(bar(SM::kODone + (n - 1) % NB), (uint32_t)((n - 1) / NB))) s_bad[half] = 1;
                    tc::fence_after();
                    // maxima over the tile's keys, of logit * log2(e)
                    fw_ld<H>(tS, p);
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const bool see = page_ok && base + r < lims[i];
                        const uint32_t u = __reduce_max_sync(0xffffffffu, float_to_ordered(see ? p[i] * sl2 : -INFINITY));
                        if (lane == i % 32) s_red[wq * H + i] = ordered_to_float(u);
                    }
                    fw_bar(bid);
                    if (r < H) {
                        const float mx = fmaxf(fmaxf(s_red[r], s_red[H + r]), fmaxf(s_red[2 * H + r], s_red[3 * H + r]));
                        const float old = -nms[r];
                        const bool grow = mx - old > kFwGrow;  // from -inf, too; not where nothing is visible yet (-inf, NaN)
                        s_fac[r] = grow ? ex2_approx(old - mx) : 1.0f;
                        if (grow) nms[r] = -mx;
                    }
                    fw_bar(bid);
                    load_off();
#pragma unroll
                    for (int i = 0; i < H; ++i) l[i] *= s_fac[i];
#pragma unroll 1
                    for (int c = 0; t > 0 && c < rows; c += 8) {  // (the columns behind are the other warpgroup's)
                        float o[8];
                        uint32_t u[8];
                        tc::tmem_ld8(tO + c, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(o[i] * s_fac[c + i]);
                        tc::tmem_st8(tO + c, u);
                    }
                    probs(t, tS, std::true_type{}, flags);
                }
                // a key behind the sequence's end weighs nothing, but 0 x NaN is NaN: its V row becomes zero
                if (half == 0 && base + kPfTile > seg.len) {
                    if (!pf_wait(bar(SM::kVFull + vs), (uint32_t)(n / VS))) s_bad[half] = 1;  // seen at the next barrier
                    if (base + r >= seg.len) {
#pragma unroll
                        for (int h = 0; h < SM::KH; ++h) {
                            uint4 *row = reinterpret_cast<uint4 *>(s + SM::V + vs * SM::OP + h * 16384 + r * 128);
#pragma unroll
                            for (int i = 0; i < 8; ++i) row[i ^ (r & 7)] = make_uint4(0, 0, 0, 0);  // (eight lanes, all banks)
                        }
                    }
                }
                deliver(buf);
                ++t;
            }
            if (!ok) break;
            // the warp's row sums: each step halves the rows a lane holds (8, 16 or 32 rows over 32 lanes)
#pragma unroll
            for (int h = 16; h >= H; h >>= 1)
#pragma unroll
                for (int i = 0; i < H; ++i) l[i] += __shfl_xor_sync(0xffffffffu, l[i], h);
#pragma unroll
            for (int h = H / 2; h > 0; h >>= 1) {
                const bool up = lane & h;
#pragma unroll
                for (int i = 0; i < H / 2; ++i) {
                    if (i < h) {
                        const float send = up ? l[i] : l[i + h], keep = up ? l[i + h] : l[i];
                        l[i] = keep + __shfl_xor_sync(0xffffffffu, send, h);
                    }
                }
            }
            if (lane < H) s_red[wq * H + lane] = l[0];
            const int64_t at = (int64_t)seg.place() * (seg.b < 0 ? d.strideP : d.strideO) + row0;
            float *O = (seg.b < 0 ? w.Op : w.Oo) + at * D;
            fw_bar(bid);
            if (r < rows) {
                const float sum = (s_red[r] + s_red[H + r]) + (s_red[2 * H + r] + s_red[3 * H + r]);
                float2 *ml = reinterpret_cast<float2 *>(seg.b < 0 ? w.mlp : w.mlo) + at + r;
                if (seg.added()) {
                    const float2 old = *ml;
                    const PfSum both(old.x, -nms[r]);
                    *ml = make_float2(both.m, pf_add(old.y, both.f0, sum, both.f1));
                    s_fac[r] = both.f0;
                    nms[r] = both.f1;
                } else {
                    *ml = make_float2(-nms[r], sum);
                }
            }
            const int last = g.n0 + seg.nt - 1;
            if (!pf_wait(bar(SM::kODone + last % NB), (uint32_t)(last / NB))) s_bad[half] = 1;  // seen at the next barrier
            tc::fence_after();
            if (seg.added()) {
                fw_bar(bid);  // the factors
#pragma unroll 1
                for (int c = 0; c < rows; c += 8) {
                    float o[8];
                    tc::tmem_ld8(tO + c, o);
                    if (r < D) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (c + i < rows) O[(size_t)(c + i) * D + r] = pf_add(O[(size_t)(c + i) * D + r], s_fac[c + i], o[i], nms[c + i]);
                    }
                    __syncwarp();
                }
            } else if (rows > 0) {
                float o[H];
                fw_ld<H>(tO, o);
                if (r < D) {
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        if (i < rows) O[(size_t)i * D + r] = o[i];
                }
                __syncwarp();
            }
            tc::fence_before();
            pf_arrive(bar(SM::kOEmpty + ob));
        }
    }
    if (!ok) s_bad[2] = 1;
    tc::fence_before();
    __syncthreads();
    if (d.wide) pdl_wait();  // the kernel before, whose partials the join reads, too
    pdl_launch_dependents();
    if (tid == 0) w.status[kPfCtas + blockIdx.x] = s_bad[0] | s_bad[1] | s_bad[2];
    if (warp == kFwSWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, SM::TMEM_COLS);
    }
}

template <int D, int NR>
static cudaError_t launch_few(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, cudaStream_t s) {
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * kChunk;
    if (!make_tmap_bf16(&tk, a.Kp, rows, D, kChunk) || !make_tmap_bf16(&tv, a.Vp, rows, D, kChunk))
        return cudaErrorInvalidValue;
    const size_t smem = FwSmem<D, NR>::dyn(d.blocks);
    cudaError_t e = allow_smem<prefix_few_kernel<D, NR>>(FwSmem<D, NR>::dyn(kPagedMaxBatch / 32));
    if (e != cudaSuccess) return e;
    HSA_PROF("prefix_few", s);
    return launch_pdl(prefix_few_kernel<D, NR>, dim3(ctas), dim3(kFwThreads), smem, s, a, d, w, tk, tv);
}

cudaError_t launch_prefix_few(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, cudaStream_t s) {
    const int rows = d.wide ? d.Ro : d.Rp;  // of the largest segment, or more; Rp >= Ro
    if (a.D == 128)
        return rows <= 16   ? launch_few<128, 16>(a, d, w, ctas, s)
               : rows <= 32 ? launch_few<128, 32>(a, d, w, ctas, s)
                            : launch_few<128, 64>(a, d, w, ctas, s);
    return rows <= 16   ? launch_few<64, 16>(a, d, w, ctas, s)
           : rows <= 32 ? launch_few<64, 32>(a, d, w, ctas, s)
                        : launch_few<64, 64>(a, d, w, ctas, s);
}

}  // namespace hsa
