// prefix_wide.cu -- segments of more than 64 query rows of the shared-prefix decode: the prefix of large batches,
// a matrix product with (requests x query heads x tokens) rows, bound by the tensor cores and the exponentials.
//
// S = Q K^T (128 rows x 128 keys, fp32 in TMEM; thread = row), P = exp2(S scale' - m) as bf16 over S in TMEM, which
// is the A operand of O += P V (128 x D, fp32 in TMEM). The accumulator is rescaled only when a row's maximum
// grows by more than 2^8 (then P would leave a comfortable range; up to that the old maximum serves as well, since
// the final quotient cancels it).
//
// Persistent, warp-specialised kernel, one CTA per SM:
//   warps 0-3, 4-7  two softmax warpgroups = two STREAMS, one thread per row. A segment of more than
//               128 rows gives each stream 128 of them and both read every tile; a smaller one gives both
//               streams the same rows and alternates the tiles between them (each keeps a partial of its own),
//               so that one stream's products run under the other's softmax either way;
//   warp 8      MMA issuer: S and O of both streams, whichever is ready;
//   warp 9      K and V tiles by TMA, page by page (64 rows of one head are contiguous);
//   warps 10-11 Q rows by cp.async.
#include <cuda.h>

#include "prefix.cuh"
#include "profile.h"

namespace hsa {

constexpr int kPfMmaWarp = 8, kPfTmaWarp = 9, kPfQWarp = 10, kPfQWarps = 2;
constexpr int kPfThreads = 32 * (kPfQWarp + kPfQWarps);

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
    static constexpr uint32_t BCUM = PLAN + (sizeof(PfPlan) + 15) / 16 * 16;  // int[blocks + 1]
    static constexpr size_t dyn(int blocks) { return BCUM + 4 * ((size_t)blocks + 1) + 1024; }  // slack: 1 KB alignment
    static constexpr uint32_t S_COL = 0, O_COL = 2 * kPfTile, TMEM_COLS = 512;
};
static_assert(PfSmem<128>::dyn(256) <= 227 * 1024 && PfSmem<64>::dyn(256) <= 227 * 1024, "shared memory budget");

// Do both streams read every tile of the segment (each for rows of its own)? The tiles of stream s otherwise.
__device__ __forceinline__ bool pf_both(const PfSeg &s) { return s.nr > kPfTile; }
__device__ __forceinline__ int pf_count(const PfSeg &s, int sid) { return pf_both(s) ? s.nt : (s.nt + 1 - sid) >> 1; }

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) prefix_wide_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                    const bool take_prefix, const bool take_own,
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
    int32_t *s_bcum = reinterpret_cast<int32_t *>(s + SM::BCUM);
    auto bar = [&](int i) { return sb + SM::BAR + 8u * (uint32_t)i; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kPfMmaWarp) tc::tmem_alloc(sb + SM::TMEM, SM::TMEM_COLS);
    if (warp == kPfTmaWarp && lane == 0) {
        pf_prefetch_tmap(&tmK);
        pf_prefetch_tmap(&tmV);
    }
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
    pdl_launch_dependents();  // the few-rows kernel may come in as SMs fall free; the join waits for this grid's end
    pf_schedule<kPfThreads>(a, d, take_prefix, take_own, s_plan, s_bcum);
    pf_publish<kPfThreads>(d, take_prefix, take_own, s_plan, s_bcum, w);
    bool ok = true;
    PfWalk walk(a, *s_plan, s_bcum, d);
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
            const bool both = pf_both(seg);
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
                const bool both = pf_both(c.seg);
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
                c.cnt = pf_count(c.seg, sid);
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
                const bool both = pf_both(c.seg);
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
                        if (both || pf_count(c.seg, sid ^ 1) == 0) tc::commit_w(bar(SM::kQEmpty + c.q));
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
            const int cnt = pf_count(seg, sid);
            if (cnt == 0) continue;
            const bool both = pf_both(seg);
            const int rr = both ? sid * kPfTile + r : r;
            const bool mine = rr < seg.nr;
            const bool active = rr - lane < seg.nr;  // does this warp hold any row?
            // rows that are nobody's compute something that is never read
            const int lim = mine ? pf_limit(a, seg, d, rr) : INT32_MAX;
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
                if (mine) reinterpret_cast<float2 *>(seg.b < 0 ? w.mlp : w.mlo)[at] = make_float2(m * sl2, l);
            }
            tc::fence_before();
            tc::mbar_arrive(bar(SM::kOEmpty + sid));
        }
    }
    if (!ok) *s_bad = 1;
    tc::fence_before();
    __syncthreads();
    if (tid == 0) w.status[blockIdx.x] = *s_bad;
    if (warp == kPfMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, SM::TMEM_COLS);
    }
}

template <int D>
static cudaError_t launch_wide(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, bool prefix, bool own,
                               cudaStream_t s) {
    CUtensorMap tk, tv;
    const uint64_t rows = (uint64_t)a.num_pages * a.Hkv * kChunk;
    if (!make_tmap_bf16(&tk, a.Kp, rows, D, kChunk) || !make_tmap_bf16(&tv, a.Vp, rows, D, kChunk))
        return cudaErrorInvalidValue;
    const size_t smem = PfSmem<D>::dyn(d.blocks);
    cudaError_t e = allow_smem<prefix_wide_kernel<D>>(smem);
    if (e != cudaSuccess) return e;
    HSA_PROF("prefix_wide", s);
    return launch_pdl(prefix_wide_kernel<D>, dim3(ctas), dim3(kPfThreads), smem, s, a, d, w, prefix, own, tk, tv);
}

cudaError_t launch_prefix_wide(const PrefixArgs &a, const PfDims &d, const PfWork &w, int ctas, bool prefix, bool own,
                               cudaStream_t s) {
    return a.D == 128 ? launch_wide<128>(a, d, w, ctas, prefix, own, s) : launch_wide<64>(a, d, w, ctas, prefix, own, s);
}

}  // namespace hsa
