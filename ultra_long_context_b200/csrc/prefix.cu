// prefix.cu -- the shared-prefix decode: its launches, its workspace, and the join of the segments' partials.
// How the work is divided stands in prefix.cuh.
#include <type_traits>

#include "prefix.cuh"
#include "profile.h"

namespace hsa {

// Joins a row's partials: M = max m_i, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i. `wpr` warps of a block (1, 2, 4
// or 8) share a row's partials, each with a maximum of its own, so that a few rows of many partials are not
// read one after the other. Bound by latency: the plan, then a row's statistics and, at the same time, its first
// partials: 4 us, of which 1 us is the launch, wherever a row has few partials; 7 us for 2048 rows of 19 (20 MB). More warps
// per row, more loads in flight or fewer registers took longer (up to 109 us for 101 in all with four times the warps).
// blockIdx.y is the request.
constexpr int kPfJoinThreads = 256, kPfJoinWarps = kPfJoinThreads / 32, kPfJoinLoads = 8;
constexpr int kPfJoinFill = 16;  // warps per SM, about, from which on rows are not split further

template <int D>
__global__ void __launch_bounds__(kPfJoinThreads) prefix_join_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                     int ctas, int wpr, int request_rows) {
    constexpr int V = D / 32;  // columns per lane
    using Vec = std::conditional_t<V == 4, float4, float2>;
    __shared__ float s_acc[kPfJoinWarps][D], s_M[kPfJoinWarps], s_L[kPfJoinWarps];
    pdl_launch_dependents();  // what follows may set itself up; it waits for this grid's end before it reads
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp & (wpr - 1);
    const int b = blockIdx.y, bl = b & ~31, hr_n = a.Hkv * d.Rgo;
    const int want = (int)blockIdx.x * (kPfJoinWarps / wpr) + warp / wpr, rem = min(want, request_rows - 1);
    const int h = rem / d.Ro, ro = rem - h * d.Ro;  // (row counts stay below 2^31 / D)
    const int rp = b * d.Ro + ro, rg = rp / d.gp, rr = rp - rg * d.gp, nr = min(d.gp, d.Rp - rg * d.gp);
    const int per = d.wide && nr <= kPfTile ? 2 : 1;  // streams with a partial of the row
    pdl_wait();
    if (blockIdx.x == 0 && b == 0 && warp == 0) {
        int bad = 0;
        for (int i = lane; i < ctas; i += 32) bad |= (d.wide ? w.status[i] : 0) | w.status[kPfCtas + i];
        bad = __any_sync(0xffffffffu, bad != 0);
        if (lane == 0) *w.err = bad;
    }
    const PfPlan p = *w.planP, po = *w.planO;
    const int cum0 = w.bcum[bl >> 5];
    // the lengths of the row's block of 32 requests, a lane each
    const int64_t len = bl + lane < a.B ? pf_clamp_len(a.own_len[bl + lane], a.max_pages) : -1;
    const int wl = pf_weight(len), wt = __shfl_sync(0xffffffffu, wl, b & 31);
    const int cum = cum0 + __reduce_add_sync(0xffffffffu, lane < (b & 31) ? wl : 0);
    const bool live = __shfl_sync(0xffffffffu, (int)(len >= 0), b & 31) != 0;
    const int np = live && p.items > 0 ? p.nsplit * per : 0;  // prefix partials, and own ones: CTAs i0 .. i0 + no - 1
    int i0 = 0, no = 0;
    const int hr = h * d.Rgo + ro / kPfFewRows;
    const int64_t x0 = (int64_t)cum * hr_n + (int64_t)hr * wt;
    if (wt > 0) {
        i0 = po.cta_of(x0);
        no = po.cta_of(x0 + wt - 1) - i0 + 1;
    }
    const int total = np + no;
    // partial idx: its place (rows of D), or -1
    auto place = [&](int idx) -> int {
        if (idx < np) {
            const int k = per == 2 ? idx >> 1 : idx, st = per == 2 ? idx & 1 : 0;
            return st < min(p.run, p.tiles - k * p.run) ? ((k * a.Hkv + h) * d.Rgp + rg) * d.strideP + st * nr + rr : -1;
        }
        const int i = i0 + (idx - np);
        const int nt = pf_tile_at(min(po.start(i + 1), x0 + wt) - x0) - pf_tile_at(max(po.start(i), x0) - x0);
        return nt > 0 ? (b * hr_n + hr + i) * d.strideO + ro % kPfFewRows : -1;
    };
    float M = -INFINITY, acc[V] = {}, L = 0.0f;
    for (int base = wi; base < total; base += 32 * wpr) {
        const int idx = base + wpr * lane, at = idx < total ? place(idx) : -1;
        float2 ml = {-INFINITY, 0.0f};
        if (at >= 0) ml = reinterpret_cast<const float2 *>(idx < np ? w.mlp : w.mlo)[at];
        const float *src = at < 0 ? nullptr : (idx < np ? w.Op : w.Oo) + (size_t)at * D;
        const int cnt = min(32, (total - base + wpr - 1) / wpr);
        float f = 0.0f;
#pragma unroll 1
        for (int k0 = 0; k0 < cnt; k0 += kPfJoinLoads) {
            Vec o[kPfJoinLoads];
#pragma unroll
            for (int k = 0; k < kPfJoinLoads; ++k) {
                const auto O = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k0 + k));
                o[k] = Vec{};
                if (O) o[k] = *reinterpret_cast<const Vec *>(O + lane * V);
            }
            if (k0 == 0) {
                float top = ml.x;
#pragma unroll
                for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                const float M1 = fmaxf(M, top), g = M > -INFINITY ? ex2_approx(M - M1) : 0.0f;
                f = ml.x > -INFINITY ? ex2_approx(ml.x - M1) : 0.0f;
                M = M1;
                L = fmaf(ml.y, f, L * g);
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] *= g;
            }
#pragma unroll
            for (int k = 0; k < kPfJoinLoads; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k0 + k);
                if (fk == 0.0f) continue;  // (what a row without a visible key left there may be anything)
                acc[0] = fmaf(fk, o[k].x, acc[0]);
                acc[1] = fmaf(fk, o[k].y, acc[1]);
                if constexpr (V == 4) {
                    acc[2] = fmaf(fk, o[k].z, acc[2]);
                    acc[3] = fmaf(fk, o[k].w, acc[3]);
                }
            }
        }
    }
    L = warp_sum(L);
    if (wpr > 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
        if (lane == 0) {
            s_M[warp] = M;
            s_L[warp] = L;
        }
        __syncthreads();
        if (wi > 0) return;
        const float M0 = M;
        for (int k = 1; k < wpr; ++k) M = fmaxf(M, s_M[warp + k]);
        const float f0 = M0 > -INFINITY ? ex2_approx(M0 - M) : 0.0f;
        L *= f0;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= f0;
        for (int k = 1; k < wpr; ++k) {
            const float f = s_M[warp + k] > -INFINITY ? ex2_approx(s_M[warp + k] - M) : 0.0f;
            L = fmaf(s_L[warp + k], f, L);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(s_acc[warp + k][lane * V + i], f, acc[i]);
        }
    }
    if (want >= request_rows) return;
    const int64_t row = (int64_t)b * request_rows + rem;
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + row * D + lane * V);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) out[i] = pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if (lane == 0 && a.lse) a.lse[row] = L > 0.0f ? fmaf(M, 0.6931471805599453f, logf(L)) : -INFINITY;
}

static size_t pf_layout(void *ws, const PfDims &d, int D, PfWork *w) {
    char *base = static_cast<char *>(ws);
    size_t used = 0;
    auto take = [&](size_t n) {
        char *p = base ? base + used : nullptr;
        used += (n + 255) / 256 * 256;
        return p;
    };
    w->err = reinterpret_cast<int32_t *>(take(sizeof(int32_t)));  // first: hsa_workspace_status reads it
    w->planP = reinterpret_cast<PfPlan *>(take(sizeof(PfPlan)));
    w->planO = reinterpret_cast<PfPlan *>(take(sizeof(PfPlan)));
    w->status = reinterpret_cast<int32_t *>(take(2 * kPfCtas * sizeof(int32_t)));
    w->bcum = reinterpret_cast<int32_t *>(take(((size_t)d.blocks + 1) * sizeof(int32_t)));
    w->mlp = reinterpret_cast<float *>(take((size_t)d.max_items * d.strideP * 2 * sizeof(float)));
    w->mlo = reinterpret_cast<float *>(take((size_t)d.max_slots * d.strideO * 2 * sizeof(float)));
    w->Op = reinterpret_cast<float *>(take((size_t)d.max_items * d.strideP * D * sizeof(float)));
    w->Oo = reinterpret_cast<float *>(take((size_t)d.max_slots * d.strideO * D * sizeof(float)));
    return used;
}

size_t prefix_workspace(int B, int H, int Hkv, int Tq, int D, int max_prefix_pages, int max_pages) {
    (void)max_pages;
    PfWork w{};
    return pf_layout(nullptr, PfDims(B, H, Hkv, Tq, D, max_prefix_pages), D, &w);
}

cudaError_t launch_prefix_decode(const PrefixArgs &a, cudaStream_t s) {
    const PfDims d(a.B, a.H, a.Hkv, a.Tq, a.D, a.max_prefix_pages);
    PfWork w{};
    pf_layout(a.workspace, d, a.D, &w);
    const int sms = sm_count(), ctas = sms < kPfCtas ? sms : kPfCtas;
    cudaError_t e = cudaSuccess;
    if (d.wide) e = launch_prefix_wide(a, d, w, ctas, s);
    if (e == cudaSuccess) e = launch_prefix_few(a, d, w, ctas, s);
    if (e != cudaSuccess) return e;
    const int request_rows = a.H * a.Tq;
    int wpr = kPfJoinWarps;
    while (wpr > 1 && kPfJoinWarps / wpr < request_rows && (int64_t)a.B * request_rows * wpr > kPfJoinFill * kPfCtas) wpr /= 2;
    const int per_block = kPfJoinWarps / wpr;
    const dim3 grid((request_rows + per_block - 1) / per_block, a.B);
    HSA_PROF("prefix_join", s);
    return a.D == 128 ? launch_pdl(prefix_join_kernel<128>, grid, dim3(kPfJoinThreads), 0, s, a, d, w, ctas, wpr, request_rows)
                      : launch_pdl(prefix_join_kernel<64>, grid, dim3(kPfJoinThreads), 0, s, a, d, w, ctas, wpr, request_rows);
}

}  // namespace hsa
