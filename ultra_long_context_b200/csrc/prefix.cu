// prefix.cu -- the shared-prefix decode: its launches, its workspace, and the join of the segments' partials.
// How the work is divided stands in prefix.cuh.
#include "prefix.cuh"
#include "profile.h"

namespace hsa {

// Joins a row's partials: M = max m_i, out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i. `wpr` warps of a block (1, 2, 4
// or 8) share a row's partials, each with a maximum of its own, so that a few rows of many partials are not
// read one after the other.
constexpr int kPfJoinThreads = 256, kPfJoinWarps = kPfJoinThreads / 32;

template <int D>
__global__ void __launch_bounds__(kPfJoinThreads) prefix_join_kernel(const PrefixArgs a, const PfDims d, const PfWork w,
                                                                     int ctas, int wpr) {
    __shared__ float s_acc[kPfJoinWarps][D], s_M[kPfJoinWarps], s_L[kPfJoinWarps];
    pdl_launch_dependents();  // what follows may set itself up; it waits for this grid's end before it reads
    pdl_wait();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x < 32) {
        int bad = 0;
        for (int i = lane; i < ctas; i += 32) bad |= (d.wide ? w.status[i] : 0) | w.status[kPfCtas + i];
        bad = __any_sync(0xffffffffu, bad != 0);
        if (lane == 0) *w.err = bad;
    }
    const int warp = threadIdx.x >> 5, wi = warp & (wpr - 1);
    const int64_t rows = (int64_t)a.B * a.H * a.Tq;
    const int64_t want = (int64_t)blockIdx.x * (kPfJoinWarps / wpr) + warp / wpr, row = min(want, rows - 1);
    const PfPlan p = *w.planP, po = *w.planO;
    const int b = (int)(row / ((int64_t)a.H * a.Tq)), hr_n = a.Hkv * d.Rgo;
    const int rem = (int)(row % ((int64_t)a.H * a.Tq)), h = rem / d.Ro, ro = rem % d.Ro;
    // the lengths of the row's block of 32 requests, a lane each
    const int bl = b & ~31;
    const int64_t len = bl + lane < a.B ? pf_clamp_len(a.own_len[bl + lane], a.max_pages) : -1;
    int sum = pf_weight(len);
    const int wt = __shfl_sync(0xffffffffu, sum, b & 31);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    const int64_t cum = w.bcum[bl >> 5] + __shfl_sync(0xffffffffu, sum, b & 31) - wt;
    const bool live = __shfl_sync(0xffffffffu, (int)(len >= 0), b & 31) != 0;
    int np = 0, per = 1, nr = 0, rr = 0, rg = 0;      // prefix partials: np runs of `per` streams
    int i0 = 0, no = 0, orr = 0, obase = 0;           // own partials: CTAs i0 .. i0 + no - 1
    int64_t x0 = 0;
    if (live) {
        const int rp = b * d.Ro + ro;
        rg = rp / d.gp;
        rr = rp - rg * d.gp;
        nr = min(d.gp, d.Rp - rg * d.gp);
        per = d.wide && nr <= kPfTile ? 2 : 1;
        np = p.items > 0 ? p.nsplit : 0;
        if (wt > 0) {
            const int hr = h * d.Rgo + ro / kPfFewRows;
            x0 = cum * hr_n + (int64_t)hr * wt;
            i0 = po.cta_of(x0);
            no = po.cta_of(x0 + wt - 1) - i0 + 1;
            obase = b * hr_n + hr;
            orr = ro % kPfFewRows;
        }
    }
    const int total = np * per + no;
    // partial idx: its place (rows of D), or -1
    auto place = [&](int idx) -> int64_t {
        if (idx < np * per) {
            const int k = idx / per, st = idx - k * per;
            const int nt = min(p.run, p.tiles - k * p.run);
            if (st >= nt) return -1;
            return (int64_t)((k * a.Hkv + h) * d.Rgp + rg) * d.strideP + st * nr + rr;
        }
        const int i = i0 + (idx - np * per);
        const int nt = pf_tile_at(min(po.start(i + 1), x0 + wt) - x0) - pf_tile_at(max(po.start(i), x0) - x0);
        return nt > 0 ? (int64_t)(obase + i) * d.strideO + orr : -1;
    };
    const float2 *mlp = reinterpret_cast<const float2 *>(w.mlp), *mlo = reinterpret_cast<const float2 *>(w.mlo);
    float M = -INFINITY;
    for (int idx = wi + wpr * lane; idx < total; idx += 32 * wpr) {
        const int64_t at = place(idx);
        if (at >= 0) M = fmaxf(M, (idx < np * per ? mlp : mlo)[at].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    constexpr int V = D / 32;  // columns per lane
    float acc[V] = {}, L = 0.0f;
    if (M > -INFINITY) {
        for (int base = wi; base < total; base += 32 * wpr) {
            const int idx = base + wpr * lane;
            int64_t at = idx < total ? place(idx) : -1;
            float f = 0.0f;
            if (at >= 0) {
                const float2 ml = (idx < np * per ? mlp : mlo)[at];
                f = ml.x > -INFINITY ? ex2_approx(ml.x - M) : 0.0f;
                L = fmaf(ml.y, f, L);
            }
            const float *src = at < 0 || f == 0.0f ? nullptr : (idx < np * per ? w.Op : w.Oo) + at * D;
            const int cnt = min(32, (total - base + wpr - 1) / wpr);
#pragma unroll 8
            for (int k = 0; k < cnt; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                const float *O = reinterpret_cast<const float *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), k));
                if (!O) continue;
                if constexpr (V == 4) {
                    const float4 o = *reinterpret_cast<const float4 *>(O + lane * V);
                    acc[0] = fmaf(fk, o.x, acc[0]);
                    acc[1] = fmaf(fk, o.y, acc[1]);
                    acc[2] = fmaf(fk, o.z, acc[2]);
                    acc[3] = fmaf(fk, o.w, acc[3]);
                } else {
                    const float2 o = *reinterpret_cast<const float2 *>(O + lane * V);
                    acc[0] = fmaf(fk, o.x, acc[0]);
                    acc[1] = fmaf(fk, o.y, acc[1]);
                }
            }
        }
        L = warp_sum(L);
    }
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
    if (want >= rows) return;
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
    const int64_t rows = (int64_t)a.B * a.H * a.Tq;
    int wpr = kPfJoinWarps;
    while (wpr > 1 && rows * wpr > 16 * kPfCtas) wpr /= 2;  // about 16 warps per SM at most
    const int per_block = kPfJoinWarps / wpr;
    const unsigned grid = (unsigned)((rows + per_block - 1) / per_block);
    HSA_PROF("prefix_join", s);
    return a.D == 128 ? launch_pdl(prefix_join_kernel<128>, dim3(grid), dim3(kPfJoinThreads), 0, s, a, d, w, ctas, wpr)
                      : launch_pdl(prefix_join_kernel<64>, dim3(grid), dim3(kPfJoinThreads), 0, s, a, d, w, ctas, wpr);
}

}  // namespace hsa
