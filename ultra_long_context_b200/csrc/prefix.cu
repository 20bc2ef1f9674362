// prefix.cu -- softmax attention of a decode batch over a shared prefix and each request's own pages.
//
// One block per query row; a warp's lanes hold D / 8 dims of a key each, and every group of D / 8 lanes
// keeps its own running maximum, sum and output, joined in shared memory at the end.
#include "common.cuh"
#include "launch.h"
#include "profile.h"

namespace hsa {

constexpr int kPrefixThreads = 256;

template <int D>
__global__ void __launch_bounds__(kPrefixThreads) prefix_decode_kernel(PrefixArgs a) {
    constexpr int LPK = D / 8, GROUPS = kPrefixThreads / LPK;
    __shared__ float s_m[GROUPS], s_l[GROUPS], s_o[GROUPS][D];
    const int tid = threadIdx.x, g = tid / LPK, sub = tid % LPK;
    const int64_t row = blockIdx.x;
    if (row == 0 && tid == 0) *static_cast<int32_t *>(a.workspace) = 0;  // the call's status: no wait here can run out
    const int i = (int)(row % a.Tq), b = (int)(row / ((int64_t)a.H * a.Tq));
    const int hk = (int)(row / a.Tq % a.H) / (a.H / a.Hkv);
    const int64_t cap_p = (int64_t)a.max_prefix_pages * kChunk, cap_o = (int64_t)a.max_pages * kChunk;
    const int64_t P = cap_p > 0 ? max((int64_t)0, min(a.prefix_len[0], cap_p)) : 0;
    const int64_t n = min(a.own_len[b], cap_o);
    const int64_t last = n - a.Tq + i;
    const int64_t see_p = n < 0 ? 0 : max((int64_t)0, P + min((int64_t)0, last + 1));
    const int64_t see_o = n < 0 ? 0 : max((int64_t)0, last + 1);
    float q[8], o[8] = {0, 0, 0, 0, 0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    const uint4 qv = *reinterpret_cast<const uint4 *>(a.q + row * D + sub * 8);
    const uint32_t qw[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        q[2 * e] = bf16_lo(qw[e]) * a.scale;
        q[2 * e + 1] = bf16_hi(qw[e]) * a.scale;
    }
    const unsigned gmask = LPK == 16 ? 0xffffu << (16 * ((tid & 31) / 16)) : 0xffu << (8 * ((tid & 31) / 8));
    for (int64_t t = g; t < see_p + see_o; t += GROUPS) {
        const bool pre = t < see_p;
        const int64_t pos = pre ? t : t - see_p;
        const int page = pre ? a.prefix_table[pos / kChunk] : a.block_table[(int64_t)b * a.max_pages + pos / kChunk];
        if (page < 0 || page >= a.num_pages) continue;
        const int64_t at = (((int64_t)page * a.Hkv + hk) * kChunk + pos % kChunk) * D + sub * 8;
        float s = dot8(*reinterpret_cast<const uint4 *>(a.Kp + at), q);
#pragma unroll
        for (int w = LPK / 2; w > 0; w >>= 1) s += __shfl_xor_sync(gmask, s, w);
        const float mn = fmaxf(m, s), f = expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
        const uint4 vv = *reinterpret_cast<const uint4 *>(a.Vp + at);
        const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            o[2 * e] = fmaf(p, bf16_lo(vw[e]), o[2 * e] * f);
            o[2 * e + 1] = fmaf(p, bf16_hi(vw[e]), o[2 * e + 1] * f);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s_o[g][sub * 8 + e] = o[e];
    if (sub == 0) {
        s_m[g] = m;
        s_l[g] = l;
    }
    __syncthreads();
    for (int d = tid; d < D; d += kPrefixThreads) {
        float top = -INFINITY, z = 0.0f, x = 0.0f;
        for (int k = 0; k < GROUPS; ++k) top = fmaxf(top, s_m[k]);
        if (top > -INFINITY)
            for (int k = 0; k < GROUPS; ++k) {
                const float f = expf(s_m[k] - top);
                z = fmaf(s_l[k], f, z);
                x = fmaf(s_o[k][d], f, x);
            }
        a.out[row * D + d] = (uint16_t)(pack_bf16x2(z > 0.0f ? x / z : 0.0f, 0.0f) & 0xffffu);
        if (d == 0 && a.lse) a.lse[row] = z > 0.0f ? top + logf(z) : -INFINITY;
    }
}

size_t prefix_workspace(int B, int H, int Hkv, int Tq, int D, int max_prefix_pages, int max_pages) { return 256; }

cudaError_t launch_prefix_decode(const PrefixArgs &a, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.B * a.H * a.Tq);
    HSA_PROF("prefix_decode", s);
    if (a.D == 128) prefix_decode_kernel<128><<<grid, kPrefixThreads, 0, s>>>(a);
    else prefix_decode_kernel<64><<<grid, kPrefixThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace hsa
