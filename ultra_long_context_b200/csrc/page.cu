// page.cu -- the paged cache's bookkeeping (block tables and slot maps from request lengths) and the
// write of new key/value rows into their slots.
//
// Plan. With p(n) = ceil(n / 64), request b adding n tokens to its c needs p(c + n) - p(c) pages; the
// running sum of the needs gives its place in the ring of free pages, the running sum of the n its rows
// in the packed step. Position pos of a request is in a new page exactly when pos / 64 >= p(c), and the
// token with pos % 64 == 0 is then one of the new ones, so one pass over the packed tokens writes both
// the slots and the table entries: a token finds its request by binary search in the running sums.
// It is bound by latency: two dependent loads, one block scan of three sums (a second one only where the slot map is too
// short), a load and a store for each finished request that a team of warps has, one after the other, one search.
// One thread-block cluster of up to 8 blocks does all of it in one launch: every block scans all the lengths for itself (at
// most 96 KB out of L2), and the cluster barrier stands between the last read of `cache_len` and `pool` and the first write
// of what may be the same memory. A thread takes a run of up to 16 consecutive tokens, one search
// for all, four lookups in flight; finished requests are listed by the block that owns them (request % blocks) and
// copied by eight warps each. Blocks of 1024 threads before a second block, since a cluster's barrier costs more than
// four warps' work (1500 requests and as many tokens 14 us in clusters of small blocks, 9 in one of four of 1024). Measured: 64
// requests that add a token each, three finished, 5.0 us, 1500 requests 9.2 us, 256 with prompts of 87,000 tokens 14.4 us (0.75 MB;
// 0.12 us at the HBM's rate).
//
// Append. A copy: each 16-byte vector is read and written once, two steps in flight, bound by HBM: 32768 tokens x 8 heads x
// 128 (263 MB) 45.1 us = 5.84 TB/s; 3001 tokens 2.5 us and 64 tokens 2.0 us, bound by latency.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"
#include "profile.h"

namespace hsa {

int sm_count() {
    static std::atomic<int> counts[64];
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return sms;
    const bool known = dev >= 0 && dev < 64;
    if (known && (sms = counts[dev].load(std::memory_order_relaxed)) > 0) return sms;
    sms = 148;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && known)
        counts[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

__device__ __forceinline__ int ring_index(int64_t i, int n) {
    const int64_t r = i % n;
    return (int)(r < 0 ? r + n : r);
}

constexpr int kPlanMaxWarps = 32;
constexpr int kPlanMaxCtas = 8;   // a portable cluster
constexpr int kPlanTokens = 4;    // packed tokens a thread looks up at once, so that their loads overlap

// What a request asks for: packed rows, pages given back, new pages. (Page sums stay below B * max_pages < 2^31.)
struct PlanSum {
    int64_t rows;
    int back, need;
    __device__ void add(const PlanSum &o) {
        rows += o.rows;
        back += o.back;
        need += o.need;
    }
    __device__ PlanSum from_below(int o) const {
        return {__shfl_up_sync(0xffffffffu, rows, o), __shfl_up_sync(0xffffffffu, back, o), __shfl_up_sync(0xffffffffu, need, o)};
    }
    __device__ PlanSum of_lane(int l) const {
        return {__shfl_sync(0xffffffffu, rows, l), __shfl_sync(0xffffffffu, back, l), __shfl_sync(0xffffffffu, need, l)};
    }
};

__device__ __forceinline__ PlanSum plan_warp_scan(PlanSum x) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const PlanSum y = x.from_below(o);
        if (lane >= o) x.add(y);
    }
    return x;
}

// Exclusive block scan (warp shuffles, then the warps' sums). s_warp is free again after the next barrier.
__device__ __forceinline__ PlanSum plan_scan(const PlanSum &v, PlanSum *s_warp, PlanSum *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const PlanSum x = plan_warp_scan(v);
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    const PlanSum w = plan_warp_scan(lane < warps ? s_warp[lane] : PlanSum{0, 0, 0});  // every warp sums all warps
    *total = w.of_lane(31);
    const PlanSum b = w.of_lane(warp > 0 ? warp - 1 : 0);
    return {x.rows - v.rows + (warp > 0 ? b.rows : 0), x.back - v.back + (warp > 0 ? b.back : 0),
            x.need - v.need + (warp > 0 ? b.need : 0)};
}

// Pages of 64 for n >= 0.
__device__ __forceinline__ int plan_pages(int64_t n) { return (int)((uint64_t)(n + kChunk - 1) / kChunk); }

__global__ void __launch_bounds__(32 * kPlanMaxWarps) page_plan_kernel(PagePlanArgs a, int run) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    int64_t *s_len = reinterpret_cast<int64_t *>(smem_raw);            // [B] cache_len
    int32_t *s_new = reinterpret_cast<int32_t *>(s_len + a.B);         // [B] new_len; 0 once refused
    int32_t *s_cu = s_new + a.B;                                       // [B + 1] packed rows
    int32_t *s_at = s_cu + a.B + 1;                                    // [B] first page's place in the ring's order
    int32_t *s_gone = s_at + a.B;                                      // [B] finished requests
    __shared__ PlanSum s_warp[2][kPlanMaxWarps];
    __shared__ int s_refused, s_got, s_ngone;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, block = blockDim.x;
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks(), nthr = ctas * block;
    const int64_t cap = (int64_t)a.max_pages * kChunk;
    const int64_t taken = a.pool[0], returned = a.pool[1];
    for (int b = tid; b < a.B; b += block) {
        s_len[b] = a.cache_len[b];
        s_new[b] = a.new_len[b];
    }
    if (tid == 0) s_refused = s_got = s_ngone = 0;
    __syncthreads();
    const int per = (a.B + block - 1) / block;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    PlanSum sum{0, 0, 0}, total;
    // rows_before: packed rows of the requests before it
    auto asks = [&](int b, int64_t rows_before) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        PlanSum q{max(n, 0), 0, 0};
        if (c >= 0 && c <= cap) {
            if (n < 0) q.back = plan_pages(c);
            if (n > 0 && c + n <= cap && rows_before + n <= a.max_tokens) q.need = plan_pages(c + n) - plan_pages(c);
        }
        return q;
    };
    for (int b = lo; b < hi; ++b) sum.add(asks(b, 0));
    PlanSum before = plan_scan(sum, s_warp[0], &total);
    if (total.rows > a.max_tokens) {  // some have no room in the slot map and get no pages: sum the needs again
        PlanSum again{0, 0, 0}, total2;
        int64_t r = before.rows;
        for (int b = lo; b < hi; ++b) {
            again.need += asks(b, r).need;
            r += max(s_new[b], 0);
        }
        before.need = plan_scan(again, s_warp[1], &total2).need;
    }
    const int64_t avail = min(max(returned - taken, (int64_t)0), (int64_t)a.num_free);
    int got = 0, refused = 0;
    for (int b = lo; b < hi; ++b) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        const PlanSum q = asks(b, before.rows);
        s_cu[b] = (int)min(before.rows, (int64_t)INT32_MAX);
        s_at[b] = n < 0 ? before.back : before.need;
        before.add(q);
        bool ok = c >= 0 && c <= cap;
        if (n < 0 && ok && b % ctas == rank) s_gone[atomicAdd(&s_ngone, 1)] = b;  // this block's share, in any order
        if (n > 0) {
            ok = ok && c + n <= cap && before.rows <= a.max_tokens && (q.need == 0 || before.need <= avail);
            if (ok && q.need > 0) got = before.need;  // those that get pages are the first that ask for any
        }
        if (!ok) {
            ++refused;
            s_new[b] = 0;
        }
    }
    if (tid == 0) s_cu[a.B] = (int)min(total.rows, (int64_t)INT32_MAX);
    got = __reduce_max_sync(0xffffffffu, got);
    refused = __reduce_add_sync(0xffffffffu, refused);
    if (lane == 0 && got) atomicMax(&s_got, got);
    if (lane == 0 && refused) atomicAdd(&s_refused, refused);
    // every block has read cache_len and pool, which the outputs may overwrite
    if (ctas > 1) cluster.sync();
    else __syncthreads();

    const int gtid = rank * block + tid;
    if (gtid == 0) {
        a.pool_out[0] = taken + s_got;
        a.pool_out[1] = returned + total.back;
        a.pool_out[2] = s_refused;
    }
    for (int b = gtid; b <= a.B; b += nthr) {
        a.cu_new[b] = s_cu[b];
        if (b < a.B) a.total_len[b] = s_new[b] < 0 ? 0 : s_len[b] + s_new[b];
    }
    const int ring0 = ring_index(taken, a.num_free), ring1 = ring_index(returned, a.num_free);
    // finished requests' pages: eight warps (or all there are) to a request
    const int team = min(block, 256);
    for (int i = tid / team; i < s_ngone; i += block / team) {
        const int b = s_gone[i], held = plan_pages(s_len[b]);
        const int32_t *row = a.block_table + (int64_t)b * a.max_pages;
        const int64_t first = ring_index((int64_t)ring1 + s_at[b], a.num_free);
        for (int j = tid % team; j < held; j += team) {
            // more pages than the ring holds cannot come back; if they do all the same, it goes round
            const int64_t k = first + j;
            a.free_pages[k < a.num_free ? k : k % a.num_free] = row[j];
        }
    }
    // packed tokens: `run` consecutive ones to a thread, kPlanTokens at a time
    const int live = (int)min(total.rows, (int64_t)a.max_tokens);
    const int top = a.B > 1 ? 1 << (31 - __clz(a.B - 1)) : 0;
    for (int64_t t0 = (int64_t)gtid * run; t0 < a.max_tokens; t0 += (int64_t)nthr * run) {
        // the last request whose rows begin at or before the token: requests without rows begin where the next does
        int b = 0;
        for (int step = top; step > 0; step >>= 1)
            if (b + step < a.B && s_cu[b + step] <= t0) b += step;
        const int64_t t_end = min(t0 + run, (int64_t)a.max_tokens);
        for (int64_t t1 = t0; t1 < t_end; t1 += kPlanTokens) {
            int id[kPlanTokens], off[kPlanTokens];
            int32_t *entry[kPlanTokens];
#pragma unroll
            for (int u = 0; u < kPlanTokens; ++u) {
                const int64_t t = t1 + u;
                id[u] = -1;
                off[u] = 0;
                entry[u] = nullptr;
                if (t >= t_end || t >= live) continue;
                while (b + 1 < a.B && s_cu[b + 1] <= t) ++b;
                if (s_new[b] <= 0) continue;
                const int64_t c = s_len[b], pos = c + (t - s_cu[b]), pg = pos / kChunk;
                const int held = plan_pages(c);
                int32_t *slot = a.block_table + (int64_t)b * a.max_pages + pg;
                off[u] = (int)(pos % kChunk);
                if (pg < held) {
                    id[u] = *slot;
                } else {
                    const int64_t k = (int64_t)ring0 + s_at[b] + (pg - held);
                    id[u] = a.free_pages[k >= a.num_free ? k - a.num_free : k];
                    if (off[u] == 0) entry[u] = slot;
                }
            }
#pragma unroll
            for (int u = 0; u < kPlanTokens; ++u) {
                if (t1 + u >= t_end) continue;
                a.slots[t1 + u] = id[u] < 0 ? -1 : (int64_t)id[u] * kChunk + off[u];
                if (entry[u]) *entry[u] = id[u];
            }
        }
    }
}

size_t page_plan_smem(int B) { return (size_t)B * (sizeof(int64_t) + 4 * sizeof(int32_t)) + sizeof(int32_t); }

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
    const size_t smem = page_plan_smem(a.B);
    cudaError_t e = allow_smem<page_plan_kernel>(page_plan_smem(kPagedMaxBatch));
    if (e != cudaSuccess) return e;
    // a thread to each token and request up to one block of 1024, then more blocks
    const int64_t work = (int64_t)a.max_tokens + a.B;
    int threads = 128, ctas = 1;
    while (threads < 1024 && threads < work) threads *= 2;
    while (ctas < kPlanMaxCtas && (int64_t)ctas * threads < work) ctas *= 2;
    // tokens to a thread: one while there are threads enough, then as many as there are to each, up to 16
    const int64_t each = (a.max_tokens + (int64_t)ctas * threads - 1) / ((int64_t)ctas * threads);
    const int run = (int)(each < 1 ? 1 : each > 16 ? 16 : each);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)ctas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    HSA_PROF("page_plan", s);
    return cudaLaunchKernelEx(&cfg, page_plan_kernel, a, run);
}

constexpr int kAppendThreads = 256;

// One 16-byte vector of K and of V per thread and step; vpt vectors per token (Hkv * D / 8), vpr per head. Index: 32 bits
// where they suffice, for the divisions.
template <typename Index>
__global__ void __launch_bounds__(kAppendThreads) page_append_kernel(
    const uint16_t *__restrict__ K, int64_t k_stride, const uint16_t *__restrict__ V, int64_t v_stride,
    const int64_t *__restrict__ slots, Index vecs, Index vpt, int vpr_log2, uint16_t *__restrict__ Kp,
    uint16_t *__restrict__ Vp, int64_t num_slots) {
    constexpr int U = 2;  // steps whose loads are in flight together
    const Index step = (Index)gridDim.x * kAppendThreads;
    for (Index i0 = (Index)blockIdx.x * kAppendThreads + threadIdx.x; i0 < vecs; i0 += U * step) {
        uint4 kv[U], vv[U];
        int64_t dst[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Index i = i0 + u * step;
            dst[u] = -1;
            if (i >= vecs) continue;
            const Index tok = i / vpt;
            const int v = (int)(i - tok * vpt), head = v >> vpr_log2, x = v - (head << vpr_log2);
            const int64_t slot = slots[tok];
            if (slot < 0 || slot >= num_slots) continue;
            kv[u] = ld_stream16(K + (int64_t)tok * k_stride + (int64_t)v * 8);
            vv[u] = ld_stream16(V + (int64_t)tok * v_stride + (int64_t)v * 8);
            // page slot / 64 holds vpt * 64 vectors, head-major
            dst[u] = (slot / kChunk) * (int64_t)vpt * kChunk + (((int64_t)head * kChunk + slot % kChunk) << vpr_log2) + x;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (dst[u] < 0) continue;
            reinterpret_cast<uint4 *>(Kp)[dst[u]] = kv[u];
            reinterpret_cast<uint4 *>(Vp)[dst[u]] = vv[u];
        }
    }
}

cudaError_t launch_page_append(const uint16_t *K, int64_t k_stride, const uint16_t *V, int64_t v_stride,
                               const int64_t *slots, int n, int Hkv, int D, uint16_t *Kp, uint16_t *Vp, int num_pages,
                               cudaStream_t s) {
    if (n <= 0) return cudaSuccess;
    const int vpr_log2 = D == 128 ? 4 : 3, vpt = Hkv << vpr_log2;
    const int64_t vecs = (int64_t)n * vpt, slots_n = (int64_t)num_pages * kChunk;
    const int64_t want = (vecs + kAppendThreads - 1) / kAppendThreads, most = (int64_t)sm_count() * 16;
    const unsigned grid = (unsigned)(want < most ? want : most);
    HSA_PROF("page_append", s);
    if (vecs < (1u << 30))
        page_append_kernel<uint32_t><<<grid, kAppendThreads, 0, s>>>(K, k_stride, V, v_stride, slots, (uint32_t)vecs,
                                                                     (uint32_t)vpt, vpr_log2, Kp, Vp, slots_n);
    else
        page_append_kernel<int64_t><<<grid, kAppendThreads, 0, s>>>(K, k_stride, V, v_stride, slots, vecs, vpt, vpr_log2,
                                                                    Kp, Vp, slots_n);
    return cudaGetLastError();
}

}  // namespace hsa
