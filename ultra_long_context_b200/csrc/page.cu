// page.cu -- the paged cache's bookkeeping (block tables and slot maps from request lengths) and the
// write of new key/value rows into their slots.
//
// Plan. With p(n) = ceil(n / 64), request b adding n tokens to its c needs p(c + n) - p(c) pages; the
// running sum of the needs gives its place in the ring of free pages, the running sum of the n its rows
// in the packed step. Position pos of a request is in a new page exactly when pos / 64 >= p(c), and the
// token with pos % 64 == 0 is then one of the new ones, so one pass over the packed tokens writes both
// the slots and the table entries: a token finds its request by binary search in the running sums.
// It is bound by latency: two dependent loads, two block scans, one search per token. One thread-block
// cluster does all of it in one launch: every block scans all the lengths for itself (at most 96 KB out
// of L2), and the cluster barrier stands between the last read of `cache_len` and `pool` and the first
// write of what may be the same memory.
//
// Append. A copy: each 16-byte vector is read and written once, bound by HBM (small calls by latency).
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

// Exclusive block scan of one value per thread (warp shuffles, then the warps' sums).
template <typename T>
__device__ __forceinline__ T plan_scan(T v, T *s_warp, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    T w = lane < warps ? s_warp[lane] : 0;  // every warp sums the warps before it
    const T mine = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    return __shfl_sync(0xffffffffu, w - mine, warp) + x - v;
}

// Pages of 64 for n >= 0.
__device__ __forceinline__ int plan_pages(int64_t n) { return (int)((uint64_t)(n + kChunk - 1) / kChunk); }

__global__ void __launch_bounds__(32 * kPlanMaxWarps) page_plan_kernel(PagePlanArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    int64_t *s_len = reinterpret_cast<int64_t *>(smem_raw);            // [B] cache_len
    int32_t *s_new = reinterpret_cast<int32_t *>(s_len + a.B);         // [B] new_len; 0 once refused
    int32_t *s_cu = s_new + a.B;                                       // [B + 1] packed rows
    int32_t *s_at = s_cu + a.B + 1;                                    // [B] first page's place in the ring's order
    int32_t *s_gone = s_at + a.B;                                      // [B] finished requests
    __shared__ int64_t s_rows[kPlanMaxWarps];
    __shared__ int s_back[kPlanMaxWarps], s_need[kPlanMaxWarps], s_refused, s_got, s_ngone;
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
    // packed rows, and the pages that finished requests give back (page sums stay below B * max_pages < 2^31)
    int64_t rows = 0, total_rows;
    int back = 0, total_back;
    for (int b = lo; b < hi; ++b) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        rows += max(n, 0);
        back += n < 0 && c >= 0 && c <= cap ? plan_pages(c) : 0;
    }
    rows = plan_scan(rows, s_rows, &total_rows);
    back = plan_scan(back, s_back, &total_back);
    int need = 0, total_need;
    int64_t r = rows;
    for (int b = lo; b < hi; ++b) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        s_cu[b] = (int)min(r, (int64_t)INT32_MAX);
        r += max(n, 0);
        if (n < 0 && c >= 0 && c <= cap) {
            s_at[b] = back;
            back += plan_pages(c);
            // this block's share of them, in any order: each has its own places in the ring
            if (b % ctas == rank) s_gone[atomicAdd(&s_ngone, 1)] = b;
        } else if (n > 0 && c >= 0 && c <= cap && c + n <= cap && r <= a.max_tokens) {
            need += plan_pages(c + n) - plan_pages(c);
        }
    }
    if (tid == 0) s_cu[a.B] = (int)min(total_rows, (int64_t)INT32_MAX);
    need = plan_scan(need, s_need, &total_need);
    const int64_t avail = min(max(returned - taken, (int64_t)0), (int64_t)a.num_free);
    int got = 0, refused = 0;
    r = rows;
    for (int b = lo; b < hi; ++b) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        const bool known = c >= 0 && c <= cap;
        r += max(n, 0);
        if (n <= 0) {
            refused += !known;
            if (!known) s_new[b] = 0;
            continue;
        }
        bool ok = known && c + n <= cap && r <= a.max_tokens;
        if (ok) {
            const int k = plan_pages(c + n) - plan_pages(c);
            s_at[b] = need;
            need += k;
            ok = k == 0 || need <= avail;
            if (ok && k > 0) got = need;  // those that get pages are the first that ask for any
        }
        refused += !ok;
        if (!ok) s_new[b] = 0;
    }
    got = __reduce_max_sync(0xffffffffu, got);
    refused = __reduce_add_sync(0xffffffffu, refused);
    if (lane == 0 && got) atomicMax(&s_got, got);
    if (lane == 0 && refused) atomicAdd(&s_refused, refused);
    cluster.sync();  // every block has read cache_len and pool, which the outputs may overwrite

    const int gtid = rank * block + tid;
    if (gtid == 0) {
        a.pool_out[0] = taken + s_got;
        a.pool_out[1] = returned + total_back;
        a.pool_out[2] = s_refused;
    }
    for (int b = gtid; b <= a.B; b += nthr) {
        a.cu_new[b] = s_cu[b];
        if (b < a.B) a.total_len[b] = s_new[b] < 0 ? 0 : s_len[b] + s_new[b];
    }
    const int ring0 = ring_index(taken, a.num_free), ring1 = ring_index(returned, a.num_free);
    const int live = (int)min(total_rows, (int64_t)a.max_tokens);
    const int top = a.B > 1 ? 1 << (31 - __clz(a.B - 1)) : 0;
    for (int64_t t0 = gtid; t0 < a.max_tokens; t0 += (int64_t)kPlanTokens * nthr) {
        int req[kPlanTokens], id[kPlanTokens];
        int64_t pos[kPlanTokens];
        int32_t *entry[kPlanTokens];
        // the last request whose rows begin at or before the token: requests without rows begin where the next does
#pragma unroll
        for (int u = 0; u < kPlanTokens; ++u) req[u] = 0;
        for (int step = top; step > 0; step >>= 1) {
#pragma unroll
            for (int u = 0; u < kPlanTokens; ++u) {
                const int m = req[u] + step;
                if (m < a.B && s_cu[m] <= t0 + (int64_t)u * nthr) req[u] = m;
            }
        }
#pragma unroll
        for (int u = 0; u < kPlanTokens; ++u) {
            const int64_t t = t0 + (int64_t)u * nthr;
            const int b = req[u];
            id[u] = -1;
            entry[u] = nullptr;
            if (t >= live || s_new[b] <= 0) continue;
            const int64_t c = s_len[b];
            pos[u] = c + (t - s_cu[b]);
            const int64_t pg = pos[u] / kChunk;
            const int held = plan_pages(c);
            int32_t *slot = a.block_table + (int64_t)b * a.max_pages + pg;
            if (pg < held) {
                id[u] = *slot;
            } else {
                const int64_t k = (int64_t)ring0 + s_at[b] + (pg - held);
                id[u] = a.free_pages[k >= a.num_free ? k - a.num_free : k];
                if (pos[u] % kChunk == 0) entry[u] = slot;
            }
            pos[u] %= kChunk;
        }
#pragma unroll
        for (int u = 0; u < kPlanTokens; ++u) {
            const int64_t t = t0 + (int64_t)u * nthr;
            if (t >= a.max_tokens) continue;
            const bool placed = t < live && s_new[req[u]] > 0;
            a.slots[t] = placed ? (int64_t)id[u] * kChunk + pos[u] : -1;
            if (entry[u]) *entry[u] = id[u];
        }
    }
    // finished requests' pages, a warp to a request
    for (int i = tid >> 5; i < s_ngone; i += block >> 5) {
        const int b = s_gone[i], held = plan_pages(s_len[b]);
        const int32_t *row = a.block_table + (int64_t)b * a.max_pages;
        const int first = ring_index((int64_t)ring1 + s_at[b], a.num_free);
#pragma unroll 4
        for (int j = lane; j < held; j += 32) {
            // more pages than the ring holds cannot come back; if they do all the same, it goes round
            const int64_t k = (int64_t)first + j;
            a.free_pages[k < a.num_free ? k : k % a.num_free] = row[j];
        }
    }
}

size_t page_plan_smem(int B) { return (size_t)B * (sizeof(int64_t) + 4 * sizeof(int32_t)) + sizeof(int32_t); }

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
    const size_t smem = page_plan_smem(a.B);
    cudaError_t e = allow_smem<page_plan_kernel>(smem);
    if (e != cudaSuccess) return e;
    // a thread to each token and request up to one block of 1024, then more blocks
    const int64_t work = (int64_t)a.max_tokens + a.B;
    int threads = 128, ctas = 1;
    while (threads < 1024 && threads < work) threads *= 2;
    while (ctas < kPlanMaxCtas && (int64_t)ctas * threads < work) ctas *= 2;
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
    return cudaLaunchKernelEx(&cfg, page_plan_kernel, a);
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
