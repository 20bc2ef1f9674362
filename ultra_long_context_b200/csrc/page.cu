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

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMaxCtas = 8;  // a portable cluster

// Exclusive block scan of one value per thread (warp shuffles, then the warps' sums); *total: the block's sum.
__device__ __forceinline__ int64_t plan_scan(int64_t v, int64_t *s_warp, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int64_t w = lane < kPlanWarps ? s_warp[lane] : 0;
        int64_t z = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += y;
        }
        if (lane < kPlanWarps) s_warp[lane] = z - w;
        if (lane == 31) s_warp[kPlanWarps] = z;
    }
    __syncthreads();
    const int64_t res = s_warp[warp] + x - v;
    *total = s_warp[kPlanWarps];
    __syncthreads();  // s_warp is used again
    return res;
}

__device__ __forceinline__ int ring_index(int64_t i, int n) {
    const int64_t r = i % n;
    return (int)(r < 0 ? r + n : r);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(PagePlanArgs a) {
    namespace cg = cooperative_groups;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    int64_t *s_len = reinterpret_cast<int64_t *>(smem_raw);            // [B] cache_len
    int32_t *s_new = reinterpret_cast<int32_t *>(s_len + a.B);         // [B] new_len; 0 once refused
    int32_t *s_cu = s_new + a.B;                                       // [B + 1] packed rows
    int32_t *s_at = s_cu + a.B + 1;                                    // [B] first page's place in the ring's order
    __shared__ int64_t s_warp[kPlanWarps + 1];
    __shared__ int s_refused;
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank(), nthr = (int)cluster.num_blocks() * kPlanThreads;
    const int64_t cap = (int64_t)a.max_pages * kChunk;
    const int64_t taken = a.pool[0], returned = a.pool[1];
    for (int b = tid; b < a.B; b += kPlanThreads) {
        s_len[b] = a.cache_len[b];
        s_new[b] = a.new_len[b];
    }
    if (tid == 0) s_refused = 0;
    __syncthreads();
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int lo = min(a.B, tid * per), hi = min(a.B, lo + per);
    // packed rows, and the pages that finished requests give back
    int64_t rows = 0, back = 0, total_rows, total_back;
    for (int b = lo; b < hi; ++b) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        rows += max(n, 0);
        back += n < 0 && c >= 0 && c <= cap ? (c + kChunk - 1) / kChunk : 0;
    }
    rows = plan_scan(rows, s_warp, &total_rows);
    back = plan_scan(back, s_warp, &total_back);
    int64_t need = 0, total_need;
    int64_t r = rows;
    for (int b = lo; b < hi; ++b) {
        const int n = s_new[b];
        const int64_t c = s_len[b];
        s_cu[b] = (int)min(r, (int64_t)INT32_MAX);
        r += max(n, 0);
        if (n < 0 && c >= 0 && c <= cap) {
            s_at[b] = (int)back;
            back += (c + kChunk - 1) / kChunk;
        } else if (n > 0 && c >= 0 && c <= cap && c + n <= cap && r <= a.max_tokens) {
            need += (c + n + kChunk - 1) / kChunk - (c + kChunk - 1) / kChunk;
        }
    }
    if (tid == 0) s_cu[a.B] = (int)min(total_rows, (int64_t)INT32_MAX);
    need = plan_scan(need, s_warp, &total_need);
    const int64_t avail = min(max(returned - taken, (int64_t)0), (int64_t)a.num_free);
    int64_t got = 0;
    int refused = 0;
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
            const int64_t k = (c + n + kChunk - 1) / kChunk - (c + kChunk - 1) / kChunk;
            s_at[b] = (int)min(need, (int64_t)INT32_MAX);
            need += k;
            ok = k == 0 || need <= avail;
            got += ok ? k : 0;
        }
        refused += !ok;
        if (!ok) s_new[b] = 0;
    }
    // what this block's requests took (every block finds the same; block 0 writes it)
    int64_t total_got;
    plan_scan(got, s_warp, &total_got);
    if (refused) atomicAdd(&s_refused, refused);
    __syncthreads();
    cluster.sync();  // every block has read cache_len and pool, which the outputs may overwrite

    const int gtid = rank * kPlanThreads + tid;
    if (gtid == 0) {
        a.pool_out[0] = taken + total_got;
        a.pool_out[1] = returned + total_back;
        a.pool_out[2] = s_refused;
    }
    for (int b = gtid; b <= a.B; b += nthr) {
        a.cu_new[b] = s_cu[b];
        if (b < a.B) a.total_len[b] = s_new[b] < 0 ? 0 : s_len[b] + s_new[b];
    }
    const int ring0 = ring_index(taken, a.num_free);
    const int live = (int)min(total_rows, (int64_t)a.max_tokens);
    for (int t = gtid; t < a.max_tokens; t += nthr) {
        int64_t slot = -1;
        if (t < live) {
            int l = 0, h = a.B;  // the last request whose rows begin at or before t and that has any
            while (h - l > 1) {
                const int m = (l + h) >> 1;
                if (s_cu[m] <= t) l = m;
                else h = m;
            }
            const int n = s_new[l];
            if (n > 0) {
                const int64_t c = s_len[l], pos = c + (t - s_cu[l]);
                const int64_t pg = pos / kChunk, held = (c + kChunk - 1) / kChunk;
                int32_t *entry = a.block_table + (int64_t)l * a.max_pages + pg;
                int32_t id;
                if (pg < held) {
                    id = *entry;
                } else {
                    int64_t k = (int64_t)ring0 + s_at[l] + (pg - held);
                    id = a.free_pages[k >= a.num_free ? k - a.num_free : k];
                    if (pos % kChunk == 0) *entry = id;
                }
                slot = (int64_t)id * kChunk + pos % kChunk;
            }
        }
        a.slots[t] = slot;
    }
    // finished requests' pages, a warp to a request
    for (int b = gtid >> 5; b < a.B; b += nthr >> 5) {
        if (s_new[b] >= 0) continue;
        const int held = (int)((s_len[b] + kChunk - 1) / kChunk);
        for (int j = tid & 31; j < held; j += 32)
            a.free_pages[ring_index(returned + s_at[b] + j, a.num_free)] = a.block_table[(int64_t)b * a.max_pages + j];
    }
}

size_t page_plan_smem(int B) { return (size_t)B * (sizeof(int64_t) + 3 * sizeof(int32_t)) + sizeof(int32_t); }

cudaError_t launch_page_plan(const PagePlanArgs &a, cudaStream_t s) {
    const size_t smem = page_plan_smem(a.B);
    cudaError_t e = allow_smem<page_plan_kernel>(smem);
    if (e != cudaSuccess) return e;
    int ctas = 1;
    while (ctas < kPlanMaxCtas && (int64_t)ctas * 4 * kPlanThreads < (int64_t)a.max_tokens + a.B) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
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

// One 16-byte vector of K and of V per thread and step; VPT vectors per token (Hkv * D / 8).
__global__ void __launch_bounds__(kAppendThreads) page_append_kernel(
    const uint16_t *__restrict__ K, int64_t k_stride, const uint16_t *__restrict__ V, int64_t v_stride,
    const int64_t *__restrict__ slots, int64_t vecs, int vpt, int vpr, uint16_t *__restrict__ Kp,
    uint16_t *__restrict__ Vp, int64_t num_slots) {
    const int64_t step = (int64_t)gridDim.x * kAppendThreads;
    for (int64_t i = (int64_t)blockIdx.x * kAppendThreads + threadIdx.x; i < vecs; i += step) {
        const int64_t tok = i / vpt;
        const int v = (int)(i - tok * vpt), head = v / vpr, x = v - head * vpr;
        const int64_t slot = slots[tok];
        if (slot < 0 || slot >= num_slots) continue;
        const uint4 kv = ld_stream16(K + tok * k_stride + (int64_t)v * 8);
        const uint4 vv = ld_stream16(V + tok * v_stride + (int64_t)v * 8);
        // page slot / 64 holds vpt * 64 vectors, head-major
        const int64_t dst = (slot / kChunk) * vpt * kChunk + ((int64_t)head * kChunk + slot % kChunk) * vpr + x;
        reinterpret_cast<uint4 *>(Kp)[dst] = kv;
        reinterpret_cast<uint4 *>(Vp)[dst] = vv;
    }
}

cudaError_t launch_page_append(const uint16_t *K, int64_t k_stride, const uint16_t *V, int64_t v_stride,
                               const int64_t *slots, int n, int Hkv, int D, uint16_t *Kp, uint16_t *Vp, int num_pages,
                               cudaStream_t s) {
    if (n <= 0) return cudaSuccess;
    const int vpr = D / 8, vpt = Hkv * vpr;
    const int64_t vecs = (int64_t)n * vpt;
    const int sms = sm_count();
    const int64_t want = (vecs + kAppendThreads - 1) / kAppendThreads;
    const unsigned grid = (unsigned)(want < (int64_t)sms * 8 ? want : (int64_t)sms * 8);
    HSA_PROF("page_append", s);
    page_append_kernel<<<grid, kAppendThreads, 0, s>>>(K, k_stride, V, v_stride, slots, vecs, vpt, vpr, Kp, Vp,
                                                       (int64_t)num_pages * kChunk);
    return cudaGetLastError();
}

}  // namespace hsa
