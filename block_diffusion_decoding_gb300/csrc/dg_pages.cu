// dg_pages.cu -- a pool of cache pages on the device: pages handed out to sequences
// that grow, shared and copied by sequences that fork, and taken back.
//
// free_pages [0, n_free) are the pages of nobody, a stack: handed out from its end.
// refs counts the sequences that hold a page; a sequence holds the pages of the first
// places of its row of the table, the places behind them are negative.  Which page goes
// where depends on the arguments alone: the decisions are made by one CTA in the order of
// the sequences, by prefix sums of what each one needs, and only counts that no order
// changes are added by atomics.  All of it but the copies is bound by latency: a few reads
// that depend on one another, 2 to 4 us, beside which the host's 5 for a launch counts.
#include "dg_serve_kernels.h"

namespace dg {

namespace {

// Inclusive sums over the kPoolThreads threads, none above `most` (at which the
// values are cut too: 2 most fits 32 bits); *total: of all of them.
DG_DEVICE int block_scan(int v, int most, int *warp_sums, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = min(v, most);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v = min(v + x, most);
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w = min(w + x, most);
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[31];
    return warp > 0 ? min(v + warp_sums[warp - 1], most) : v;
}

DG_DEVICE int count_free(const PagePoolArgs &a)
{
    const int n = *a.n_free, cut = min(max(n, 0), a.n_pages);
    if (cut != n && threadIdx.x == 0) report_error(a.ws, DG_ERR_DEVICE, 1121);
    return cut;
}

DG_DEVICE int cached(const PagePoolArgs &a, int b)
{
    const int kv = a.kv_len[b], cut = min(max(kv, 0), a.max_pages * a.page_size);
    if (cut != kv) report_error(a.ws, DG_ERR_DEVICE, 1122);
    return cut;
}

constexpr int32_t kPageFreed = -(1 << 30);   // refs of a page that a release has just taken back

}  // namespace

// Pages for the tokens that the next append brings, a sequence a thread; then a thread a
// page handed out, which looks its sequence up among the sums.
__global__ void __launch_bounds__(kPoolThreads) paged_reserve_kernel(PagePoolArgs a)
{
    __shared__ int sums[32];
    __shared__ int s_end[kPoolThreads], s_have[kPoolThreads];   // places up to and with a sequence's
    __shared__ int s_given;
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int n_free = count_free(a);
    int given = 0;                               // pages that have been handed out
    bool run_short = false;
    for (int b0 = 0; b0 < a.B; b0 += kPoolThreads) {
        const int b = b0 + tid;
        int need = 0, have = 0;
        if (b < a.B) {
            const int kv = cached(a, b);
            const int64_t n = static_cast<int64_t>(a.q_start[b + 1]) - a.q_start[b];
            if (n < 0) report_error(a.ws, DG_ERR_DEVICE, 1123);
            const int64_t want = (kv + (n > 0 ? n : 0) + a.page_size - 1) / a.page_size;
            if (want > a.max_pages) report_error(a.ws, DG_ERR_DEVICE, 1124);
            const int upto = static_cast<int>(want < a.max_pages ? want : a.max_pages);
            // (pages of an earlier call whose tokens were not kept are still there)
            const int32_t *row = a.page_table + static_cast<int64_t>(b) * a.max_pages;
            int end = upto;
            have = min(kv / a.page_size, upto);
            while (have < end) {
                const int mid = (have + end) >> 1;
                if (row[mid] >= 0) have = mid + 1;
                else end = mid;
            }
            need = upto - have;
        }
        const int left = run_short ? 0 : n_free - given;
        int total;
        const int end = block_scan(need, left + 1, sums, &total);
        if (need > 0 && end > left) report_error(a.ws, DG_ERR_DEVICE, 1125);
        s_end[tid] = end;
        s_have[tid] = have;
        if (tid == 0) s_given = 0;
        __syncthreads();
        if (need > 0 && end <= left) atomicMax(&s_given, end);
        __syncthreads();
        const int now = s_given;
        for (int x = tid; x < now; x += kPoolThreads) {
            int lo = 0, hi = kPoolThreads - 1;   // the first sequence whose places end past x
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_end[mid] > x) hi = mid;
                else lo = mid + 1;
            }
            const int page = a.free_pages[n_free - 1 - given - x];
            if (page < 0 || page >= a.n_pages) {
                report_error(a.ws, DG_ERR_DEVICE, 1126);
                continue;
            }
            a.page_table[static_cast<int64_t>(b0 + lo) * a.max_pages + s_have[lo] + x -
                         (lo > 0 ? s_end[lo - 1] : 0)] = page;
            a.refs[page] = 1;
        }
        given += now;
        run_short |= total > left;
        __syncthreads();
    }
    if (tid == 0) *a.n_free = n_free - given;
}

// Which forks are made, and the page of each one's copy.
__global__ void __launch_bounds__(kPoolThreads) paged_fork_kernel(PagePoolArgs a)
{
    __shared__ int sums[32];
    __shared__ int s_dst[kPoolThreads];
    griddep_wait();
    griddep_launch_dependents();
    const int i = threadIdx.x;
    const int n_free = count_free(a);
    PageForkJob job{-1, -1, 0, -1};
    bool made = false;
    s_dst[i] = i < a.n ? a.dst[i] : -1;
    __syncthreads();
    if (i < a.n) {
        const int src = a.src[i], dst = s_dst[i];
        made = src >= 0 && src < a.B && dst >= 0 && dst < a.B && src != dst;
        for (int j = 0; j < i && made; ++j) made = s_dst[j] != dst;
        if (made) {
            made = a.kv_len[dst] == 0 && a.page_table[static_cast<int64_t>(dst) * a.max_pages] < 0;
            job = PageForkJob{src, dst, cached(a, src), -1};
        }
    }
    const bool copies = made && job.kv % a.page_size != 0;
    int total;
    const int end = block_scan(copies ? 1 : 0, kPoolThreads, sums, &total);    // (all lengths have been read)
    if (copies) {
        if (end <= n_free) job.page = a.free_pages[n_free - end];
        made = end <= n_free && job.page >= 0 && job.page < a.n_pages;
    }
    if (i < a.n) {
        if (made) {
            a.kv_len[job.dst] = job.kv;
            if (copies) a.refs[job.page] = 1;
        } else {
            report_error(a.ws, DG_ERR_DEVICE, 1127);
            job.dst = -1;
        }
        a.jobs[i] = job;
    }
    if (i == 0) *a.n_free = n_free - min(total, n_free);
}

// The forks' tables, the counts of the pages they share, and the copies of their
// last, unfinished pages in every layer: a block a fork's table, or kForkBytes of a
// page, 128 bytes of it on their way in each thread.  Bound by memory: 128 forks of 8
// prompts, 16 layers of 8 heads of 128, 0.55 GB read and written, 55 us by itself (10
// TB/s: what was read, and part of what was written, stays in L2) and 66 with the
// decisions and the release that follows them.
__global__ void __launch_bounds__(kForkThreads) paged_fork_copy_kernel(PagePoolArgs a)
{
    constexpr int Batch = 8;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t row_bytes = 2LL * a.row;
    const int chunks = static_cast<int>((a.page_size * row_bytes + kForkBytes - 1) / kForkBytes);
    const int64_t copies = static_cast<int64_t>(a.n) * a.layers * 2 * chunks;
    for (int64_t unit = blockIdx.x; unit < copies + a.n; unit += gridDim.x) {
        if (unit < a.n) {
            const PageForkJob job = a.jobs[unit];
            if (job.dst < 0) continue;
            const int32_t *from = a.page_table + static_cast<int64_t>(job.src) * a.max_pages;
            int32_t *to = a.page_table + static_cast<int64_t>(job.dst) * a.max_pages;
            const int full = job.kv / a.page_size;
            for (int m = threadIdx.x; m < full; m += kForkThreads) {
                const int page = from[m];
                to[m] = page;
                if (page >= 0 && page < a.n_pages) atomicAdd(a.refs + page, 1);
                else report_error(a.ws, DG_ERR_DEVICE, 1128);
            }
            if (threadIdx.x == 0 && job.page >= 0) to[full] = job.page;
            continue;
        }
        const int64_t x = unit - a.n;
        const int chunk = static_cast<int>(x % chunks);
        const int kind = static_cast<int>(x / chunks & 1);
        const int layer = static_cast<int>(x / chunks / 2 % a.layers);
        const PageForkJob job = a.jobs[x / chunks / 2 / a.layers];
        if (job.dst < 0 || job.page < 0) continue;
        const int64_t bytes = job.kv % a.page_size * row_bytes;
        const int64_t at = static_cast<int64_t>(chunk) * kForkBytes;
        if (at >= bytes) continue;
        const int n = static_cast<int>(min(bytes - at, static_cast<int64_t>(kForkBytes))) / 16;
        const int page = a.page_table[static_cast<int64_t>(job.src) * a.max_pages + job.kv / a.page_size];
        uint16_t *pool = (kind ? a.v : a.k) + layer * a.layer_stride + at / 2;
        const bool there = page >= 0 && page < a.n_pages;    // (else it reads as zeros)
        if (!there && threadIdx.x == 0) report_error(a.ws, DG_ERR_DEVICE, 1128);
        const uint4 *from = reinterpret_cast<const uint4 *>(pool + (there ? page : 0) * a.page_stride);
        uint4 *to = reinterpret_cast<uint4 *>(pool + job.page * a.page_stride);
        for (int e0 = threadIdx.x; e0 < n; e0 += Batch * kForkThreads) {
            uint4 v[Batch];
#pragma unroll
            for (int e = 0; e < Batch; ++e) {
                v[e] = make_uint4(0, 0, 0, 0);
                if (there && e0 + e * kForkThreads < n) v[e] = from[e0 + e * kForkThreads];
            }
#pragma unroll
            for (int e = 0; e < Batch; ++e)
                if (e0 + e * kForkThreads < n) to[e0 + e * kForkThreads] = v[e];
        }
    }
}

namespace {

// Gives a place's page back.
DG_DEVICE void give_back(const PagePoolArgs &a, int32_t *place)
{
    const int page = *place;
    if (page < 0) return;
    *place = -1;
    if (page >= a.n_pages) {
        report_error(a.ws, DG_ERR_DEVICE, 1132);
        return;
    }
    const int before = atomicSub(a.refs + page, 1);
    if (before == 1) {
        atomicExch(a.refs + page, kPageFreed);
    } else if (before < 1) {                     // nobody's already
        atomicAdd(a.refs + page, 1);
        report_error(a.ws, DG_ERR_DEVICE, 1133);
    }
}

// The pages that have been given back go onto the free ones, the lowest first.  One
// CTA of kPoolThreads; neighbouring threads look at neighbouring pages.
DG_DEVICE void collect(const PagePoolArgs &a, int *sums)
{
    constexpr int Per = 8;                       // pages a thread looks at in a turn
    constexpr int Warps = kPoolThreads / 32;
    __shared__ int s_before[Per * Warps];        // pages given back, by 32 of them
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int n_free = count_free(a);
    for (int p0 = 0; p0 < a.n_pages; p0 += Per * kPoolThreads) {
        int32_t refs[Per];
#pragma unroll
        for (int e = 0; e < Per; ++e) {
            const int page = p0 + e * kPoolThreads + tid;
            refs[e] = page < a.n_pages ? __ldcg(a.refs + page) : 0;
        }
        uint32_t freed[Per];
#pragma unroll
        for (int e = 0; e < Per; ++e) {
            freed[e] = __ballot_sync(0xFFFFFFFFu, refs[e] <= kPageFreed / 2);
            if (lane == 0) s_before[e * Warps + warp] = __popc(freed[e]);
        }
        __syncthreads();
        const int count = tid < Per * Warps ? s_before[tid] : 0;
        int total;
        const int end = block_scan(count, Per * kPoolThreads, sums, &total);
        if (tid < Per * Warps) s_before[tid] = end - count;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < Per; ++e) {
            if (!(freed[e] >> lane & 1u)) continue;
            const int page = p0 + e * kPoolThreads + tid;
            const int at = n_free + s_before[e * Warps + warp] + __popc(freed[e] & ((1u << lane) - 1u));
            a.refs[page] = 0;
            if (at < a.n_pages) a.free_pages[at] = page;
            else report_error(a.ws, DG_ERR_DEVICE, 1134);
        }
        n_free = min(n_free + total, a.n_pages);
        __syncthreads();                         // (before the next turn's counts)
    }
    if (threadIdx.x == 0) *a.n_free = n_free;
}

}  // namespace

// Takes the pages of up to kPoolThreads sequences back, by one CTA.
__global__ void __launch_bounds__(kPoolThreads) paged_release_small_kernel(PagePoolArgs a)
{
    __shared__ int sums[32];
    __shared__ int s_seq[kPoolThreads];          // -1: not (or no longer) one
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    int seq = tid < a.n ? a.dst[tid] : -1;
    s_seq[tid] = seq;
    __syncthreads();
    if (tid < a.n) {
        bool bad = seq < 0 || seq >= a.B;
        for (int j = 0; j < tid && !bad; ++j) bad = s_seq[j] == seq;
        if (bad) {
            report_error(a.ws, DG_ERR_DEVICE, 1131);
            seq = -1;
        } else {
            a.kv_len[seq] = 0;
        }
    }
    __syncthreads();
    s_seq[tid] = seq;
    __syncthreads();
    for (int x = tid; x < a.n * a.max_pages; x += kPoolThreads) {
        const int i = x / a.max_pages;
        if (s_seq[i] >= 0)
            give_back(a, a.page_table + static_cast<int64_t>(s_seq[i]) * a.max_pages + x - i * a.max_pages);
    }
    __syncthreads();
    collect(a, sums);
}

// Takes a sequence's pages back, blockIdx.x its place in the list: up to 16 blocks share
// a long table (2 sequences of 4096 places: 15.5 us with one each).
__global__ void __launch_bounds__(kReleaseThreads) paged_release_kernel(PagePoolArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int i = blockIdx.x;
    const int seq = a.dst[i];
    bool twice = false;
    for (int j = threadIdx.x; j < i; j += kReleaseThreads) twice |= a.dst[j] == seq;
    const bool bad = seq < 0 || seq >= a.B;
    if (__syncthreads_or(twice) || bad) {
        if (blockIdx.y == 0 && threadIdx.x == 0) report_error(a.ws, DG_ERR_DEVICE, 1131);
        return;
    }
    int32_t *row = a.page_table + static_cast<int64_t>(seq) * a.max_pages;
    for (int m = blockIdx.y * kReleaseThreads + threadIdx.x; m < a.max_pages; m += gridDim.y * kReleaseThreads)
        give_back(a, row + m);
    if (blockIdx.y == 0 && threadIdx.x == 0) a.kv_len[seq] = 0;
}

// The pages that the releases took back.
__global__ void __launch_bounds__(kPoolThreads) paged_collect_kernel(PagePoolArgs a)
{
    __shared__ int sums[32];
    griddep_wait();
    griddep_launch_dependents();
    collect(a, sums);
}

}  // namespace dg
