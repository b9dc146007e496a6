// dg_tree.cu -- drafted trees: the plan of a batch of them (which nodes each one
// sees, and at which positions they are), and the commit of the paths that were
// accepted.
#include "dg_serve_kernels.h"

namespace dg {

namespace {

// Sequence b's rows of the batch, cut to it.
struct Rows {
    int s0, n;
};
DG_DEVICE Rows rows_of(const int32_t *q_start, int b, int T)
{
    const int s0 = min(max(__ldg(q_start + b), 0), T);
    return {s0, min(max(__ldg(q_start + b + 1), s0), T) - s0};
}

}  // namespace

// A node sees itself and its ancestors: a thread walks up its node's parents, whose
// indices fall, and so meets the mask's words in falling order.
__global__ void __launch_bounds__(kTreePlanThreads) tree_plan_kernel(TreePlanArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x * kTreePlanThreads + threadIdx.x;
    if (t < a.B) {
        const int r0 = __ldg(a.q_start + t), r1 = __ldg(a.q_start + t + 1), kv = __ldg(a.kv_len + t);
        if (r0 < 0 || r1 < r0 || r1 > a.T || kv < 0 || kv > a.max_kv) report_error(a.ws, DG_ERR_DEVICE, 1101);
    }
    if (t >= a.T) return;
    // the last sequence that begins at or before this row
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.q_start + mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    const Rows s = rows_of(a.q_start, lo, a.T);
    const int i = t - s.s0;
    if (i < 0 || i >= s.n) return;               // nobody's row
    uint32_t *row = a.mask + static_cast<int64_t>(t) * a.words;
    int w = a.words - 1, depth = 0;
    uint32_t bits = 0;
    if (i >= 32 * a.words) report_error(a.ws, DG_ERR_DEVICE, 1102);
    for (int at = i; at >= 0; ++depth) {
        for (; w > at >> 5; --w) {
            row[w] = bits;
            bits = 0;
        }
        if (w == at >> 5 && (a.window == 0 || depth < a.window)) bits |= 1u << (at & 31);
        const int up = __ldg(a.parents + s.s0 + at);
        if (up >= at || up < -1) {
            report_error(a.ws, DG_ERR_DEVICE, 1103);
            at = -1;
        } else {
            at = up;
        }
    }
    for (; w >= 0; --w) {
        row[w] = bits;
        bits = 0;
    }
    if (a.positions != nullptr) {
        const int kv = min(max(__ldg(a.kv_len + lo), 0), a.max_kv);
        a.positions[t] = (a.appended ? kv - s.n : kv) + depth - 1;
    }
}

// The accepted path of each sequence, by a warp: from the root (its first node)
// on to the first child whose token is the one sampled at its parent.
__global__ void __launch_bounds__(kTreeWalkThreads) tree_walk_kernel(TreeCommitArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int b = (blockIdx.x * kTreeWalkThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (b >= a.B) return;
    const int r0 = __ldg(a.q_start + b), r1 = __ldg(a.q_start + b + 1), k0 = a.kv_len[b];
    const Rows s = rows_of(a.q_start, b, a.T);
    const int kv = min(max(k0, 0), a.max_kv);
    const int base = kv - s.n;
    if (lane == 0 && (r0 != s.s0 || r1 != s.s0 + s.n || kv != k0 || base < 0))
        report_error(a.ws, DG_ERR_DEVICE, 1111);
    int32_t *path = a.path + static_cast<int64_t>(b) * a.path_max;
    int n = 0, next = -1;
    if (s.n > 0 && base >= 0) {
        int at = 0;
        for (;;) {
            if (lane == 0) path[n] = at;
            ++n;
            next = __ldg(a.sampled + s.s0 + at);
            if (n == a.path_max) break;
            int child = -1;
            for (int c0 = at + 1; c0 < s.n && child < 0; c0 += 32) {
                const int c = c0 + lane;
                const bool fits = c < s.n && __ldg(a.parents + s.s0 + c) == at && __ldg(a.tokens + s.s0 + c) == next;
                const uint32_t any = __ballot_sync(0xFFFFFFFFu, fits);
                if (any != 0) child = c0 + __ffs(any) - 1;
            }
            if (child < 0) break;
            at = child;
        }
    }
    for (int j = n + lane; j < a.path_max; j += 32) path[j] = 0;
    if (lane == 0) {
        a.n_path[b] = n;
        a.next[b] = next;
        a.kv_out[b] = n > 0 ? base + n : kv;
    }
}

// Moves the accepted nodes' keys and values of every layer to the places behind the
// cached tokens: node path[j] to place j of the tree's.  path[j] rises and is at
// least j, so in the order of j no place is written before it has been read; a
// thread has 16 bytes of every token and keeps that order by itself.
__global__ void __launch_bounds__(kTreeMoveThreads) tree_move_kernel(TreeCommitArgs a)
{
    constexpr int Batch = 8;
    __shared__ int64_t from[kTreeMoveThreads], to[kTreeMoveThreads];   // (-1: no such page)
    griddep_wait();
    griddep_launch_dependents();
    const int chunks = (a.row / 8 + kTreeMoveThreads - 1) / kTreeMoveThreads;
    const int64_t units = static_cast<int64_t>(a.B) * a.layers * 2 * chunks;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int c = static_cast<int>(unit % chunks) * kTreeMoveThreads + threadIdx.x;
        const int64_t rest = unit / chunks;
        const int kind = static_cast<int>(rest & 1);
        const int layer = static_cast<int>((rest >> 1) % a.layers);
        const int b = static_cast<int>((rest >> 1) / a.layers);
        const int n = a.n_path[b];
        const int base = a.kv_out[b] - n;
        const int32_t *path = a.path + static_cast<int64_t>(b) * a.path_max;
        if (n == 0 || path[n - 1] == n - 1) continue;     // nothing, or all in place
        uint16_t *pool = (kind ? a.v : a.k) + layer * a.layer_stride;
        for (int j0 = 0; j0 < n; j0 += kTreeMoveThreads) {
            const int m = min(kTreeMoveThreads, n - j0);
            __syncthreads();                              // the offsets before have been read
            if (static_cast<int>(threadIdx.x) < m) {
                const int j = j0 + threadIdx.x;
                auto place = [&](int key) -> int64_t {
                    const int page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + key / a.page_size);
                    if (page < 0 || page >= a.n_pages) {
                        report_error(a.ws, DG_ERR_DEVICE, 1112);
                        return -1;
                    }
                    return page * a.page_stride + static_cast<int64_t>(key % a.page_size) * a.row;
                };
                const bool moves = path[j] != j;
                from[threadIdx.x] = moves ? place(base + path[j]) : -1;
                to[threadIdx.x] = moves ? place(base + j) : -1;
            }
            __syncthreads();
            if (c >= a.row / 8) continue;
            for (int j = 0; j < m; j += Batch) {
                uint4 x[Batch];
#pragma unroll
                for (int e = 0; e < Batch; ++e) {
                    x[e] = make_uint4(0, 0, 0, 0);
                    if (j + e < m && from[j + e] >= 0)
                        x[e] = *reinterpret_cast<const uint4 *>(pool + from[j + e] + 8 * c);
                }
#pragma unroll
                for (int e = 0; e < Batch; ++e)
                    if (j + e < m && to[j + e] >= 0) *reinterpret_cast<uint4 *>(pool + to[j + e] + 8 * c) = x[e];
            }
        }
        __syncthreads();
    }
}

}  // namespace dg
