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
// indices fall, and so meets the mask's words in falling order.  Bound by latency, the
// search for the row's sequence and a read for each ancestor, which its neighbours' walks
// have brought into L1: 2.6 us for a tree of 16 nodes, 5.5 for 256 of up to 64, within the
// 6.2 us that a call from Python takes (in shared memory the parents would cost a barrier
// and be read as often).
__global__ void __launch_bounds__(kTreePlanThreads) tree_plan_kernel(TreePlanArgs a)
{
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x * kTreePlanThreads + threadIdx.x;
    if (t < a.B) {
        const int r0 = __ldg(a.q_start + t), r1 = __ldg(a.q_start + t + 1), kv = __ldg(a.kv_len + t);
        // (lengths that count the nodes are at least as many)
        if (r0 < 0 || r1 < r0 || r1 > a.T || kv < (a.appended ? r1 - r0 : 0) || kv > a.max_kv)
            report_error(a.ws, DG_ERR_DEVICE, 1101);
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
    // (a mask has room for no path that is longer, and a chain of any length ends soon)
    for (int at = i; at >= 0 && depth < 32 * kMaskWords; ++depth) {
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
        a.positions[t] = max(a.appended ? kv - s.n : kv, 0) + depth - 1;
    }
}

// The accepted path of a sequence, and its keys' and values' moves to the places behind
// the cached tokens: node path[j] to place j of the tree's.  A block has up to 128
// times 16 bytes of every token, of the keys or the values of one layer.  Each block
// walks the path for itself, which takes a read of the tree and some votes, less than
// a launch; the first one of a sequence writes it down.  path[j] rises and is at least
// j, so in the order of j no place is written before it has been read, and a thread
// keeps that order by itself.
// Bound by latency: lengths and tree, pages, tokens, one after another.  64 trees of up
// to 32 nodes, 16 layers of 8 heads of 128 (9.2 MB): 8.4 us, one tree of 16, two layers:
// 6.5; with the walk in a kernel of its own the 64 took 8.2, and a second launch of the
// host's time, which the calls back to back are.
__global__ void __launch_bounds__(kTreeCommitThreads) tree_commit_kernel(TreeCommitArgs a)
{
    constexpr int Batch = 8;                     // tokens a thread has in flight
    constexpr int Kept = 4;                      // nodes of the first 128 that a lane of the walk keeps
    __shared__ int path[kTreeCommitThreads];
    __shared__ int64_t from[kTreeCommitThreads], to[kTreeCommitThreads];   // (-1: no move)
    __shared__ int found;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunks = (a.row / 8 + kTreeCommitThreads - 1) / kTreeCommitThreads;
    const int64_t units = static_cast<int64_t>(a.B) * a.layers * 2 * chunks;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int c = static_cast<int>(unit % chunks) * kTreeCommitThreads + threadIdx.x;
        const int64_t rest = unit / chunks;
        const int kind = static_cast<int>(rest & 1);
        const int layer = static_cast<int>((rest >> 1) % a.layers);
        const int b = static_cast<int>((rest >> 1) / a.layers);
        const bool scribe = rest == static_cast<int64_t>(b) * a.layers * 2 && unit % chunks == 0;
        const int r0 = __ldg(a.q_start + b), r1 = __ldg(a.q_start + b + 1), k0 = __ldg(a.kv_len + b);
        const int s0 = min(max(r0, 0), a.T), n = min(max(r1, s0), a.T) - s0;
        const int kv = min(max(k0, 0), a.max_kv), base = kv - n;
        const bool can = n > 0 && base >= 0;
        if (scribe && threadIdx.x == 0 && (r0 != s0 || r1 != s0 + n || kv != k0 || base < 0))
            report_error(a.ws, DG_ERR_DEVICE, 1111);
        int parent[Kept], token[Kept], drawn[Kept];
        if (threadIdx.x < 32 && can) {
#pragma unroll
            for (int e = 0; e < Kept; ++e) {
                const int i = 32 * e + lane;
                parent[e] = i < n ? __ldg(a.parents + s0 + i) : -1;
                token[e] = i < n ? __ldg(a.tokens + s0 + i) : 0;
                drawn[e] = i < n ? __ldg(a.sampled + s0 + i) : 0;
            }
        }
        uint16_t *pool = (kind ? a.v : a.k) + layer * a.layer_stride;
        int at = -1, taken = 0;                  // the walk's: last node, tokens; of warp 0
        int next = -1;
        bool more = can;
        for (int j0 = 0; more || j0 == 0; j0 += kTreeCommitThreads) {
            __syncthreads();                     // the batch before has been moved
            if (threadIdx.x < 32) {
                int m = 0;
                while (more && m < kTreeCommitThreads) {
                    int child = -1;
                    if (at < 0) {
                        child = 0;
                    } else {
#pragma unroll
                        for (int e = 0; e < Kept; ++e) {
                            const bool fits = 32 * e + lane > at && 32 * e + lane < n && parent[e] == at && token[e] == next;
                            const uint32_t any = __ballot_sync(0xFFFFFFFFu, fits);
                            if (child < 0 && any != 0) child = 32 * e + __ffs(any) - 1;
                        }
                        for (int i0 = max(at + 1, 32 * Kept); i0 < n && child < 0; i0 += 32) {
                            const int i = i0 + lane;
                            const bool fits = i < n && __ldg(a.parents + s0 + i) == at && __ldg(a.tokens + s0 + i) == next;
                            const uint32_t any = __ballot_sync(0xFFFFFFFFu, fits);
                            if (any != 0) child = i0 + __ffs(any) - 1;
                        }
                    }
                    if (child < 0) {
                        more = false;
                        break;
                    }
                    at = child;
                    if (at < 32 * Kept) {
#pragma unroll
                        for (int e = 0; e < Kept; ++e) {
                            const int x = __shfl_sync(0xFFFFFFFFu, drawn[e], at & 31);
                            if (at >> 5 == e) next = x;
                        }
                    } else {
                        next = __ldg(a.sampled + s0 + at);
                    }
                    if (lane == 0) {
                        path[m] = at;
                        if (scribe) a.path[static_cast<int64_t>(b) * a.path_max + taken] = at;
                    }
                    ++m;
                    if (++taken == a.path_max) more = false;
                }
                if (lane == 0) found = more ? -m : m;      // (the last batch: not negative)
            }
            __syncthreads();
            const int count = found;
            const int m = abs(count);
            more = count < 0;
            if (static_cast<int>(threadIdx.x) < m) {
                const int j = j0 + threadIdx.x, node = path[threadIdx.x];
                auto place = [&](int key) -> int64_t {
                    const int page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + key / a.page_size);
                    if (page < 0 || page >= a.n_pages) {
                        report_error(a.ws, DG_ERR_DEVICE, 1112);
                        return -1;
                    }
                    return page * a.page_stride + static_cast<int64_t>(key % a.page_size) * a.row;
                };
                from[threadIdx.x] = node != j ? place(base + node) : -1;
                to[threadIdx.x] = node != j ? place(base + j) : -1;
            }
            __syncthreads();
            if (c < a.row / 8) {
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
        }
        if (scribe && threadIdx.x < 32) {
            for (int j = taken + lane; j < a.path_max; j += 32) a.path[static_cast<int64_t>(b) * a.path_max + j] = 0;
            if (lane == 0) {
                a.n_path[b] = taken;
                a.next[b] = next;
                a.kv_out[b] = taken > 0 ? base + taken : kv;
            }
        }
    }
}

}  // namespace dg
