// Arguments and launch constants of the kernels around drafted trees: their plan
// and commit (dg_tree.cu), the page pool (dg_pages.cu) and the draw of tokens from
// logits (dg_sample.cu).
#pragma once

#include "dg_kernels.h"

namespace dg {

// ---------------------------------------------------------------- draws from logits
struct SampleArgs {
    const void *logits;             // [R, V], rows `stride` elements apart
    int64_t stride;
    int R, V;
    int ctas;                       // a row's CTAs, a cluster
    int rows_warp;                  // 512-byte pieces of a row that a warp reads
    const float *temperature, *top_p, *min_p, *u;   // [R]; null (but u): not applied
    const int32_t *top_k;
    int32_t *token;
    float *logprob;                 // may be null
};
constexpr int kSampleThreads = 256, kSampleWarps = kSampleThreads / 32;
constexpr int kSampleCtas = 4;        // CTAs of an SM
constexpr int kSampleCluster = 16;    // CTAs of a row at most
constexpr int kSampleRows = 400;      // rows_warp at most
int sample_smem_bytes();
__global__ void sample_bf16_kernel(const __grid_constant__ SampleArgs a);
__global__ void sample_fp32_kernel(const __grid_constant__ SampleArgs a);

// ---------------------------------------------------------------- drafted trees
struct TreePlanArgs {
    const int32_t *parents, *q_start, *kv_len;
    int T, B, max_kv;
    int window, appended, words;
    uint32_t *mask;                 // [T, words]
    int32_t *positions;             // [T] or null
    WsHeader *ws;
};
constexpr int kTreePlanThreads = 128;
constexpr int kMaskWords = 128;       // of a row of the mask at most
__global__ void tree_plan_kernel(TreePlanArgs a);

struct TreeCommitArgs {
    const int32_t *tokens, *parents, *sampled, *q_start, *kv_len, *page_table;
    int T, B, max_kv;
    int32_t *path, *n_path, *next, *kv_out;
    int path_max;
    uint16_t *k, *v;
    int64_t page_stride, layer_stride;
    int page_size, n_pages, max_pages, layers;
    int row;                        // values of a token in a page: Hkv D
    WsHeader *ws;
};
constexpr int kTreeCommitThreads = 128;
__global__ void tree_commit_kernel(TreeCommitArgs a);

// ---------------------------------------------------------------- page pool
struct PageForkJob {
    int32_t src, dst, kv;           // dst < 0: not made
    int32_t page;                   // the copy's, or -1: nothing to copy
};
struct PagePoolArgs {
    int32_t *free_pages, *n_free, *refs;
    int32_t *page_table, *kv_len;
    const int32_t *q_start;
    int n_pages, max_pages, page_size, B;
    const int32_t *src, *dst;       // fork: [n]; release: dst alone
    int n;
    uint16_t *k, *v;
    int64_t page_stride, layer_stride;
    int layers, row;
    PageForkJob *jobs;
    WsHeader *ws;
};
constexpr int kPoolThreads = 1024;    // of the single-CTA kernels: sequences of a turn, forks of a call
constexpr int kForkThreads = 256;
constexpr int kForkBytes = 32768;     // of a page that a block copies
constexpr int kReleaseThreads = 256;
constexpr int kReleaseSmall = 4096;  // places in tables and pages of a release by one CTA
__global__ void paged_reserve_kernel(PagePoolArgs a);
__global__ void paged_fork_kernel(PagePoolArgs a);
__global__ void paged_fork_copy_kernel(PagePoolArgs a);
__global__ void paged_release_small_kernel(PagePoolArgs a);
__global__ void paged_release_kernel(PagePoolArgs a);
__global__ void paged_collect_kernel(PagePoolArgs a);

}  // namespace dg
