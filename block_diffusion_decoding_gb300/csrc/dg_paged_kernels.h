// Arguments and launch constants of the q / k norm, rotation and append kernels
// (dg_qkv.cu) and of the paged attention (dg_paged_attn.cu, dg_paged_pair.cu).
#pragma once

#include "dg_kernels.h"

namespace dg {

// ---------------------------------------------------------------- q / k norm, rotation, paged append
struct QkvArgs {
    const uint16_t *q, *k, *v;          // [T, heads, D], rows *_stride elements apart
    int64_t q_stride, k_stride, v_stride;
    uint16_t *q_out, *k_out;            // k_out: dense destination only
    int64_t qo_stride, ko_stride;
    const int32_t *positions;           // [T] (paged: null = the index in the cache)
    const uint64_t *steps;              // [rot / 2] turns per position, 64-bit fixed point
    const uint16_t *q_weight, *k_weight;
    float eps, weight_offset;
    int T, D, rot, interleaved;
    int nq, nk;                         // q heads, k (and v) heads of the pass
    int lanes, lanes_log2;              // lanes of a head's group
    float inv_d;                        // 1 / D
    int chunks, q_chunks, k_chunks;     // groups per token, those for q and for k
    // paged destination
    uint16_t *k_cache, *v_cache;
    int64_t page_stride;                // elements between pages
    int page_size, n_pages, max_pages, B;
    const int32_t *page_table, *kv_len, *q_start;
    int32_t *kv_len_out;
    WsHeader *ws;
};
constexpr int kQkvThreads = 128;
constexpr int kQkvSeqSmem = 512;    // sequences whose first rows are staged in shared memory
// by the heads of a group
__global__ void qk_norm_rope_kernel_1(QkvArgs a);
__global__ void qk_norm_rope_kernel_4(QkvArgs a);
__global__ void qk_norm_rope_kernel_8(QkvArgs a);
__global__ void paged_append_kernel_1(QkvArgs a);
__global__ void paged_append_kernel_4(QkvArgs a);
__global__ void paged_append_kernel_8(QkvArgs a);

// ---------------------------------------------------------------- paged attention
// What a CTA left for the merge: slot 0 holds a part that continues an item
// begun by an earlier CTA, slot 1 one that a later CTA continues.
struct PagedDesc {
    int32_t last;        // slot 1 in use: the CTA with the item's last part, else -1
    int32_t rows;        // its folded rows
    int32_t frow0;       // first folded row of the item within its sequence
    int32_t s0;          // first token of its sequence
    int32_t head0;       // first query head of its kv head
    int32_t part0;       // slot 0 in use
    int32_t pad[2];
};
struct PagedArgs {
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    int T, B, Hq, Hkv, G, D;
    int page_size, box_rows, n_pages, max_pages;
    const int32_t *page_table, *kv_len, *q_start;
    // the tensors behind the maps, for what is read outside the tiles
    const uint16_t *k_pages, *v_pages, *k_new, *v_new;
    int64_t page_stride, k_stride, v_stride;
    int has_new, causal, window;
    int small;           // the division of the work fits 32-bit integers
    int checks;
    float scale_log2;
    int out_wide;        // output rows are 32-byte aligned
    int slot_rows;       // rows of a part slot
    float *part_o;       // [2 CTAs][D / 4][slot_rows][4] unnormalised rows
    float2 *part_ml;     // [2 CTAs][slot_rows] (reference max in base 2, sum)
    PagedDesc *desc;     // [CTAs]
    WsHeader *ws;
};
// Drafted trees: of the new tokens a row sees those that its bits name, and every
// cached key before them (with a window: after its position - window).
struct PagedTreeArgs : PagedArgs {
    const uint32_t *mask;       // [T, words]
    const int32_t *positions;   // [T], read with a window
    int words;
};
constexpr int kPagedThreads = 256;   // warps as kAttnThreads, and 7 walks the parts
__global__ void paged_attn_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                                       const __grid_constant__ CUtensorMap map_v,
                                       const __grid_constant__ CUtensorMap map_kn,
                                       const __grid_constant__ CUtensorMap map_vn, PagedArgs a);
__global__ void paged_attn_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                                       const __grid_constant__ CUtensorMap map_v,
                                       const __grid_constant__ CUtensorMap map_kn,
                                       const __grid_constant__ CUtensorMap map_vn, PagedArgs a);
__global__ void paged_tree_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                                       const __grid_constant__ CUtensorMap map_v,
                                       const __grid_constant__ CUtensorMap map_kn,
                                       const __grid_constant__ CUtensorMap map_vn, PagedTreeArgs a);
__global__ void paged_tree_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                                       const __grid_constant__ CUtensorMap map_v,
                                       const __grid_constant__ CUtensorMap map_kn,
                                       const __grid_constant__ CUtensorMap map_vn, PagedTreeArgs a);
constexpr int kMergeThreads = 256;   // at least as many as there are units
constexpr int kMergeParts = 2;       // parts whose loads a thread has in flight
__global__ void paged_merge_kernel(PagedArgs a, int units);
int paged_attn_smem_bytes(int D);
// Chunks: query tiles of 256 rows on 2-CTA clusters (dg_paged_pair.cu)
constexpr int kPagedPairThreads = 384;
constexpr int kPagedPairRows = 256;
constexpr int kPagedPairRegs = 168;   // registers a thread it is launched with
__global__ void paged_attn_pair_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                                            const __grid_constant__ CUtensorMap map_v,
                                            const __grid_constant__ CUtensorMap map_kn,
                                            const __grid_constant__ CUtensorMap map_vn, PagedArgs a);
__global__ void paged_attn_pair_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                                            const __grid_constant__ CUtensorMap map_v,
                                            const __grid_constant__ CUtensorMap map_kn,
                                            const __grid_constant__ CUtensorMap map_vn, PagedArgs a);
__global__ void paged_tree_pair_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                                            const __grid_constant__ CUtensorMap map_v,
                                            const __grid_constant__ CUtensorMap map_kn,
                                            const __grid_constant__ CUtensorMap map_vn, PagedTreeArgs a);
__global__ void paged_tree_pair_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                                            const __grid_constant__ CUtensorMap map_v,
                                            const __grid_constant__ CUtensorMap map_kn,
                                            const __grid_constant__ CUtensorMap map_vn, PagedTreeArgs a);
int paged_pair_smem_bytes(int D);

}  // namespace dg
