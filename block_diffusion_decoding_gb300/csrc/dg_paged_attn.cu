// dg_paged_attn.cu -- attention of the new tokens of a ragged batch over a
// paged KV cache (and, when given, over the tokens' own keys beside it).
//
// Query row (token i, head h) of a sequence sees the keys 0 .. last of its
// sequence: all of them, or causally those up to its own position, or the
// last `window` of those.  The heads of a kv head are folded into the rows of
// a 128-row query tile (row = i G + head in group), so a K/V tile is read
// once for all of them and one new token fills G rows.
//
// The grid is one CTA per SM; the division of the work is dg_paged.cuh's.  A
// CTA works through its parts with its K and V rings running ahead across
// parts, so the memory stream does not stop at an item's end.  Per part:
//   TMEM        O [128 x D] fp32 | S0, S1 [128 x BKV] fp32 | Q [128 x D] bf16
//               (the bf16 P of a tile overwrites the S it came from);
//   warp 0      TMA: K tiles, one box per page piece, into a 4-stage ring;
//   warp 6      TMA: V tiles into a 3-stage ring;
//   warp 1      UMMA issuer: S(0), S(1), PV(0), S(2), PV(1), ...;
//   warps 2-5   Q rows into TMEM, then the softmax, one query row a thread,
//               with a reference maximum that moves only when a tile exceeds
//               it by 2^8; then the output row, or the unnormalised fp32 row
//               with its maximum and sum for paged_merge_kernel.
// A tile whose end is past the last key is loaded, and multiplied with P,
// only up to the next multiple of 16 keys; the softmax warps zero the V rows
// between the last key and there, so that whatever bits the page holds behind
// the sequence (0 x NaN) cannot reach the output.
#include "dg_paged.cuh"

namespace dg {

template <int D>
struct PagedGeom {
    static constexpr int BKV = (D == 128) ? 128 : 64;      // keys per tile
    static constexpr int NA = D / 64;                      // 64-dim atoms
    static constexpr int KVBytes = BKV * D * 2;            // 32 KB
    static constexpr int KVAtomBytes = BKV * 128;
    static constexpr int NK = 4;
    static constexpr int NV = 3;
    static constexpr int OffK = 0;
    static constexpr int OffV = OffK + NK * KVBytes;
    static constexpr int OffBar = OffV + NV * KVBytes;
    static constexpr int Smem = OffBar + 256 + 1024;
    static constexpr int ColO = 0;
    static constexpr int ColS = D;
    static constexpr int ColQ = D + 2 * BKV;
    static_assert(ColQ + D / 2 <= 512, "TMEM columns");
    static_assert(Smem + sizeof(PagedScan) <= 232448, "shared memory");
};

int paged_attn_smem_bytes(int D)
{
    return D == 128 ? PagedGeom<128>::Smem : PagedGeom<256>::Smem;
}

// One ring's loads (K or V) over all parts.  The whole warp: lane l loads the
// box (page piece l / NA, 64-dim atom l % NA) of a tile; the page ids of 32
// pieces ahead are held one per lane, the next 32 already on their way.
template <int D, int NS>
__device__ __forceinline__ void paged_ring_producer(uint8_t *ring, uint64_t *full, uint64_t *empty,
                                                    const CUtensorMap *map_c,
                                                    const CUtensorMap *map_n, const PagedArgs &a,
                                                    const PagedRange &range, int where)
{
    using Gm = PagedGeom<D>;
    const int lane = threadIdx.x & 31;
    const uint64_t pol = policy_evict_first();
    const int R = a.box_rows, per_tile = Gm::BKV / R, batch = 32 / per_tile;
    uint32_t armed = 0, armed_par = 0;
    uint32_t it = 0;
    bool ok = true;
    PagedWalk<128, Gm::BKV> walk;
    walk.start(a, range);
    PagedPart p;
    while (ok && walk.next(a, p)) {
        const int32_t *table = a.page_table + static_cast<int64_t>(p.b) * a.max_pages;
        const int tv0 = p.lo + p.t0, tv1 = p.lo + p.t1;
        auto fetch = [&](int tile) -> int32_t {   // page of piece `lane` from this tile on
            const int key = tile * Gm::BKV + lane * R;
            return key < p.s.kv && tile < tv1 ? __ldg(table + key / a.page_size) : 0;
        };
        int32_t pages = fetch(tv0), ahead = fetch(tv0 + batch);
        for (int tv = tv0; tv < tv1; ++tv, ++it) {
            const int in = (tv - tv0) % batch;
            if (in == 0 && tv > tv0) {
                pages = ahead;
                ahead = fetch(tv + batch);
            }
            const int s = static_cast<int>(it % NS);
            const uint32_t use = it / NS;
            ok = mbar_wait(&empty[s], (use & 1u) ^ 1u, a.ws, where);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            uint8_t *dst = ring + s * Gm::KVBytes;
            if (tv < p.nkp) {
                const int key0 = tv * Gm::BKV;
                const int boxes = (min(Gm::BKV, p.s.kv - key0) + R - 1) / R;
                const int box = lane / Gm::NA, at = lane % Gm::NA;
                int32_t page = __shfl_sync(0xFFFFFFFFu, pages, in * per_tile + min(box, per_tile - 1));
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(boxes * R * D * 2));
                __syncwarp();
                if (box < boxes) {
                    // a page id outside the cache: the box lies outside the
                    // tensor, which reads as zeros
                    if (page < 0 || page >= a.n_pages) {
                        report_error(a.ws, DG_ERR_DEVICE, 912);
                        page = a.n_pages;
                    }
                    const int key = key0 + box * R;
                    tma_load_4d(dst + at * Gm::KVAtomBytes + box * R * 128, map_c, &full[s], at * 64,
                                p.g, key % a.page_size, page, pol);
                }
            } else {
                if (lane == 0) mbar_arrive_expect_tx(&full[s], Gm::KVBytes);
                __syncwarp();
                if (lane < Gm::NA)
                    tma_load_3d(dst + lane * Gm::KVAtomBytes, map_n, &full[s], lane * 64, p.g,
                                p.s.s0 + (tv - p.nkp) * Gm::BKV, pol);
            }
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | ((use & 1u) << s);
        }
    }
    // every copy has landed before the CTA leaves
    for (int s = 0; s < NS; ++s)
        if (armed >> s & 1u) mbar_wait(&full[s], armed_par >> s & 1u, a.ws, where + 1);
}

template <int D>
__device__ __forceinline__ void paged_attn_body(const CUtensorMap *map_k, const CUtensorMap *map_v,
                                                const CUtensorMap *map_kn,
                                                const CUtensorMap *map_vn, const PagedArgs &a)
{
    using Gm = PagedGeom<D>;
    constexpr int BKV = Gm::BKV, NK = Gm::NK, NV = Gm::NV;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PagedScan scan;
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Gm::OffBar);
    uint64_t *k_full = bars;                 // [NK]
    uint64_t *k_empty = k_full + NK;         // [NK]
    uint64_t *v_full = k_empty + NK;         // [NV]
    uint64_t *v_empty = v_full + NV;         // [NV]
    uint64_t *s_full = v_empty + NV;         // [2]
    uint64_t *pv_done = s_full + 2;          // [2]
    uint64_t *p_full = pv_done + 2;          // [2]
    uint64_t *q_ready = p_full + 2;
    uint64_t *o_full = q_ready + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_full + 1);

    // inputs may come from the previous kernel of the stream; nor is TMEM
    // taken before that kernel has given its own back
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < NK; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&pv_done[s], 1);
            mbar_init(&p_full[s], 4);
        }
        mbar_init(q_ready, 4);
        mbar_init(o_full, 1);
        fence_barrier_init();
        tma_prefetch_desc(map_k);
        tma_prefetch_desc(map_v);
        if (a.has_new) {
            tma_prefetch_desc(map_kn);
            tma_prefetch_desc(map_vn);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    paged_divide<128, BKV, kPagedThreads>(a, blockIdx.x, gridDim.x, scan);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const PagedRange range = scan.r;

    if (warp == 0) {
        paged_ring_producer<D, NK>(smem + Gm::OffK, k_full, k_empty, map_k, map_kn, a, range, 921);
    } else if (warp == 6) {
        paged_ring_producer<D, NV>(smem + Gm::OffV, v_full, v_empty, map_v, map_vn, a, range, 923);
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA
        if (lane == 0) {
            const uint32_t idesc_s = make_idesc_bf16(128, BKV, 0);
            const uint32_t idesc_o = make_idesc_bf16(128, D, 1);
            const uint32_t sk0 = smem_u32(smem + Gm::OffK);
            const uint32_t sv0 = smem_u32(smem + Gm::OffV);
            uint32_t it0 = 0, parts = 0;    // tiles and parts before this part
            bool ok = true;
            PagedWalk<128, BKV> walk;
            walk.start(a, range);
            PagedPart p;
            while (ok && walk.next(a, p)) {
                const int nt = p.t1 - p.t0;
                if (nt == 0) continue;
                ok = mbar_wait(q_ready, parts & 1u, a.ws, 931);
                tc_fence_after();
                auto issue_s = [&](int j) -> bool {
                    const uint32_t it = it0 + j;
                    const int s = static_cast<int>(it % NK);
                    if (!mbar_wait(&k_full[s], (it / NK) & 1u, a.ws, 932)) return false;
                    tc_fence_after();
                    const uint32_t sk = sk0 + s * Gm::KVBytes;
                    const uint32_t d = tmem + Gm::ColS + (it & 1) * BKV;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t bdesc = make_sdesc_sw128(
                            sk + (kk >> 2) * Gm::KVAtomBytes + (kk & 3) * 32, 16, 1024);
                        umma_bf16_ts(d, tmem + Gm::ColQ + kk * 8, bdesc, idesc_s, kk != 0);
                    }
                    umma_commit(&k_empty[s]);
                    umma_commit(&s_full[it & 1]);
                    return true;
                };
                auto issue_pv = [&](int j) -> bool {
                    const uint32_t it = it0 + j;
                    const int s = static_cast<int>(it % NV);
                    if (!mbar_wait(&p_full[it & 1], (it >> 1) & 1u, a.ws, 933)) return false;
                    if (!mbar_wait(&v_full[s], (it / NV) & 1u, a.ws, 934)) return false;
                    tc_fence_after();
                    const uint32_t sv = sv0 + s * Gm::KVBytes;
                    const uint32_t pa = tmem + Gm::ColS + (it & 1) * BKV;
                    const int tv = p.lo + p.t0 + j;
                    const int valid = tv < p.nkp ? p.s.kv - tv * BKV
                                                 : p.s.n - (tv - p.nkp) * BKV;
                    const int steps = min(BKV, valid + 15) / 16;
                    for (int kk = 0; kk < steps; ++kk) {
                        const uint64_t bdesc =
                            make_sdesc_sw128(sv + kk * 2048, Gm::KVAtomBytes, 1024);
                        umma_bf16_ts(tmem + Gm::ColO, pa + kk * 8, bdesc, idesc_o, (j | kk) != 0);
                    }
                    umma_commit(&v_empty[s]);
                    umma_commit(&pv_done[it & 1]);
                    return true;
                };
                if (ok) ok = issue_s(0);
                for (int j = 1; j < nt && ok; ++j) ok = issue_s(j) && issue_pv(j - 1);
                if (ok) ok = issue_pv(nt - 1);
                umma_commit(o_full);
                it0 += nt;
                ++parts;
            }
            // every UMMA and commit is done before the CTA leaves
            if (parts > 0) mbar_wait(o_full, (parts - 1) & 1u, a.ws, 935);
        }
    } else {
        // -------------------------------------------------------------- softmax
        const int q = warp & 3;                  // TMEM lane quadrant of the warp
        const int r = q * 32 + lane;             // row within the query tile
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        uint32_t it = 0, parts = 0;
        bool ok = true;
        PagedDesc de{-1, 0, 0, 0, 0, 0, {0, 0}};
        PagedWalk<128, BKV> walk;
        walk.start(a, range);
        PagedPart p;
        while (ok && walk.next(a, p)) {
            const int nt = p.t1 - p.t0;
            const bool live = r < p.rows;
            const int frow = p.frow0 + (live ? r : 0);
            const int i = frow / a.G, hj = frow - i * a.G;
            const int64_t tok = p.s.s0 + i;
            const int head = p.g * a.G + hj;
            uint16_t *row_out = a.out + tok * a.out_stride + static_cast<int64_t>(head) * D;
            if (nt == 0) {                       // no key to see: a zero row
                if (live) {
#pragma unroll 1
                    for (int c = 0; c < D / 8; ++c)
                        reinterpret_cast<uint4 *>(row_out)[c] = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            const bool busy = q * 32 < p.rows;   // the warp has a live row
            {
                // Q row into TMEM (rows past the tile's last are zero)
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + tok * a.q_stride + static_cast<int64_t>(head) * D);
                if (busy) {
#pragma unroll
                    for (int c0 = 0; c0 < D / 2; c0 += 32) {
                        uint32_t w[32];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint4 v = live ? src[(c0 >> 2) + k] : make_uint4(0, 0, 0, 0);
                            w[4 * k] = v.x;
                            w[4 * k + 1] = v.y;
                            w[4 * k + 2] = v.z;
                            w[4 * k + 3] = v.w;
                        }
                        tmem_st32(tmem + lane_off + Gm::ColQ + c0, w);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_ready);
            }
            // position of this row, and the keys it sees
            const int pos = (a.has_new ? p.s.kv : p.s.kv - p.s.n) + i;
            float m_ref = -INFINITY, l = 0.f;
            for (int j = 0; j < nt; ++j, ++it) {
                const int sb = static_cast<int>(it & 1u);
                const int tv = p.lo + p.t0 + j;
                const bool paged = tv < p.nkp;
                const int valid = min(BKV, paged ? p.s.kv - tv * BKV : p.s.n - (tv - p.nkp) * BKV);
                const int key0 = paged ? tv * BKV : p.s.kv + (tv - p.nkp) * BKV;
                if (valid & 15) {
                    // V rows from the last key to the next multiple of 16: zero
                    const int s = static_cast<int>(it % NV);
                    ok = mbar_wait(&v_full[s], (it / NV) & 1u, a.ws, 941);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    uint8_t *sv = smem + Gm::OffV + s * Gm::KVBytes;
                    const int chunks = (((valid + 15) & ~15) - valid) * 8;
                    for (int c = threadIdx.x - 64; c < chunks * Gm::NA; c += 128)
                        *reinterpret_cast<uint4 *>(sv + c / chunks * Gm::KVAtomBytes + valid * 128 +
                                                   c % chunks * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                ok = mbar_wait(&s_full[sb], (it >> 1) & 1u, a.ws, 942);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                tc_fence_after();
                if (busy) {
                    const uint32_t ts = tmem + lane_off + Gm::ColS + sb * BKV;
                    uint32_t sr[BKV];
#pragma unroll
                    for (int c0 = 0; c0 < BKV; c0 += 32)
                        tmem_ld32_nowait(ts + c0, *reinterpret_cast<uint32_t(*)[32]>(&sr[c0]));
                    tmem_wait_ld();
                    // first and last visible column
                    const int c_hi = a.causal ? min(valid - 1, pos - key0) : valid - 1;
                    const int c_lo = a.window > 0 ? pos - a.window + 1 - key0 : 0;
                    if (__any_sync(0xFFFFFFFFu, c_hi < BKV - 1 || c_lo > 0)) {
#pragma unroll
                        for (int c = 0; c < BKV; ++c)
                            if (c > c_hi || c < c_lo) sr[c] = __float_as_uint(-INFINITY);
                    }
                    // the scale is positive, so the scaled maximum is the maximum scaled
                    float rmax = -INFINITY;
#pragma unroll
                    for (int c = 0; c < BKV; c += 2)
                        rmax = max3(rmax, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                    const float tmax = rmax * a.scale_log2;
                    float factor = 1.f;
                    bool rescale = false;
                    if (m_ref == -INFINITY) {
                        m_ref = tmax;
                    } else if (tmax > m_ref + 8.f) {
                        factor = fast_exp2(m_ref - tmax);
                        l *= factor;
                        m_ref = tmax;
                        rescale = true;
                    }
                    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
                    const float mexp = (m_ref == -INFINITY) ? 0.f : m_ref;
                    const float2 nm2 = make_float2(-mexp, -mexp);
                    float2 acc = make_float2(0.f, 0.f);
                    uint32_t pk[BKV / 2];
#pragma unroll
                    for (int c = 0; c < BKV; c += 2) {
                        const float2 d2 = fma2(
                            make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sc2, nm2);
                        const float2 p2 = make_float2(fast_exp2(d2.x), fast_exp2(d2.y));
                        acc = add2(acc, p2);
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(p2.x, p2.y);
                        pk[c >> 1] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    l += acc.x + acc.y;
                    if (__any_sync(0xFFFFFFFFu, rescale)) {
                        // O holds the PVs up to the tile before: wait for the last one
                        ok = mbar_wait(&pv_done[sb ^ 1], ((it - 1) >> 1) & 1u, a.ws, 943);
                        if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            const uint32_t ta = tmem + lane_off + Gm::ColO + c0;
                            tmem_ld32_nowait(ta, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * factor);
                            tmem_st32(ta, o);
                        }
                    }
#pragma unroll
                    for (int c0 = 0; c0 < BKV / 2; c0 += 32)
                        tmem_st32(ts + c0, *reinterpret_cast<const uint32_t(*)[32]>(&pk[c0]));
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[sb]);
            }
            if (!ok) break;
            // ---------------------------------------------------------- epilogue
            ok = mbar_wait(o_full, parts & 1u, a.ws, 944);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            ++parts;
            tc_fence_after();
            const int slot = 2 * blockIdx.x + (p.last >= 0 ? 1 : 0);
            const int64_t prow = static_cast<int64_t>(slot) * a.slot_rows + r;
            if (!p.whole) {
                if (p.last >= 0)
                    de = PagedDesc{p.last, p.rows, p.frow0, p.s.s0, p.g * a.G, de.part0, {0, 0}};
                else
                    de.part0 = 1;
                if (live) a.part_ml[prow] = make_float2(m_ref, l);
            }
            const float inv_l = (l > 0.f) ? 1.f / l : l == 0.f ? 0.f : l;   // no visible key: zero; NaN stays
            bool badv = a.checks && live && !isfinite(l);
            if (busy) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32_nowait(tmem + lane_off + Gm::ColO + c0, o);
                    tmem_wait_ld();
                    if (!live) continue;
                    if (a.checks) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) badv |= !isfinite(__uint_as_float(o[k]));
                    }
                    if (p.whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(row_out + c0);
#pragma unroll
                        for (int k = 0; k < 32; k += 8) {
                            uint32_t w4[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(
                                    __uint_as_float(o[k + 2 * e]) * inv_l,
                                    __uint_as_float(o[k + 2 * e + 1]) * inv_l);
                                w4[e] = *reinterpret_cast<const uint32_t *>(&h2);
                            }
                            dst[k >> 3] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                        }
                    } else {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.part_o + prow * D + c0);
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            dst[k >> 2] = make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                    }
                }
            }
            if (badv) report_error(a.ws, DG_ERR_DEVICE, 945);
            tc_fence_before();   // O is read before the next part's first PV
        }
        if (threadIdx.x == 64) a.desc[blockIdx.x] = de;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_attn_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v,
                           const __grid_constant__ CUtensorMap map_kn,
                           const __grid_constant__ CUtensorMap map_vn, PagedArgs a)
{
    paged_attn_body<128>(&map_k, &map_v, &map_kn, &map_vn, a);
}

__global__ void __launch_bounds__(kPagedThreads, 1)
    paged_attn_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v,
                           const __grid_constant__ CUtensorMap map_kn,
                           const __grid_constant__ CUtensorMap map_vn, PagedArgs a)
{
    paged_attn_body<256>(&map_k, &map_v, &map_kn, &map_vn, a);
}

// Joins the parts of the items that were cut: CTA (c, y) takes rows of the
// item whose first part CTA c left in its slot 1; the others are slot 0 of
// CTAs c + 1 .. last, taken in that order.  out = sum 2^(m_z - M) O_z /
// sum 2^(m_z - M) l_z.  Items of few rows (single tokens) give a row to a
// whole block, its 8 warps each a share of the parts; larger ones a row to a
// warp.
__global__ void __launch_bounds__(256) paged_merge_kernel(PagedArgs a)
{
    __shared__ float s_acc[8][256];
    __shared__ float2 s_ml[8];
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x;
    const PagedDesc de = a.desc[c];
    if (de.last < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = a.D / 32;            // 4 or 8 consecutive dims per lane
    const bool block_row = de.rows <= static_cast<int>(gridDim.y);
    for (int r0 = block_row ? blockIdx.y : blockIdx.y * 8; r0 < de.rows;
         r0 += block_row ? gridDim.y : gridDim.y * 8) {
        const int r = block_row ? r0 : r0 + warp;
        const bool live = r < de.rows;
        float M = -INFINITY, den = 0.f;
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
        const int step = block_row ? 8 : 1;
        if (live) {
            for (int z0 = c + (block_row ? warp : 0); z0 <= de.last; z0 += 4 * step) {
                float2 ml[4];
                float4 v[4][2];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int z = z0 + k * step;
                    const bool have = z <= de.last && (z == c || a.desc[z].part0 != 0);
                    ml[k] = make_float2(-INFINITY, 0.f);
                    v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (have) {
                        const int64_t row =
                            static_cast<int64_t>(2 * z + (z == c ? 1 : 0)) * a.slot_rows + r;
                        ml[k] = a.part_ml[row];
                        const float4 *src =
                            reinterpret_cast<const float4 *>(a.part_o + row * a.D + lane * per);
                        v[k][0] = src[0];
                        if (per == 8) v[k][1] = src[1];
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (ml[k].y == 0.f) continue;        // no visible key in this part
                    if (ml[k].x > M) {
                        const float f = fast_exp2(M - ml[k].x);   // 0 while M = -inf
                        den *= f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] *= f;
                        M = ml[k].x;
                    }
                    const float w = fast_exp2(ml[k].x - M);
                    den = fmaf(w, ml[k].y, den);
                    const float x[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                                        v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, x[e], acc[e]);
                }
            }
        }
        if (block_row) {
            __syncthreads();             // the row before has been read
            if (lane == 0) s_ml[warp] = make_float2(M, den);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < per) s_acc[warp][lane * per + e] = acc[e];
            __syncthreads();
            if (warp > 0) continue;
            float Mt = -INFINITY, dt = 0.f;
            for (int w = 0; w < 8; ++w)
                if (s_ml[w].y != 0.f) Mt = fmaxf(Mt, s_ml[w].x);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            for (int w = 0; w < 8; ++w) {
                const float2 ml = s_ml[w];
                if (ml.y == 0.f) continue;
                const float f = fast_exp2(ml.x - Mt);
                dt = fmaf(f, ml.y, dt);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < per) acc[e] = fmaf(f, s_acc[w][lane * per + e], acc[e]);
            }
            den = dt;
        }
        if (!live) continue;
        const float inv = den == 0.f ? 0.f : 1.f / den;
        if (a.checks) {
            bool bad = !isfinite(den);
#pragma unroll
            for (int e = 0; e < 8; ++e) bad |= !isfinite(acc[e]);
            if (bad) report_error(a.ws, DG_ERR_DEVICE, 951);
        }
        const int frow = de.frow0 + r;
        const int i = frow / a.G, hj = frow - i * a.G;
        uint16_t *dst = a.out + static_cast<int64_t>(de.s0 + i) * a.out_stride +
                        static_cast<int64_t>(de.head0 + hj) * a.D + lane * per;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            if (e < per) {
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
                *reinterpret_cast<uint32_t *>(dst + e) = *reinterpret_cast<const uint32_t *>(&h2);
            }
        }
    }
}

}  // namespace dg
