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
//               (P overwrites the S it came from, as two bf16 halves, see below);
//   warp 0      TMA: K tiles, one box per page piece, into a 3-stage ring;
//   warp 6      TMA: V tiles into a 3-stage ring;
//   warp 7      the walk over the parts;
//   warp 1      UMMA issuer: S(0), S(1), PV(0), S(2), PV(1), ...;
//   warps 2-5   Q rows into TMEM, then the softmax, one query row a thread,
//               with a reference maximum that moves only when a tile exceeds
//               it by 2^8; then the output row, or the unnormalised fp32 row
//               with its maximum and sum for paged_merge_kernel.
// Items of up to 16 rows (8 at head dim 256), as nearly all single tokens are,
// would keep one warp busy with 128 columns a row while three idle.  There every
// warp has a copy of the rows in its own TMEM lanes and takes a quarter of each
// tile's columns, with a maximum, a sum and an O of its own (its P is zero in the
// others' columns); at the end they exchange their rows through shared memory.
// P is multiplied as hi + lo, each bf16: hi = the bf16 below the one that p is cut
// off to, lo = bf16(p - hi): neither is negative, nor zero where p is not, so that
// an infinite value stays the infinity it is.  This kernel serves few rows, whose
// time is the memory's, so the second product is free, and the output is off by
// little more than its own rounding (with one bf16 P by sqrt 2 of that).
// A tile whose end is past the last key is loaded, and multiplied with P,
// only up to the next multiple of 16 keys; the softmax warps zero the V rows
// between the last key and there, so that whatever bits the page holds behind
// the sequence (0 x NaN) cannot reach the output.
//
// Bound by HBM: every key and value of a sequence is read once, by bulk copies
// that run up to three tiles of each ahead (192 KB in flight per SM).  64 single
// tokens over caches of 16000 tokens and less (16 query heads on 8, D = 128,
// 2.2 GB): 326-329 us, 6.7 TB/s, 98-99% of a plain copy's rate; with the
// columns of a tile in one warp it took 340.  One token over 300 keys takes
// 12.0-12.6 us, a chain of latencies: launch, the division of the work (1.7 us),
// the queries (1.5 us), the first K tile, three tiles of softmax, the join of the
// four warps' rows (1.5 us) and the merge kernel, which finds nothing to do.
#include "dg_paged.cuh"

namespace dg {

template <int D>
struct PagedGeom {
    static constexpr int Dim = D;
    static constexpr int Rows = 128;                       // query rows per tile
    static constexpr int BKV = (D == 128) ? 128 : 64;      // keys per tile
    static constexpr int NA = D / 64;                      // 64-dim atoms
    static constexpr int KVBytes = BKV * D * 2;            // 32 KB
    static constexpr int KVAtomBytes = BKV * 128;
    static constexpr int NK = 3;
    static constexpr int NV = 3;
    // items of few rows (see below): rows, and the buffer in which the four warps
    // exchange theirs: [warp][row][D] fp32, and (maximum, sum) pairs
    static constexpr int FewRows = (D == 128) ? 16 : 8;
    static constexpr int XBytes = 4 * FewRows * D * 4;
    static constexpr int OffK = 0;
    static constexpr int OffV = OffK + NK * KVBytes;
    static constexpr int OffX = OffV + NV * KVBytes;
    static constexpr int OffXml = OffX + XBytes;
    static constexpr int OffBar = OffXml + 4 * FewRows * 8;
    static constexpr int Smem = OffBar + 256 + 1024;
    static constexpr int ColO = 0;
    static constexpr int ColS = D;
    static constexpr int ColQ = D + 2 * BKV;
    static_assert(ColQ + D / 2 <= 512, "TMEM columns");
    static_assert(Smem + sizeof(PagedRing) + 16 <= 232448, "shared memory");
};

int paged_attn_smem_bytes(int D)
{
    return D == 128 ? PagedGeom<128>::Smem : PagedGeom<256>::Smem;
}

template <int N>
DG_DEVICE void tmem_put(uint32_t taddr, const uint32_t (&r)[N])
{
    if constexpr (N == 16) tmem_st16(taddr, r);
    else tmem_st8(taddr, r);
}

template <int D>
__device__ __forceinline__ void paged_attn_body(const CUtensorMap *map_k, const CUtensorMap *map_v,
                                                const CUtensorMap *map_kn,
                                                const CUtensorMap *map_vn, const PagedArgs &a)
{
    using Gm = PagedGeom<D>;
    constexpr int BKV = Gm::BKV, NK = Gm::NK, NV = Gm::NV;
    extern __shared__ uint8_t smem_raw[];
    __shared__ PagedRing ring;
    __shared__ uint32_t zeroed[3];           // by part modulo 3: a hidden value was zeroed
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
    uint64_t *drained = o_full + 1;
    uint64_t *x_full = drained + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(x_full + 1);

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
        mbar_init(drained, 1);
        mbar_init(x_full, 4);
        zeroed[0] = zeroed[1] = zeroed[2] = 0;
        fence_barrier_init();
        tma_prefetch_desc(map_k);
        tma_prefetch_desc(map_v);
        if (a.has_new) {
            tma_prefetch_desc(map_kn);
            tma_prefetch_desc(map_vn);
        }
    }
    // inputs may come from the previous kernel of the stream; nor is TMEM
    // taken before that kernel has given its own back
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    // the walking warp needs nothing that the others set up, and they its ring
    if (warp == 7) {
        if (lane == 0) {
            paged_ring_init(ring, 3 + 4);    // K, V, UMMA, softmax warps
            fence_barrier_init();
        }
        __syncwarp();
        start_arrive<kPagedThreads>();
    } else {
        tc_fence_before();
        start_sync<kPagedThreads>();
        tc_fence_after();
    }
    const uint32_t tmem = *tmem_slot;    // (not the walking warp's)

    if (warp == 7) {
        paged_walk<Gm>(a, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x), ring, 927, nullptr,
                       [] {});
    } else if (warp == 0) {
        paged_ring_producer<Gm, NK>(smem + Gm::OffK, k_full, k_empty, map_k, map_kn, a, ring, 921);
    } else if (warp == 6) {
        paged_ring_producer<Gm, NV>(smem + Gm::OffV, v_full, v_empty, map_v, map_vn, a, ring, 924);
    } else if (warp == 1) {
        // -------------------------------------------------------------- MMA
        // (the whole warp, see elect_lane)
        const uint32_t idesc_s = make_idesc_bf16(128, BKV, 0);
        const uint32_t idesc_o = make_idesc_bf16(128, D, 1);
        // descriptors of the rings' first tiles; the address sits in the low
        // bits in units of 16 bytes
        const uint64_t dk0 = make_sdesc_sw128(smem_u32(smem + Gm::OffK), 16, 1024);
        const uint64_t dv0 = make_sdesc_sw128(smem_u32(smem + Gm::OffV), Gm::KVAtomBytes, 1024);
        const bool lead = elect_lane();
        int ks = 0, vs = 0;                  // ring stages and their parities
        uint32_t kpar = 0, vpar = 0;
        uint32_t ns = 0, np = 0, parts = 0;  // S and PV tiles issued, parts
        bool ok = true;
        PagedItem p;
        for (uint32_t k = 0; ok && paged_take(a, ring, k, p, false, 930); ++k) {
            const int nt = p.tv1 - p.tv0;
            if (nt == 0) continue;
            ok = mbar_wait_poll(q_ready, parts & 1u, a.ws, 931);
            ++parts;
            const int steps_kv = paged_steps(p.kv, BKV), steps_new = paged_steps(p.n, BKV);
            const int j_kv = (p.kv + BKV - 1) / BKV - 1 - p.tv0;   // last tile of the pages
            const int j_new = j_kv + (p.n + BKV - 1) / BKV;        // of the new tokens
            for (int j = 0; j <= nt && ok; ++j) {
                if (j < nt) {
                    // S(j) overwrites the buffer of P(j - 2), whose PV was issued before
                    ok = mbar_wait_poll(&k_full[ks], kpar, a.ws, 932);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t dk = dk0 + ks * (Gm::KVBytes >> 4);
                    const uint32_t d = tmem + Gm::ColS + (ns & 1) * BKV;
                    if (lead) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            umma_bf16_ts(d, tmem + Gm::ColQ + kk * 8,
                                         dk + (((kk >> 2) * Gm::KVAtomBytes + (kk & 3) * 32) >> 4),
                                         idesc_s, kk != 0);
                        umma_commit(&k_empty[ks]);
                        umma_commit(&s_full[ns & 1]);
                    }
                    ++ns;
                    if (++ks == NK) {
                        ks = 0;
                        kpar ^= 1u;
                    }
                }
                if (j > 0) {
                    const int jp = j - 1;
                    ok = mbar_wait_poll(&v_full[vs], vpar, a.ws, 934) &&
                         mbar_wait_poll(&p_full[np & 1], (np >> 1) & 1u, a.ws, 933);
                    if (!ok) break;
                    tc_fence_after();
                    const int steps = jp == j_kv ? steps_kv : jp == j_new ? steps_new : BKV / 16;
                    const uint64_t dv = dv0 + vs * (Gm::KVBytes >> 4);
                    const uint32_t pa = tmem + Gm::ColS + (np & 1) * BKV;
                    if (lead) {
                        umma_bf16_ts(tmem + Gm::ColO, pa, dv, idesc_o, jp != 0);
                        umma_bf16_ts(tmem + Gm::ColO, pa + BKV / 2, dv, idesc_o, 1);
                        auto both = [&](int kk) {
                            umma_bf16_ts(tmem + Gm::ColO, pa + kk * 8, dv + kk * 128, idesc_o, 1);
                            umma_bf16_ts(tmem + Gm::ColO, pa + BKV / 2 + kk * 8, dv + kk * 128, idesc_o,
                                         1);
                        };
                        if (steps == BKV / 16) {
#pragma unroll
                            for (int kk = 1; kk < BKV / 16; ++kk) both(kk);
                        } else {
                            for (int kk = 1; kk < steps; ++kk) both(kk);
                        }
                        umma_commit(&v_empty[vs]);
                        umma_commit(&pv_done[np & 1]);
                        if (jp + 1 == nt) umma_commit(o_full);
                    }
                    ++np;
                    if (++vs == NV) {
                        vs = 0;
                        vpar ^= 1u;
                    }
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        // every UMMA and commit is done before the CTA leaves
        if (lead) umma_commit(drained);
        __syncwarp();
        mbar_wait_poll(drained, 0, a.ws, 935);
    } else {
        // -------------------------------------------------------------- softmax
        const int q = warp & 3;                  // TMEM lane quadrant of the warp
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t to = tmem + lane_off + Gm::ColO;
        constexpr int CH = BKV / 4;              // columns of a warp with few rows
        uint32_t it = 0, parts = 0, swaps = 0;
        bool ok = true;
        PagedDesc de{-1, 0, 0, 0, 0, 0, {0, 0}};
        PagedItem p;
        for (uint32_t k = 0; ok && paged_take(a, ring, k, p, false, 940); ++k) {
            const int nt = p.tv1 - p.tv0;
            const bool few = p.rows <= Gm::FewRows;
            const int r = few ? lane : q * 32 + lane;   // row within the query tile
            const bool live = r < p.rows;
            const int frow = p.frow0 + (live ? r : 0);
            const int i = frow / a.G, hj = frow - i * a.G;
            const int64_t tok = p.s0 + i;
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
            const bool busy = few || q * 32 < p.rows;   // the warp has a live row
            {
                // Q row into TMEM (rows past the tile's last are zero)
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + tok * a.q_stride + static_cast<int64_t>(head) * D);
                if (busy) {
#pragma unroll 1
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
            const int pos = (a.has_new ? p.kv : p.kv - p.n) + i;
            const PagedEdge edge = paged_edge(a, p);
            const int buf = static_cast<int>(parts % 3u);
            float m_ref = -INFINITY, l = 0.f;

            // Moves the reference to a tile's maximum if that exceeds it by 2^8;
            // false: a wait ran out.
            auto refer = [&](float tmax) -> bool {
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
                if (!__any_sync(0xFFFFFFFFu, rescale)) return true;
                // O holds the PVs up to the tile before: wait for the last one
                const bool done = mbar_wait_poll(&pv_done[(it & 1u) ^ 1u], ((it - 1) >> 1) & 1u, a.ws, 943);
                if (!__all_sync(0xFFFFFFFFu, done)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32_nowait(to + c0, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                    tmem_st32(to + c0, o);
                }
                return true;
            };
            // P of a pair of columns as hi + lo; their sum joins acc
            auto weigh = [&](uint32_t s0, uint32_t s1, float nm, float2 &acc, uint32_t &hi, uint32_t &lo) {
                const float2 d2 = fma2(make_float2(__uint_as_float(s0), __uint_as_float(s1)),
                                       make_float2(a.scale_log2, a.scale_log2), make_float2(nm, nm));
                const float2 p2 = make_float2(fast_exp2(d2.x), fast_exp2(d2.y));
                acc = add2(acc, p2);
                // p down to the bf16 below the one it is cut off to
                const int px = __viaddmax_s32(__float_as_int(p2.x), -0x10000, 0) & ~0xFFFF;
                const int py = __viaddmax_s32(__float_as_int(p2.y), -0x10000, 0) & ~0xFFFF;
                hi = __byte_perm(px, py, 0x7632);
                const float2 r2 = add2(p2, make_float2(-__int_as_float(px), -__int_as_float(py)));
                const __nv_bfloat162 l2 = __floats2bfloat162_rn(r2.x, r2.y);
                lo = *reinterpret_cast<const uint32_t *>(&l2);
            };

            for (int j = 0; j < nt; ++j, ++it) {
                const int sb = static_cast<int>(it & 1u);
                const int valid = paged_valid<BKV>(p, p.tv0 + j);
                const int key0 = paged_key0<BKV>(p, p.tv0 + j);
                const bool border = paged_border(a, edge, key0, valid);
                if ((valid & 15) != 0 || border) {
                    const int s = static_cast<int>(it % NV);
                    uint8_t *v_tile = smem + Gm::OffV + s * Gm::KVBytes;
                    ok = mbar_wait_poll(&v_full[s], (it / NV) & 1u, a.ws, 941);
                    if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                    if (valid & 15) paged_zero_tail<Gm>(v_tile, valid, threadIdx.x - 64);
                    if (border && paged_look<Gm>(v_tile, valid, threadIdx.x - 64)) zeroed[buf] = 1;
                }
                // first and last visible column
                const int c_hi = a.causal ? min(valid - 1, pos - key0) : valid - 1;
                const int c_lo = a.window > 0 ? pos - a.window + 1 - key0 : 0;
                ok = mbar_wait_poll(&s_full[sb], (it >> 1) & 1u, a.ws, 942);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                tc_fence_after();
                const uint32_t ts = tmem + lane_off + Gm::ColS + sb * BKV;
                if (few) {
                    uint32_t sr[CH];
                    if (CH == 32) {
                        tmem_ld32_nowait(ts + q * CH, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                        tmem_wait_ld();
                    } else {
                        tmem_ld16_issue(ts + q * CH, *reinterpret_cast<uint32_t(*)[16]>(&sr[0]));
                        tmem_wait_ld16(*reinterpret_cast<uint32_t(*)[16]>(&sr[0]));
                    }
                    float rmax = -INFINITY;
#pragma unroll
                    for (int c = 0; c < CH; ++c) {
                        if (q * CH + c > c_hi || q * CH + c < c_lo) sr[c] = __float_as_uint(-INFINITY);
                        rmax = fmaxf(rmax, __uint_as_float(sr[c]));
                    }
                    ok = refer(rmax * a.scale_log2);
                    if (!ok) break;
                    const float nm = (m_ref == -INFINITY) ? 0.f : -m_ref;
                    float2 acc = make_float2(0.f, 0.f);
                    uint32_t hi[CH / 2], lo[CH / 2], none[CH / 2];
#pragma unroll
                    for (int c = 0; c < CH / 2; ++c) {
                        weigh(sr[2 * c], sr[2 * c + 1], nm, acc, hi[c], lo[c]);
                        none[c] = 0u;
                    }
                    l += acc.x + acc.y;
#pragma unroll 1
                    for (int h = 0; h < 4; ++h) {   // the other warps' columns: none of this one's
                        if (h == q) continue;
                        tmem_put<CH / 2>(ts + h * (CH / 2), none);
                        tmem_put<CH / 2>(ts + BKV / 2 + h * (CH / 2), none);
                    }
                    tmem_put<CH / 2>(ts + q * (CH / 2), hi);
                    tmem_put<CH / 2>(ts + BKV / 2 + q * (CH / 2), lo);
                    tmem_wait_st();
                } else if (busy) {
                    uint32_t sr[BKV];
#pragma unroll
                    for (int c0 = 0; c0 < BKV; c0 += 32)
                        tmem_ld32_nowait(ts + c0, *reinterpret_cast<uint32_t(*)[32]>(&sr[c0]));
                    tmem_wait_ld();
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
                    ok = refer(rmax * a.scale_log2);
                    if (!ok) break;
                    const float nm = (m_ref == -INFINITY) ? 0.f : -m_ref;
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int c0 = 0; c0 < BKV; c0 += 32) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            weigh(sr[c0 + 2 * c], sr[c0 + 2 * c + 1], nm, acc, hi[c], lo[c]);
                        tmem_st16(ts + c0 / 2, hi);
                        tmem_st16(ts + BKV / 2 + c0 / 2, lo);
                    }
                    l += acc.x + acc.y;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[sb]);
            }
            if (!ok) break;
            // ---------------------------------------------------------- epilogue
            ok = mbar_wait_poll(o_full, parts & 1u, a.ws, 944);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            ++parts;
            tc_fence_after();
            const int slot = 2 * blockIdx.x + (p.kind == kPartFirst ? 1 : 0);
            if (p.kind == kPartFirst)
                de = PagedDesc{p.last, p.rows, p.frow0, p.s0, p.g * a.G, de.part0, {0, 0}};
            else if (p.kind == kPartLater)
                de.part0 = 1;
            if (busy && zeroed[buf] != 0)
                paged_add_hidden<BKV, D>(
                    a, p, to, 0, live, tok * a.q_stride + static_cast<int64_t>(head) * D, pos, m_ref,
                    few ? q * CH : 0, few ? (q + 1) * CH : BKV);
            if (threadIdx.x == 64) zeroed[(buf + 2) % 3] = 0;
            const bool whole = p.kind == kPartWhole;
            bool bad = false;
            if (few) {
                // Each warp has the rows over its own columns: warp q gathers
                // dims [q D / 4, (q + 1) D / 4) of all four, 4 dims a lane.
                constexpr int P4 = D / 16;       // pieces of 4 dims that a warp gathers of a row
                float4 *x = reinterpret_cast<float4 *>(smem + Gm::OffX);
                float2 *xml = reinterpret_cast<float2 *>(smem + Gm::OffXml);
                auto at = [&](int from, int row, int piece) -> float4 * {   // (spread over the banks)
                    return x + (from * Gm::FewRows + row) * (D / 4) + (piece ^ (row & 7));
                };
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32_nowait(to + c, o);
                    tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *at(q, lane, (c + e) / 4) =
                                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                            __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                    }
                    __syncwarp();
                }
                if (live) xml[q * Gm::FewRows + lane] = make_float2(m_ref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(x_full);
                ok = mbar_wait_poll(x_full, swaps & 1u, a.ws, 946);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                ++swaps;
                const int64_t first = tok * a.out_stride + static_cast<int64_t>(head) * D;
                PagedMarks marks{0, 0, 0};
                int marked = -1;                 // the token they are of
#pragma unroll 1
                for (int row0 = 0; row0 < p.rows; row0 += 32 / P4) {
                    const int row = row0 + lane / P4, piece = q * P4 + lane % P4;
                    const int64_t row_first = __shfl_sync(0xFFFFFFFFu, first, row & 31);
                    float m = -INFINITY, sum = 0.f;
                    float v[4] = {0.f, 0.f, 0.f, 0.f};
                    if (row < p.rows) {
                        float2 ml[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            ml[h] = xml[h * Gm::FewRows + row];
                            if (ml[h].y != 0.f) m = fmaxf(m, ml[h].x);
                        }
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            if (ml[h].y == 0.f) continue;   // no key of its columns
                            const float f = fast_exp2(ml[h].x - m);
                            const float4 t = *at(h, row, piece);
                            sum = fmaf(f, ml[h].y, sum);
                            if (f == 0.f) continue;         // (nor one that counts)
                            v[0] = fmaf(f, t.x, v[0]);
                            v[1] = fmaf(f, t.y, v[1]);
                            v[2] = fmaf(f, t.z, v[2]);
                            v[3] = fmaf(f, t.w, v[3]);
                        }
                    }
                    // an infinite value times the other warps' zeros is NaN
                    const uint32_t odd = __ballot_sync(
                        0xFFFFFFFFu, !(fabsf(v[0]) + fabsf(v[1]) + fabsf(v[2]) + fabsf(v[3]) < INFINITY));
                    if (odd != 0) {
                        bad = true;
#pragma unroll 1
                        for (int h = 0; h < 32 / P4; ++h) {   // the rows of this turn
                            if ((odd >> (h * P4) & ((1u << P4) - 1u)) == 0) continue;
                            const int i_h = (p.frow0 + row0 + h) / a.G;
                            if (i_h != marked) {
                                marks = paged_marks<BKV, D / 4>(a, p, i_h, q * (D / 4));
                                marked = i_h;
                            }
                            if (lane / P4 != h) continue;
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = paged_marked(marks, lane % P4 * 4 + e, v[e]);
                        }
                    }
                    if (row < p.rows) {
                        if (whole) {
                            const float inv = (sum > 0.f) ? 1.f / sum : sum == 0.f ? 0.f : sum;
                            const __nv_bfloat162 lo2 = __floats2bfloat162_rn(v[0] * inv, v[1] * inv);
                            const __nv_bfloat162 hi2 = __floats2bfloat162_rn(v[2] * inv, v[3] * inv);
                            *reinterpret_cast<uint2 *>(a.out + row_first + piece * 4) =
                                make_uint2(*reinterpret_cast<const uint32_t *>(&lo2),
                                           *reinterpret_cast<const uint32_t *>(&hi2));
                        } else {
                            *part_at(a, slot, row, piece * 4) = make_float4(v[0], v[1], v[2], v[3]);
                            if (piece == 0)
                                a.part_ml[static_cast<int64_t>(slot) * a.slot_rows + row] = make_float2(m, sum);
                        }
                        bad |= !isfinite(sum);
                    }
                    __syncwarp();
                }
                if (a.checks && bad) report_error(a.ws, DG_ERR_DEVICE, 945);
            } else {
                const float inv_l = (l > 0.f) ? 1.f / l : l == 0.f ? 0.f : l;   // no visible key: zero; NaN stays
                if (busy) bad = !paged_store_row<D>(a, to, 0, live, whole, row_out, inv_l, slot, r);
                if (!whole && live)
                    a.part_ml[static_cast<int64_t>(slot) * a.slot_rows + r] = make_float2(m_ref, l);
                if (a.checks && live && (bad || !isfinite(l))) report_error(a.ws, DG_ERR_DEVICE, 945);
            }
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

// Joins the parts of the items that were cut.  An item's first part is in slot 1
// of unit c, which describes it; the others are in slot 0 of units c + 1 ..
// last, taken in that order: out = sum 2^(m_z - M) O_z / sum 2^(m_z - M) l_z.
// A thread takes 16 dims of a row, neighbouring threads neighbouring rows, with
// the loads of kMergeParts parts in flight; a block takes the next 256 of those
// in all the items.  An item too small to fill a block (single tokens, whose
// caches may have parts from every SM) shares its parts out over the block's
// threads and joins their results in shared memory.
// Bound by latency, not bytes: the descriptors, then all of a thread's parts,
// then the row.  One 256-token canvas over 4096 keys at D = 256, 16 items in about
// 90 parts (22 MB, from L2 and HBM): 10 us from cold caches, about 6 behind the
// kernel that wrote them.  A block per possible row group instead (2432 of them
// there, most with nothing to do) took 12.4; 3, 4 and 6 parts in flight no less
// than 2.
struct MergeState {
    float M, den;
    float acc[16];
};

DG_DEVICE void merge_add(MergeState &s, float m, float l, const float (&x)[16])
{
    if (l == 0.f) return;                    // no visible key there
    if (m > s.M) {
        const float f = fast_exp2(s.M - m);  // 0 while M = -inf
        s.den *= f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s.acc[e] *= f;
        s.M = m;
    }
    const float w = fast_exp2(m - s.M);
    s.den = fmaf(w, l, s.den);
#pragma unroll
    for (int e = 0; e < 16; ++e) s.acc[e] = fmaf(w, x[e], s.acc[e]);
}

__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(PagedArgs a, int units)
{
    __shared__ float s_state[18][kMergeThreads];
    __shared__ int s_end[kMergeThreads];     // blocks of work up to and with unit t's item
    __shared__ int s_warp[kMergeThreads / 32];
    __shared__ int s_part0[kMergeThreads];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    {
        int n = 0;
        if (tid < units) {
            const PagedDesc de = a.desc[tid];
            if (de.last >= 0) n = (de.rows * (a.D / 16) + kMergeThreads - 1) / kMergeThreads;
            s_part0[tid] = de.part0;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, n, o);
            if (lane >= o) n += v;
        }
        if (lane == 31) s_warp[warp] = n;
        __syncthreads();
        for (int w = 0; w < warp; ++w) n += s_warp[w];
        s_end[tid] = n;
        __syncthreads();
    }
    const int total = s_end[kMergeThreads - 1];
    for (int job = blockIdx.x; job < total; job += gridDim.x) {
        int c = 0;                               // the first unit with s_end > job
#pragma unroll
        for (int o = kMergeThreads / 2; o > 0; o >>= 1)
            if (s_end[c + o - 1] <= job) c += o;
        const PagedDesc de = a.desc[c];
        const int p0 = (job - (c > 0 ? s_end[c - 1] : 0)) * kMergeThreads;
        const int pairs = de.rows * (a.D / 16);
        // threads that share a pair's parts
        int share = 1;
        while (share < 32 && pairs * share * 2 <= kMergeThreads) share *= 2;
        const int at = p0 + tid;
        const int part = share > 1 ? at / pairs : 0;
        const int pair = at - part * pairs;
        const bool live = part < share && pair < pairs;
        const int dg = pair / de.rows, row = pair - dg * de.rows;
        MergeState s;
        s.M = -INFINITY;
        s.den = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s.acc[e] = 0.f;
        if (live) {
            for (int z0 = c + part; z0 <= de.last; z0 += kMergeParts * share) {
                float2 ml[kMergeParts];
                float4 x[kMergeParts][4];
#pragma unroll
                for (int k = 0; k < kMergeParts; ++k) {
                    const int z = z0 + k * share;
                    ml[k] = make_float2(0.f, 0.f);
                    if (z > de.last || (z > c && s_part0[z] == 0)) continue;
                    const int slot = 2 * z + (z == c ? 1 : 0);
                    ml[k] = a.part_ml[static_cast<int64_t>(slot) * a.slot_rows + row];
                    const float4 *src = part_at(a, slot, row, dg * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[k][e] = src[static_cast<int64_t>(e) * a.slot_rows];
                }
#pragma unroll
                for (int k = 0; k < kMergeParts; ++k) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[4 * e] = x[k][e].x;
                        v[4 * e + 1] = x[k][e].y;
                        v[4 * e + 2] = x[k][e].z;
                        v[4 * e + 3] = x[k][e].w;
                    }
                    merge_add(s, ml[k].x, ml[k].y, v);
                }
            }
        }
        if (share > 1) {
            __syncthreads();                     // the job before has been read
            s_state[0][tid] = s.M;
            s_state[1][tid] = s.den;
#pragma unroll
            for (int e = 0; e < 16; ++e) s_state[2 + e][tid] = s.acc[e];
            __syncthreads();
            if (part > 0) continue;
            for (int k = 1; live && k < share; ++k) {
                const int t = tid + k * pairs;
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = s_state[2 + e][t];
                merge_add(s, s_state[0][t], s_state[1][t], x);
            }
        }
        if (!live) continue;
        if (a.checks) {
            bool bad = !isfinite(s.den);
#pragma unroll
            for (int e = 0; e < 16; ++e) bad |= !isfinite(s.acc[e]);
            if (bad) report_error(a.ws, DG_ERR_DEVICE, 951);
        }
        const int frow = de.frow0 + row;
        const int i = frow / a.G, hj = frow - i * a.G;
        store_bf16x16(a.out + static_cast<int64_t>(de.s0 + i) * a.out_stride +
                          static_cast<int64_t>(de.head0 + hj) * a.D + dg * 16,
                      s.acc, s.den == 0.f ? 0.f : 1.f / s.den, a.out_wide != 0);
    }
}

}  // namespace dg
