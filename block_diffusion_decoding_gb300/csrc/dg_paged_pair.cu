// dg_paged_pair.cu -- paged attention of chunks: sequences with more folded
// query rows than one 128-row tile.
//
// What dg_paged_attn.cu computes, on 2-CTA clusters that issue 2-SM UMMAs.
// A query tile has 256 rows, 128 per CTA, and both CTAs share every tile of
// 128 keys: CTA r stages keys [64 r, 64 r + 64) of K and dims
// [r D / 2, (r + 1) D / 2) of V, so a key costs each SM half the shared-memory
// traffic of a single-CTA tile and the tensor cores run at their full rate
// (2 x 512 cycles a tile at D = 128, 2 x 1024 at D = 256).
//
// One warpgroup's softmax of a 128 x 128 tile takes about 1800 cycles from
// the arrival of S to that of P (TMEM loads and maximum 450, the exchange of the
// maximum 300, exponentials and packing 1000), more than the UMMAs of a tile.
// So two warpgroups take the tiles in turn, and S is buffered (3 tiles at
// D = 128, 2 at D = 256) far enough ahead of them.  The running maximum goes
// from one to the other through shared memory right after each tile's
// maximum, long before its exponentials; each keeps the sum of its own tiles.
// P is rounded to one bf16 each (the sum keeps fp32): the tensor cores bound this
// kernel, and a second half as in dg_paged_attn.cu would add half to their work.
// The output is then off by sqrt 2 of its own rounding (2.3e-3 of its size against
// 1.7e-3).
//   TMEM        O [128 x D] fp32 | S buffers [128 x 128] fp32 (the bf16 P of a
//               tile overwrites the S it came from);
//   warp 0      TMA: K halves;    warp 2   TMA: V halves;    warp 3   the walk;
//   warp 1      UMMA issuer (even CTA): S runs NS tiles ahead of PV; the odd
//               CTA's passes on that its query rows are in place;
//   warps 4-7   softmax of the even tiles, a query row a thread; warps 8-11 of
//               the odd ones; both load Q rows, and each stores half of O.
// All copies of a tile complete on the even CTA's barrier.  Only where V is
// looked at before its product (its tail, see dg_paged_attn.cu, and values hidden
// from some rows, dg_paged.cuh) each CTA's half lands on a barrier of its own,
// and the arrival of P tells that it has been seen and is clean: there it
// releases memory, elsewhere it only tells of tcgen05 stores that have been waited
// for.  (With every V half landing so the prompt chunks took 7% longer.)
//
// Four chunks of 723 to 2000 tokens over 9905 to 16384 keys (16 query heads on 8,
// D = 128, causal, 0.69 TFLOP): 443-470 us, 1.5 PFLOP/s, under load, where the power
// cap holds the clock at about 1.65 GHz (a large library product sustains 1.72 there,
// 404 us); profiled once, from a cool GPU, the tensor pipe was active 85% of 410 us.
// What made the difference, in us under load: softmax on two
// warpgroups in turn 675 -> 546, registers moved to them 533, whole query tiles in
// turn so that K and V stay in L2 (dg_paged.cuh) 576 -> 505, load warps without
// divisions 455, scores queued right behind the product that frees their buffer
// 446.  Without the exponentials it was no faster, nor without the maximum.
// Short work is a chain of latencies: one 256-token canvas over 4096 keys at
// D = 256 takes 32.7-33.9 us, of which the tensor pipe is active a quarter: division
// and first queries 6, first keys 3, 9 tiles 11, part rows out 3, merge 6.  Five
// blocks through a window of 1024 take 34.9-36.0; 0.7 of it since the tiles that
// land on both CTAs release memory (relaxed, the products could have missed them).
#include "dg_paged.cuh"

namespace dg {

template <int D>
struct PairGeom {
    static constexpr int Dim = D;
    static constexpr int Rows = kPagedPairRows;
    static constexpr int BKV = 128;
    static constexpr int HK = BKV / 2;                     // keys of K this CTA stages
    static constexpr int NAK = D / 64;                     // 64-dim atoms of a K row
    static constexpr int NA = D / 128;                     // of this CTA's V half
    static constexpr int KAtomBytes = HK * 128;
    static constexpr int KBytes = NAK * KAtomBytes;
    static constexpr int KVAtomBytes = BKV * 128;          // V
    static constexpr int VBytes = NA * KVAtomBytes;
    static constexpr int NS = D == 128 ? 3 : 2;            // S buffers
    static constexpr int NK = D == 128 ? 6 : 3;
    static constexpr int NV = D == 128 ? 6 : 2;
    static constexpr int QAtomBytes = 128 * 128;
    static constexpr int QBytes = NAK * QAtomBytes;
    static constexpr int OffQ = 0;
    static constexpr int OffK = OffQ + QBytes;
    static constexpr int OffV = OffK + NK * KBytes;
    static constexpr int OffShared = OffV + NV * VBytes;
    static constexpr int ColO = 0;
    static constexpr int ColS = D;
    static_assert(ColS + NS * BKV <= 512, "TMEM columns");
};

struct PairShared {
    PagedRing ring;
    uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6], v_land[6];
    uint64_t s_full[3], p_full[3];    // by S buffer: P(t + NS) cannot be signalled before
                                      // the UMMA warp has seen P(t) of both CTAs
    uint64_t pv_done[2];              // by tile parity
    uint64_t m_full[2][4];            // by tile parity and lane quadrant
    uint64_t l_full[2][4];            // by warpgroup and lane quadrant
    uint64_t q_ready, o_full, o_free, drained;
    uint64_t q_first;                 // the unit's first queries, once: a load warp may come to
                                      // it any number of parts later
    uint32_t tmem;
    alignas(8) float m[2][128];       // running maximum after a tile, by its parity
    float l[2][128];                  // sum of a warpgroup's tiles of a part
    // by part modulo 3 and half of the dims: the number (from 1) of the last part
    // of which a hidden value of that half was zeroed (told to both CTAs; never
    // cleared, which would have to be ordered with the other CTA's next word)
    uint32_t zeroed[3][2];
};
static_assert(sizeof(PairShared::m) >= kPagedUnits / 2 * sizeof(int64_t), "the division's sums");
static_assert(PairGeom<128>::OffShared + sizeof(PairShared) <= 232448, "shared memory");
static_assert(PairGeom<256>::OffShared + sizeof(PairShared) <= 232448, "shared memory");

// Of the registers that the launch has: kPagedPairRegs a thread, which the host
// makes sure of before it launches.
constexpr int kPairOtherRegs = 88, kPairSoftmaxRegs = 208;
static_assert(128 * kPairOtherRegs + 256 * kPairSoftmaxRegs <= kPagedPairThreads * kPagedPairRegs,
              "registers");

int paged_pair_smem_bytes(int D)
{
    return static_cast<int>((D == 128 ? PairGeom<128>::OffShared : PairGeom<256>::OffShared) +
                            sizeof(PairShared));
}

// One ring's loads, as paged_ring_producer, for this CTA's half of every tile.
template <class Gm, bool IS_V, class Args>
__device__ __forceinline__ void pair_producer(uint8_t *buf, PairShared &sh, uint32_t lead_full, int r,
                                              const CUtensorMap *map_c, const CUtensorMap *map_n,
                                              const Args &a, int where)
{
    constexpr int NS = IS_V ? Gm::NV : Gm::NK;
    constexpr int Bytes = IS_V ? Gm::VBytes : Gm::KBytes;
    constexpr int Atom = IS_V ? Gm::KVAtomBytes : Gm::KAtomBytes;
    constexpr int Atoms = IS_V ? Gm::NA : Gm::NAK;
    constexpr int Keys = IS_V ? Gm::BKV : Gm::HK;          // keys of a tile this CTA loads
    uint64_t *full = IS_V ? sh.v_full : sh.k_full, *empty = IS_V ? sh.v_empty : sh.k_empty;
    const int lane = threadIdx.x & 31;
    const uint64_t pol = policy_evict_normal();
    const int R = a.box_rows, per_tile = Keys / R, batch = 32 / per_tile;
    const int box = lane / Atoms, at = lane % Atoms;
    const int key_off = IS_V ? 0 : r * Gm::HK;             // of this CTA's keys in a tile
    const int dim0 = (IS_V ? r * Gm::NA : 0) * 64 + at * 64;
    uint32_t armed = 0, armed_par = 0, landing = 0;        // by stage; landing: uses of v_land
    int s = 0;
    uint32_t par = 0;                                      // parity of the stages' use
    bool ok = true, first = true;
    PagedItem p;
    for (uint32_t k = 0; ok && paged_take(a, sh.ring, k, p, false, where + 2); ++k) {
        const int32_t *table = a.page_table + static_cast<int64_t>(p.b) * a.max_pages;
        const int nkp = (p.kv + Gm::BKV - 1) / Gm::BKV;
        // page of piece `lane` from this tile on, and its first row in that page
        int32_t page_row[2] = {0, 0};
        auto fetch = [&](int tile, int32_t &row) -> int32_t {
            const int t = tile + lane / per_tile;
            const int key = t * Gm::BKV + key_off + lane % per_tile * R;
            const int at_page = key / a.page_size;
            row = key - at_page * a.page_size;
            return key < p.kv && t < p.tv1 ? __ldg(table + at_page) : 0;
        };
        const PagedSpecial special = paged_special<Gm::BKV>(a, p, paged_edge(a, p));
        // tiles whose keys are all in pages and seen by every row: nearly all
        // of a long part's
        const int plain0 = IS_V ? p.tv0 + special.lo : p.tv0;
        const int plain1 = min(IS_V ? p.tv0 + special.hi : p.tv1, p.kv / Gm::BKV);
        int32_t pages = fetch(p.tv0, page_row[0]), ahead = fetch(p.tv0 + batch, page_row[1]);
        int piece = min(box, per_tile - 1);                // this lane's of the tile
        for (int tv = p.tv0; tv < p.tv1; ++tv, piece += per_tile) {
            if (piece >= batch * per_tile) {
                piece -= batch * per_tile;
                pages = ahead;
                page_row[0] = page_row[1];
                ahead = fetch(tv + batch, page_row[1]);
            }
            int32_t page = __shfl_sync(0xFFFFFFFFu, pages, piece);
            const int32_t row = __shfl_sync(0xFFFFFFFFu, page_row[0], piece);
            if (page < 0 || page >= a.n_pages) page = a.n_pages;   // (reported below)
            ok = mbar_wait_poll<false, kPagedLoadSleep>(&empty[s], par ^ 1u, a.ws, where);
            if (Gm::Dim == 256 && first && (IS_V || tv > p.tv0)) {
                // the first tiles wait for nothing but the queries and K's first
                // (not on q_ready: its phases go on with the parts, those of one
                // tile have no second one to wait with, and a parity that has
                // come round again would hold back what its next phase needs)
                ok &= mbar_wait_poll(&sh.q_first, 0, a.ws, where);
                first = false;
            }
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            uint8_t *dst = buf + s * Bytes + at * Atom;
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | (par << s);
            if (tv >= plain0 && tv < plain1) {
                if (lane == 0 && r == 0) mbar_arrive_expect_tx(&full[s], Gm::BKV * Gm::Dim * 2);
                __syncwarp();
                if (box < per_tile) {
                    // a page id outside the cache: the box lies outside the
                    // tensor, which reads as zeros
                    if (page == a.n_pages) report_error(a.ws, DG_ERR_DEVICE, 912);
                    tma_load_4d_pair(dst + box * R * 128, map_c, lead_full + s * 8, dim0, p.g, row, page,
                                     pol);
                }
                if (++s == NS) {
                    s = 0;
                    par ^= 1u;
                }
                continue;
            }
            const int valid = paged_valid<Gm::BKV>(p, tv);
            const bool paged = tv < nkp;
            const int mine = paged ? (max(0, min(Keys, valid - key_off)) + R - 1) / R : 0;   // boxes
            const bool own = IS_V && special.at(tv - p.tv0);   // lands on this CTA's own barrier
            if (lane == 0) {
                // what both halves bring, or this one alone
                const uint32_t tile_bytes =
                    paged ? static_cast<uint32_t>((valid + R - 1) / R * R * Gm::Dim * 2)
                          : static_cast<uint32_t>(Gm::BKV * Gm::Dim * 2);
                if (own) {
                    mbar_arrive_expect_tx(&sh.v_land[s], tile_bytes / 2);
                    if (r == 0) mbar_arrive(&full[s]);
                } else if (r == 0) {
                    mbar_arrive_expect_tx(&full[s], tile_bytes);
                }
            }
            __syncwarp();
            const uint32_t bar = own ? mapa_shared(smem_u32(&sh.v_land[s]), r) : lead_full + s * 8;
            if (paged) {
                if (box < mine) {
                    if (page == a.n_pages) report_error(a.ws, DG_ERR_DEVICE, 912);
                    tma_load_4d_pair(dst + box * R * 128, map_c, bar, dim0, p.g, row, page, pol);
                }
            } else if (box == 0) {
                tma_load_3d_pair(dst, map_n, bar, dim0, p.g, p.s0 + (tv - nkp) * Gm::BKV + key_off,
                                 pol);
            }
            if (own) landing ^= 1u << s;
            if (++s == NS) {
                s = 0;
                par ^= 1u;
            }
        }
    }
    // every copy has landed before the closing cluster barrier lets either
    // CTA leave: the even CTA's barriers tell of both CTAs' copies
    for (int e = 0; e < NS; ++e) {
        if (r == 0 && (armed >> e & 1u)) mbar_wait_poll(&full[e], armed_par >> e & 1u, a.ws, where + 1);
        // `landing` toggles with every use, so the last phase has parity
        // landing ^ 1 (before any use: the phase before the first, over)
        if (IS_V) mbar_wait_poll(&sh.v_land[e], (landing >> e & 1u) ^ 1u, a.ws, where + 1);
    }
}

// The lowest n bits, n limited to 0 .. 32.
DG_DEVICE uint32_t column_bits(int n)
{
    return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

template <int D, class Args>
__device__ __forceinline__ void paged_pair_body(const CUtensorMap *map_k, const CUtensorMap *map_v,
                                                const CUtensorMap *map_kn,
                                                const CUtensorMap *map_vn, const Args &a)
{
    using Gm = PairGeom<D>;
    constexpr int BKV = Gm::BKV, NK = Gm::NK, NV = Gm::NV, NS = Gm::NS;
    // no room to round the base up: nothing else is in shared memory, so it
    // starts where the swizzled tiles need it
    extern __shared__ __align__(1024) uint8_t smem[];
    PairShared &sh = *reinterpret_cast<PairShared *>(smem + Gm::OffShared);
    if (smem_u32(smem) & 1023u) {
        report_error(a.ws, DG_ERR_DEVICE, 1000);
        return;
    }

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = static_cast<int>(cluster_ctarank());
    const int unit = static_cast<int>(cluster_id_x());
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < NK; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], 1);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(&sh.v_full[s], 1);
            mbar_init(&sh.v_empty[s], 1);
            mbar_init(&sh.v_land[s], 1);
        }
        for (int s = 0; s < NS; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], 8);             // a warpgroup of each CTA
        }
        for (int h = 0; h < 2; ++h) {
            mbar_init(&sh.pv_done[h], 1);
            for (int q = 0; q < 4; ++q) {
                mbar_init(&sh.m_full[h][q], 1);
                mbar_init(&sh.l_full[h][q], 1);
            }
        }
        mbar_init(&sh.q_ready, r == 0 ? 9 : 8);      // its softmax warps; the other CTA's all at once
        mbar_init(&sh.q_first, 8);
        mbar_init(&sh.o_full, 1);
        mbar_init(&sh.o_free, 16);
        mbar_init(&sh.drained, 1);
        paged_ring_init(sh.ring, 11);                // K, V, UMMA, softmax warps
        for (int s = 0; s < 3; ++s) sh.zeroed[s][0] = sh.zeroed[s][1] = 0;
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
        tmem_alloc_pair(&sh.tmem, 512);
        tmem_relinquish_pair();
    }
    // both CTAs' barriers exist before either signals the other; the walking
    // warp looks for that when it has divided the work
    auto together = [&]() -> uint32_t {
        tc_fence_before();
        cluster_sync_all();
        tc_fence_after();
        return sh.tmem;
    };
    auto lead_of = [&](const uint64_t *bar) -> uint32_t { return mapa_shared(smem_u32(bar), 0); };

    // A softmax thread holds 128 scores: its warps take registers from the
    // other four.
    if (warp < 4) {
        reg_dec<kPairOtherRegs>();
        if (warp == 3) {
            // (the maxima's place is free until the first part is known)
            cluster_arrive_all();
            paged_walk<Gm>(a, unit, static_cast<int>(num_clusters_x()), sh.ring, 1007, sh.m,
                           [] { cluster_wait_all(); });
        } else if (warp == 0) {
            together();
            pair_producer<Gm, false>(smem + Gm::OffK, sh, lead_of(sh.k_full), r, map_k, map_kn, a, 1001);
        } else if (warp == 2) {
            together();
            pair_producer<Gm, true>(smem + Gm::OffV, sh, lead_of(sh.v_full), r, map_v, map_vn, a, 1004);
        } else if (warp == 1) {
            // -------------------------------------------------------------- MMA
            // (the whole warp of the even CTA, see elect_lane)
            const uint32_t tmem = together();
            if (r == 0) {
                const uint32_t idesc_s = make_idesc_bf16(256, BKV, 0);
                const uint32_t idesc_o = make_idesc_bf16(256, D, 1);
                // descriptors of the buffers' first tiles; the address sits in
                // the low bits in units of 16 bytes
                const uint64_t dq = make_sdesc_sw128(smem_u32(smem + Gm::OffQ), 16, 1024);
                const uint64_t dk0 = make_sdesc_sw128(smem_u32(smem + Gm::OffK), 16, 1024);
                const uint64_t dv0 = make_sdesc_sw128(smem_u32(smem + Gm::OffV), Gm::KVAtomBytes, 1024);
                int ks = 0, vs = 0, ss = 0, ps = 0;      // stages of K, V, S (written), S (read as P)
                uint32_t kpar = 0, vpar = 0, ppar = 0;
                uint32_t pv = 0, parts = 0;              // tiles multiplied with V, parts
                bool ok = true;
                const bool lead = elect_lane();
                PagedItem p;
                for (uint32_t k = 0; ok && paged_take(a, sh.ring, k, p, false, 1010); ++k) {
                    const int nt = p.tv1 - p.tv0;
                    if (nt == 0) continue;
                    ok = mbar_wait_poll<true>(&sh.q_ready, parts & 1u, a.ws, 1011);
                    ++parts;
                    const int steps_kv = paged_steps(p.kv, BKV), steps_new = paged_steps(p.n, BKV);
                    const int j_kv = (p.kv + BKV - 1) / BKV - 1 - p.tv0;   // last tile of the pages
                    const int j_new = j_kv + (p.n + BKV - 1) / BKV;        // of the new tokens
                    auto score = [&] {                   // S of the next tile
                        const uint64_t dk = dk0 + ks * (Gm::KBytes >> 4);
                        const uint32_t d = tmem + Gm::ColS + ss * BKV;
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                umma_bf16_pair(
                                    d, dq + (((kk >> 2) * Gm::QAtomBytes + (kk & 3) * 32) >> 4),
                                    dk + (((kk >> 2) * Gm::KAtomBytes + (kk & 3) * 32) >> 4), idesc_s,
                                    kk != 0);
                            umma_commit_pair(&sh.s_full[ss], 0x3);
                            umma_commit_pair(&sh.k_empty[ks], 0x3);
                        }
                        if (++ss == NS) ss = 0;
                        if (++ks == NK) {
                            ks = 0;
                            kpar ^= 1u;
                        }
                    };
                    for (int j = 0; j < min(NS, nt) && ok; ++j) {
                        ok = mbar_wait_poll(&sh.k_full[ks], kpar, a.ws, 1012);
                        if (!ok) break;
                        tc_fence_after();
                        score();
                    }
                    for (int j = 0; j < nt && ok; ++j) {
                        // all that the tile's PV and the S behind it need first,
                        // P last: both CTAs' softmax warps have written it (and
                        // read the O of the part before this one)
                        const bool more = j + NS < nt;
                        ok = (!more || mbar_wait_poll(&sh.k_full[ks], kpar, a.ws, 1012)) &&
                             mbar_wait_poll(&sh.v_full[vs], vpar, a.ws, 1014) &&
                             (j > 0 || parts < 2 ||
                              mbar_wait_poll<true>(&sh.o_free, parts & 1u, a.ws, 1016)) &&
                             mbar_wait_poll<true>(&sh.p_full[ps], ppar, a.ws, 1013);
                        if (!ok) break;
                        tc_fence_after();
                        const int steps = j == j_kv ? steps_kv : j == j_new ? steps_new : BKV / 16;
                        const uint64_t dv = dv0 + vs * (Gm::VBytes >> 4);
                        const uint32_t pa = tmem + Gm::ColS + ps * BKV;
                        if (lead) {
                            umma_bf16_pair_ts(tmem + Gm::ColO, pa, dv, idesc_o, j != 0);
                            if (steps == BKV / 16) {
#pragma unroll
                                for (int kk = 1; kk < BKV / 16; ++kk)
                                    umma_bf16_pair_ts(tmem + Gm::ColO, pa + kk * 8, dv + kk * 128, idesc_o,
                                                      1);
                            } else {
                                for (int kk = 1; kk < steps; ++kk)
                                    umma_bf16_pair_ts(tmem + Gm::ColO, pa + kk * 8, dv + kk * 128, idesc_o,
                                                      1);
                            }
                            umma_commit_pair(&sh.v_empty[vs], 0x3);
                            umma_commit_pair(&sh.pv_done[pv & 1], 0x3);
                            if (j + 1 == nt) umma_commit_pair(&sh.o_full, 0x3);
                        }
                        ++pv;
                        if (++ps == NS) {
                            ps = 0;
                            ppar ^= 1u;
                        }
                        if (++vs == NV) {
                            vs = 0;
                            vpar ^= 1u;
                        }
                        if (more) score();               // into the buffer of this tile's P
                    }
                    ok = __all_sync(0xFFFFFFFFu, ok);
                }
                // every UMMA and commit is done before the cluster leaves
                if (lead) umma_commit_pair(&sh.drained, 0x3);
                __syncwarp();
                mbar_wait_poll(&sh.drained, 0, a.ws, 1015);
            } else {
                // the odd CTA's: passes on that its query rows are in place (one
                // arrival ordered over the cluster, by a warp with no memory
                // traffic of its own to wait for)
                uint32_t parts = 0;
                PagedItem p;
                for (uint32_t k = 0; paged_take(a, sh.ring, k, p, false, 1017); ++k) {
                    if (p.tv1 == p.tv0) continue;
                    bool ok = mbar_wait_poll<false, 100>(&sh.q_ready, parts & 1u, a.ws, 1018,
                                                         kPagedWalkLimitNs);   // a whole part
                    ++parts;
                    if (!__all_sync(0xFFFFFFFFu, ok)) break;
                    if (lane == 0) mbar_arrive_cluster(lead_of(&sh.q_ready));
                }
            }
        }
    } else {
        reg_inc<kPairSoftmaxRegs>();
        const uint32_t tmem = together();
        // -------------------------------------------------------------- softmax
        const int wg = (warp - 4) >> 2;          // 0: even tiles, 1: odd tiles
        const int q = warp & 3;                  // TMEM lane quadrant of the warp
        const int rr = q * 32 + lane;            // row within this CTA's 128
        // Rows of a query tile that each CTA has.  Trees, of which many fill part of a
        // tile, share theirs out evenly, in whole warps: the CTA with more is waited for.
        auto share = [](const PagedItem &p) -> int {
            return kPagedTree<Args> ? min(128, (p.rows + 63) / 64 * 32) : 128;
        };
        const uint32_t lane_off = static_cast<uint32_t>(q * 32) << 16;
        const uint32_t to = tmem + lane_off + Gm::ColO;
        uint32_t it = 0, parts = 0;              // tiles and parts before this part
        uint32_t landing = 0;                    // uses of v_land before this part, by stage
        bool ok = true;
        PagedDesc de{-1, 0, 0, 0, 0, 0, {0, 0}};

        // The query rows of an item into shared memory, 16-byte chunks swizzled
        // as TMA would (rows past the tile's last are zero).  A warp loads its
        // 32 rows, each warpgroup half of every row; the lanes of a load lie
        // along the rows.
        auto load_q = [&](const PagedItem &p) {
            const int mine = share(p), row = r * mine + rr;
            if (q * 32 < mine && r * mine + q * 32 < p.rows) {
                constexpr int CPR = D / 16, RPL = 32 / CPR;   // chunks of a half row, rows per load
                const int frow = p.frow0 + min(row, p.rows - 1);
                const int i = frow / a.G;
                const int64_t off = static_cast<int64_t>(p.s0 + i) * a.q_stride +
                                    static_cast<int64_t>(p.g * a.G + frow - i * a.G) * D;
                const int c = wg * CPR + lane % CPR;
                uint4 v[CPR];
#pragma unroll
                for (int n = 0; n < CPR; ++n) {
                    const int64_t o = __shfl_sync(0xFFFFFFFFu, off, n * RPL + lane / CPR);
                    v[n] = __ldg(reinterpret_cast<const uint4 *>(a.q + o) + c);
                }
#pragma unroll
                for (int n = 0; n < CPR; ++n) {
                    const int rw = q * 32 + n * RPL + lane / CPR;   // row within this CTA's 128
                    if (r * mine + rw >= p.rows) v[n] = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(smem + Gm::OffQ + rw * 128 + (c >> 3) * Gm::QAtomBytes +
                                               (((c & 7) ^ (rw & 7)) << 4)) = v[n];
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.q_ready);
                if (D == 256 && it == 0) mbar_arrive(&sh.q_first);   // (no tiles before: once)
            }
        };

        PagedItem p;
        uint32_t k = 0;
        bool more = paged_take(a, sh.ring, k, p, false, 1020);
        if (more && p.tv1 > p.tv0) load_q(p);
        while (more && ok) {
            const int nt = p.tv1 - p.tv0;
            const int mine = share(p), row = r * mine + rr;   // row within the query tile
            const bool live = rr < mine && row < p.rows;
            if (p.kind == kPartFirst)
                de = PagedDesc{p.last, p.rows, p.frow0, p.s0, p.g * a.G, de.part0, {0, 0}};
            else if (p.kind == kPartLater)
                de.part0 = 1;
            const int frow = p.frow0 + (live ? row : 0);
            const int i = frow / a.G;
            const bool busy = q * 32 < mine && r * mine + q * 32 < p.rows;   // the warp has a live row
            float m_ref = -INFINITY, l = 0.f;    // reference of, and sum over, this group's tiles
            const int pos = paged_pos(a, p, i);
            const PagedSpecial special = paged_special<BKV>(a, p, paged_edge(a, p));
            const int buf = static_cast<int>(parts % 3u);
            for (int j = static_cast<int>((it ^ wg) & 1u); j < nt; j += 2) {
                const uint32_t t = it + j;       // tile of the CTA; its parity is wg
                const int ss = static_cast<int>(t % NS);
                const bool odd = special.at(j);  // else whole, and seen by every row
                uint32_t nodes[BKV / 32];        // a tree's columns, a bit each
                if constexpr (kPagedTree<Args>) {
                    const int node0 =
                        paged_key0<BKV>(p, p.tv0 + j) - (a.has_new ? p.kv : p.kv - p.n);
#pragma unroll
                    for (int w = 0; w < BKV / 32; ++w)
                        nodes[w] = odd ? paged_nodes(a, p, i, node0 + 32 * w) : 0xFFFFFFFFu;
                }
                // a wait that runs out is noticed at the tile's end: what is
                // computed until then reaches no memory but the outputs
                // (the other group's maximum is there before its next scores are)
                float m_in = -INFINITY;
                ok = true;
                if (busy && j > 0) {
                    ok = mbar_wait_poll(&sh.m_full[wg ^ 1][q], ((t - 1) >> 1) & 1u, a.ws, 1023);
                    m_in = sh.m[wg ^ 1][rr];
                }
                ok &= mbar_wait_poll(&sh.s_full[ss], (t / NS) & 1u, a.ws, 1022);
                tc_fence_after();
                const uint32_t ts = tmem + lane_off + Gm::ColS + ss * BKV;
                if (busy) {
                    uint32_t sr[BKV];
#pragma unroll
                    for (int c0 = 0; c0 < BKV; c0 += 32)
                        tmem_ld32_nowait(ts + c0, *reinterpret_cast<uint32_t(*)[32]>(&sr[c0]));
                    tmem_wait_ld();
                    if (odd) {
                        // first and last visible column
                        const int valid = paged_valid<BKV>(p, p.tv0 + j), key0 = paged_key0<BKV>(p, p.tv0 + j);
                        const int at = pos - key0;
                        const int last = kPagedTree<Args> ? (a.has_new ? p.kv : p.kv - p.n) + i - key0 : at;
                        const int c_hi = a.causal ? min(valid - 1, last) : valid - 1;
                        int c_lo = a.window > 0 ? max(at - a.window + 1, 0) : 0;
                        // (a tree's window cuts the cached keys alone)
                        if (kPagedTree<Args>)
                            c_lo = min(c_lo, max(0, (a.has_new ? p.kv : p.kv - p.n) - key0));
#pragma unroll
                        for (int c0 = 0; c0 < BKV; c0 += 32) {
                            // 32 columns' visibility, a bit each
                            uint32_t seen = column_bits(c_hi - c0 + 1) & ~column_bits(c_lo - c0);
                            if constexpr (kPagedTree<Args>) seen &= nodes[c0 / 32];
                            if (__all_sync(0xFFFFFFFFu, seen == 0xFFFFFFFFu)) continue;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(seen >> c & 1u)) sr[c0 + c] = __float_as_uint(-INFINITY);
                        }
                    }
                    // the scale is positive, so the scaled maximum is the maximum scaled
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < BKV; c += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mx[e] = max3(mx[e], __uint_as_float(sr[c + 2 * e]),
                                         __uint_as_float(sr[c + 2 * e + 1]));
                    }
                    const float tmax = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.scale_log2;
                    // the reference moves when a tile exceeds it by 2^8
                    const float m_new = m_in == -INFINITY || tmax > m_in + 8.f ? tmax : m_in;
                    sh.m[wg][rr] = m_new;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.m_full[wg][q]);
                    if (__any_sync(0xFFFFFFFFu, m_new != m_ref)) {
                        // a part's first tiles, and few others
                        if (m_ref != m_new && m_ref != -INFINITY) l *= fast_exp2(m_ref - m_new);
                        const bool moved = m_new != m_in && m_in != -INFINITY;
                        m_ref = m_new;
                        if (__any_sync(0xFFFFFFFFu, moved)) {
                            // O holds the PVs up to the tile before: wait for that one
                            const float factor = moved ? fast_exp2(m_in - m_new) : 1.f;
                            ok &= mbar_wait_poll(&sh.pv_done[wg ^ 1], ((t - 1) >> 1) & 1u, a.ws, 1024);
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 16) {
                                uint32_t o[16];
                                tmem_ld16_issue(to + c0, o);
                                tmem_wait_ld16(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
                                tmem_st16(to + c0, o);
                            }
                        }
                    }
                    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
                    const float mexp = (m_ref == -INFINITY) ? 0.f : m_ref;
                    const float2 nm2 = make_float2(-mexp, -mexp);
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c0 = 0; c0 < BKV; c0 += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float2 d2 = fma2(make_float2(__uint_as_float(sr[c0 + c]),
                                                               __uint_as_float(sr[c0 + c + 1])),
                                                   sc2, nm2);
                            const float2 p2 = make_float2(fast_exp2(d2.x), fast_exp2(d2.y));
                            acc[(c >> 1) & 1] = add2(acc[(c >> 1) & 1], p2);
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(p2.x, p2.y);
                            pk[c >> 1] = *reinterpret_cast<const uint32_t *>(&h2);
                        }
                        tmem_st16(ts + c0 / 2, pk);
                    }
                    l += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                    tmem_wait_st();
                } else if (lane == 0) {
                    mbar_arrive(&sh.m_full[wg][q]);      // its phases count the tiles
                }
                if (odd) {
                    const int valid = paged_valid<BKV>(p, p.tv0 + j);
                    const int vs = static_cast<int>(t % NV);
                    uint8_t *v_tile = smem + Gm::OffV + vs * Gm::VBytes;
                    uint32_t uses = landing >> vs;
                    special.each(j, [&](int x) { uses += static_cast<int>((it + x) % NV) == vs; });
                    ok &= mbar_wait_poll(&sh.v_land[vs], uses & 1u, a.ws, 1025);
                    bool hid = false;                    // a value of this thread's key
                    if (valid & 15) paged_zero_tail<Gm>(v_tile, valid, threadIdx.x & 127);
                    if (paged_border(a, paged_edge(a, p), paged_key0<BKV>(p, p.tv0 + j), valid) &&
                        paged_look<Gm>(v_tile, valid, threadIdx.x & 127)) {
                        hid = true;
                        sh.zeroed[buf][r] = parts + 1;
                        st_cluster(mapa_shared(smem_u32(&sh.zeroed[buf][r]), r ^ 1), parts + 1);
                    }
                    hid = __any_sync(0xFFFFFFFFu, hid);
                    tc_fence_before();
                    __syncwarp();
                    // Released: the landed V, zeros over it, and the word that
                    // the other CTA is told by.  What stays in the even CTA needs
                    // no more than its own scope.
                    if (lane == 0) {
                        if (r == 0 && !hid) mbar_arrive(&sh.p_full[ss]);
                        else mbar_arrive_cluster(lead_of(&sh.p_full[ss]));
                    }
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(lead_of(&sh.p_full[ss]));
                }
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
            }
            if (!ok) break;
            special.each(nt, [&](int x) { landing ^= 1u << ((it + x) % NV); });
            // ---------------------------------------------------------- next query, epilogue
            const PagedItem done = p;
            if (nt > 0) {
                // every S of this part is done: its last tile's arrived
                const uint32_t t = it + nt - 1;
                ok = mbar_wait_poll(&sh.s_full[t % NS], (t / NS) & 1u, a.ws, 1026);
                if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
                it += nt;
            }
            more = paged_take(a, sh.ring, ++k, p, false, 1020);
            if (more && p.tv1 > p.tv0) load_q(p);
            const int slot = 2 * unit + (done.kind == kPartFirst ? 1 : 0);
            const int head = done.g * a.G + frow - i * a.G;
            uint16_t *row_out = a.out + static_cast<int64_t>(done.s0 + i) * a.out_stride +
                                static_cast<int64_t>(head) * D;
            constexpr int Half = D / 2;          // dims each warpgroup stores
            if (nt == 0) {                       // no key to see: a zero row
                if (live) {
#pragma unroll 1
                    for (int c = 0; c < Half / 8; ++c)
                        reinterpret_cast<uint4 *>(row_out + wg * Half)[c] = make_uint4(0, 0, 0, 0);
                }
                continue;
            }
            ok = mbar_wait_poll<true>(&sh.o_full, parts & 1u, a.ws, 1027);   // (and zeroed's words)
            if (busy && ok) {
                // this group's sum in the reference of the last tile, which
                // the other group may have set; then both groups' together.
                // (Its slot has been read: O is whole only after every warp
                // was through with the part before.)
                const uint32_t t = it - 1;
                const int last = static_cast<int>(t & 1u);
                float m_last = m_ref;
                if (last != wg) {
                    ok = mbar_wait_poll(&sh.m_full[last][q], (t >> 1) & 1u, a.ws, 1028);
                    m_last = sh.m[last][rr];
                }
                if (l != 0.f && m_ref != m_last) l *= fast_exp2(m_ref - m_last);
                m_ref = m_last;
                sh.l[wg][rr] = l;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.l_full[wg][q]);
            ok = ok && mbar_wait_poll(&sh.l_full[wg ^ 1][q], parts & 1u, a.ws, 1029);
            if (!__all_sync(0xFFFFFFFFu, ok)) { ok = false; break; }
            ++parts;
            tc_fence_after();
            l += sh.l[wg ^ 1][rr];
            if (done.kind != kPartWhole && live && wg == 0)
                a.part_ml[static_cast<int64_t>(slot) * a.slot_rows + row] = make_float2(m_ref, l);
            // the sums are both groups'; so is the reference, for what is added now
            if (busy && sh.zeroed[buf][wg] == parts)
                paged_add_hidden<BKV, Half>(
                    a, done, to, wg * Half, live,
                    static_cast<int64_t>(done.s0 + i) * a.q_stride + static_cast<int64_t>(head) * D, i, pos,
                    m_ref);
            const float inv_l = (l > 0.f) ? 1.f / l : l == 0.f ? 0.f : l;   // no visible key: zero; NaN stays
            bool badv = a.checks && live && !isfinite(l);
            if (busy)
                badv |= !paged_store_row<Half>(a, to, wg * Half, live, done.kind == kPartWhole, row_out,
                                               inv_l, slot, row);
            if (badv) report_error(a.ws, DG_ERR_DEVICE, 1030);
            tc_fence_before();   // O is read before the next part's first PV
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(lead_of(&sh.o_free));
        }
        if (r == 0 && threadIdx.x == 128) a.desc[unit] = de;
    }
    tc_fence_before();
    __syncthreads();
    // no CTA releases its TMEM or leaves while the pair's UMMAs, copies,
    // commits or remote arrivals may still reach it
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(sh.tmem, 512);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPagedPairThreads, 1)
    paged_attn_pair_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v,
                                const __grid_constant__ CUtensorMap map_kn,
                                const __grid_constant__ CUtensorMap map_vn, PagedArgs a)
{
    paged_pair_body<128>(&map_k, &map_v, &map_kn, &map_vn, a);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPagedPairThreads, 1)
    paged_attn_pair_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v,
                                const __grid_constant__ CUtensorMap map_kn,
                                const __grid_constant__ CUtensorMap map_vn, PagedArgs a)
{
    paged_pair_body<256>(&map_k, &map_v, &map_kn, &map_vn, a);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPagedPairThreads, 1)
    paged_tree_pair_kernel_d128(const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v,
                                const __grid_constant__ CUtensorMap map_kn,
                                const __grid_constant__ CUtensorMap map_vn, PagedTreeArgs a)
{
    paged_pair_body<128>(&map_k, &map_v, &map_kn, &map_vn, a);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPagedPairThreads, 1)
    paged_tree_pair_kernel_d256(const __grid_constant__ CUtensorMap map_k,
                                const __grid_constant__ CUtensorMap map_v,
                                const __grid_constant__ CUtensorMap map_kn,
                                const __grid_constant__ CUtensorMap map_vn, PagedTreeArgs a)
{
    paged_pair_body<256>(&map_k, &map_v, &map_kn, &map_vn, a);
}

}  // namespace dg
