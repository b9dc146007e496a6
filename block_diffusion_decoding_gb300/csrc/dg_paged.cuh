// dg_paged.cuh -- how the paged attention kernels divide their work.
//
// The lengths of the sequences are device data, so the division is made on
// the device, by one warp of every CTA for itself, from the lengths alone.  An item is
// one query tile (ROWS folded rows = positions x heads of one kv head) of one
// kv head of one sequence; it costs a fixed part plus its visible keys.  The
// items in the order (sequence, kv head, query tile) lie end to end on a line
// of total cost W, CTA c takes the stretch from c s to (c + 1) s, s the n-th
// part of W, and a cut inside an item falls between two of its key tiles.  So the CTAs' work is
// equal whatever the lengths are, a CTA leaves at most two unfinished parts
// (one at each end of its stretch), and the parts of an item are those of
// consecutive CTAs: they are merged in that order, whoever was first.
//
// A cut has a price: a part's unfinished rows are written and read again in
// fp32, by a second kernel.  Where whole items spread almost as evenly, as many
// to each CTA as to any other, they are left whole, item i to CTA i modulo their
// number.
//
// Chunks of many query tiles do both: CTA pair u takes the items u, u + units, ...
// whole while that leaves more than one for each, and the line's rest is cut so
// that all have the same in the end.  So the pairs at work at one time are at
// neighbouring items, which share a few heads' keys and values, and find them in
// L2: in stretches of the whole line, four chunks of up to 2000 tokens over up to
// 16384 keys had every head of every sequence in use at once and read 2.4 GB from
// HBM of which 0.29 GB is distinct, and took 576 us; so they read 0.29 GB and took
// 505 (both with that build's slower load warps: dg_paged_pair.cu).
#pragma once

#include <type_traits>

#include "dg_paged_device.cuh"
#include "dg_paged_kernels.h"

namespace dg {

// The arithmetic of the division runs on the host too (checked there).
#define DG_BOTH __host__ __device__ __forceinline__

DG_BOTH int32_t paged_load(const int32_t *p)
{
#ifdef __CUDA_ARCH__
    return __ldg(p);
#else
    return *p;
#endif
}

template <typename T>
DG_BOTH T paged_min(T a, T b)
{
    return a < b ? a : b;
}
template <typename T>
DG_BOTH T paged_max(T a, T b)
{
    return a > b ? a : b;
}

// In keys, by the rows of a query tile (128: one CTA, 256: a pair of them): an
// item's fixed cost (its queries, pipeline fill, epilogue); what cutting a
// batch's items costs every unit (parts and merge); the least a unit is given.
// From sweeps over chunk and single-token batches: the pair's epilogue and merge
// move 256 rows in fp32, about 8 us, 7 key tiles.  (Item for the pair, by one
// canvas of 256 tokens over 4096 keys alone: 1152 or 1536 33.9 us instead of 32.7.
// Cut 1536: no difference.)
template <int ROWS>
struct PagedCost {
    static constexpr int Item = ROWS == 256 ? 768 : 512;
    static constexpr int Cut = ROWS == 256 ? 1024 : 512;
    static constexpr int Least = 512;
};

// I: the integers the line is measured in, 32-bit where the host has seen that
// no line of these tensors is longer (PagedArgs::small): the walk is on the
// path to every CTA's first load.
template <class I>
struct PagedSeq {
    int s0, n, kv;      // first token, tokens, cached keys
    int mt;             // query tiles of a kv head
    int mc;             // tiles whose key count still grows with the tile index
    I x0, slope, cap, fixed;

#ifdef __CUDACC__
    // Lane `at`'s.
    DG_DEVICE PagedSeq from(int at) const
    {
        auto get = [&](auto v) { return __shfl_sync(0xFFFFFFFFu, v, at); };
        return PagedSeq{get(s0), get(n), get(kv), get(mt), get(mc), get(x0), get(slope), get(cap), get(fixed)};
    }
#endif
};

// Bounds every length by what the tensors hold, so that no later index can
// leave them; *bad: 1 when something had to be cut, 2 when q_start decreases.
template <int ROWS, int BKV, class I>
DG_BOTH PagedSeq<I> paged_seq(const PagedArgs &a, int b, int *bad = nullptr)
{
    PagedSeq<I> s;
    const int r0 = paged_load(a.q_start + b), r1 = paged_load(a.q_start + b + 1);
    const int k0 = paged_load(a.kv_len + b);
    s.s0 = paged_min(paged_max(r0, 0), a.T);
    s.n = paged_min(paged_max(r1, s.s0), a.T) - s.s0;
    s.kv = paged_min(paged_max(k0, 0), a.max_pages * a.page_size);
    if (bad != nullptr) *bad = r1 < r0 ? 2 : r0 != s.s0 || r1 != s.s0 + s.n || k0 != s.kv ? 1 : 0;
    s.mt = (s.n * a.G + ROWS - 1) / ROWS;
    const I G = a.G;
    s.fixed = G * PagedCost<ROWS>::Item + 1;
    s.cap = 0;
    s.mc = s.mt;
    if (!a.causal) {
        s.slope = 0;
        s.x0 = G * (s.kv + (a.has_new ? s.n : 0));
    } else {
        s.slope = ROWS;
        s.x0 = G * paged_max(0, a.has_new ? s.kv : s.kv - s.n);
        if (a.window > 0) {
            s.cap = G * (paged_min(a.window, s.kv + s.n) + BKV) + ROWS;
            const I k = s.cap < s.x0 ? 0 : (s.cap - s.x0) / ROWS;
            s.mc = static_cast<int>(paged_min<I>(k, s.mt));
        }
    }
    return s;
}

// Cost of the first m query tiles of one kv head.
template <class I>
DG_BOTH I paged_prefix(const PagedSeq<I> &s, int m)
{
    const I k = paged_min(m, s.mc);
    return m * s.fixed + k * s.x0 + s.slope * (k * (k + 1) / 2) + (m - k) * s.cap;
}

// No negative operands.
template <class I>
DG_BOTH I paged_div(I x, I y)
{
    return sizeof(I) == 4 ? static_cast<I>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y)) : x / y;
}

// Host: whether every line of these tensors can be measured in 32 bits.
inline bool paged_small(int T, int B, int Hkv, int G, int64_t max_kv)
{
    const int64_t items = static_cast<int64_t>(Hkv) * (static_cast<int64_t>(T) * G / 128 + B);
    const int64_t cost = G * (max_kv + 2 * static_cast<int64_t>(T) + PagedCost<256>::Item + 256) + 1024;
    return cost < (1 << 30) && items < (1 << 30) / cost;
}

// The length of a unit's stretch (a unit: a CTA, or a pair of them) of a line
// of cost W.
template <int ROWS, class I>
DG_BOTH I paged_step(const PagedArgs &a, I W, int units)
{
    const I least = static_cast<I>(a.G) * PagedCost<ROWS>::Least;
    const I n = paged_min<I>(units, paged_max<I>(paged_div(W, least), 1));
    return paged_div<I>(W + n - 1, n);
}

// Whether a line of cost W, with `items` items of cost `most` at most, is left
// uncut: when the unit with most items is done before the cuts would pay.
template <int ROWS, class I>
DG_BOTH bool paged_whole(const PagedArgs &a, I W, I items, I most, int units)
{
    const I rounds = paged_div<I>(items + units - 1, units);
    // (in 64 bits: rounds x most may be longer than the line)
    return static_cast<int64_t>(rounds) * most <=
           static_cast<int64_t>(paged_div<I>(W, units)) + static_cast<int64_t>(a.G) * PagedCost<ROWS>::Cut;
}

// Whole items that every unit takes before the line's rest is cut (0: all of it
// is).  Where a sequence's heads have few query tiles the pairs do not meet at a
// head's keys, and the sums would cost more than they bring.  (16 items a sequence,
// and the sixteenth below, are estimates: neither was swept.)
template <int ROWS>
DG_BOTH int paged_rounds(const PagedArgs &a, int64_t items, int units)
{
    return ROWS == 256 && items >= 2 * units && items >= 16LL * a.B ? static_cast<int>(items / units) - 1 : 0;
}
// ... and whether they leave those who have most with no more than their share
// (and a sixteenth) of a line of cost W.
template <class I>
DG_BOTH bool paged_even(I W, int units, I most)
{
    const I share = W / units;
    return most <= share + share / 16;
}

template <class I>
struct PagedRange {
    int waves;               // whole items: u, u + units, ...
    int units;
    I at;                    // waves > 0: item u's place among those of sequence b
    I begin, end;            // this unit's stretch of the line (end <= begin: none)
    I step;                  // every unit's, or 0: they differ
    I item;                  // waves == 0: where the item that `begin` falls in begins
    int b, g, m;             // that item
};

// The item of sequence b (which begins at `base`) that position x falls in.
template <class I>
DG_BOTH void paged_locate(const PagedSeq<I> &s, int b, I base, I x, PagedRange<I> &r)
{
    const I head = paged_prefix(s, s.mt);
    I y = x - base;
    r.b = b;
    r.g = static_cast<int>(paged_div(y, head));
    y -= r.g * head;
    int lo = 0, hi = s.mt - 1;   // the last tile that begins at or before y
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (paged_prefix(s, mid) <= y) lo = mid;
        else hi = mid - 1;
    }
    r.m = lo;
    r.item = base + r.g * head + paged_prefix(s, lo);
}

constexpr int kPagedUnits = 256;     // units there may be of single CTAs; half of that of pairs
template <int ROWS>
constexpr int kPagedBounds = kPagedUnits / (ROWS / 128) / 32;   // units a lane keeps the bound of

// The line's rest after `rounds` whole items of every unit, cut so that all have
// the same: false if the whole ones are too unequal.  By one warp; q: its
// sequences' lengths in a batch of up to 32; bound: where the stretches of this
// lane's units begin; sums: shared memory, an I per unit.  (Apart from the rest
// of the division, which every small batch runs from a cold instruction cache.)
template <int ROWS, int BKV, class I>
__device__ __noinline__ bool paged_take_rounds(const PagedArgs &a, int rounds, int units, I W,
                                               PagedSeq<I> q, I (&bound)[kPagedBounds<ROWS>], void *sums)
{
    using Sum = std::conditional_t<sizeof(I) == 4, unsigned, unsigned long long>;
    constexpr int K = kPagedBounds<ROWS>;
    constexpr uint32_t all = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31;
    // what the whole items of every unit cost, an item a lane
    Sum *sum = static_cast<Sum *>(sums);
    for (int e = lane; e < units; e += 32) sum[e] = 0;
    __syncwarp();
    const I end = static_cast<I>(rounds) * units;
    I first = 0;                                 // item of the sequence
    for (int b0 = 0; first < end; b0 += 32) {
        if (a.B > 32) q = paged_seq<ROWS, BKV, I>(a, min(b0 + lane, a.B - 1));
        for (int j = 0; j < min(32, a.B - b0) && first < end; ++j) {
            const PagedSeq<I> t = q.from(j);
            if (t.mt == 0) continue;
            const I n = static_cast<I>(a.Hkv) * t.mt;
            int m = lane % t.mt, to = static_cast<int>((first + lane) % units);
            const int dm = 32 % t.mt, dto = 32 % units;
            for (I e = lane; e < n && first + e < end; e += 32) {
                atomicAdd(&sum[to], static_cast<Sum>(paged_prefix(t, m + 1) - paged_prefix(t, m)));
                m += dm;
                if (m >= t.mt) m -= t.mt;
                to += dto;
                if (to >= units) to -= units;
            }
            __syncwarp();
            first += n;
        }
    }
    I dearest = 0, taken = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int e = lane * K + k;
        bound[k] = e < units ? static_cast<I>(sum[e]) : 0;
        dearest = max(dearest, bound[k]);
        taken += bound[k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        dearest = max(dearest, __shfl_xor_sync(all, dearest, o));
        taken += __shfl_xor_sync(all, taken, o);
    }
    if (!paged_even(W, units, dearest)) return false;
    // each gets what it is short of its share of the line
    const I share = (W + units - 1) / units;
    I at = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const I left = lane * K + k < units ? max(share - bound[k], I(0)) : 0;
        bound[k] = at;
        at += left;
    }
    I incl = at;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I v = __shfl_up_sync(all, incl, o);
        if (lane >= o) incl += v;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) bound[k] = min(W, taken + incl - at + bound[k]);
    return true;
}

// Unit u of `units`: its share.  By one warp, a sequence a lane and 32 at a
// time: once over all of them for the line's cost, and again up to the one that
// the stretch begins in (a batch of up to 32 keeps its lengths in registers),
// whose lengths are left in s.  bound: where the stretches of this lane's units
// begin, if they differ.  sums: shared memory, an I per pair.
template <int ROWS, int BKV, class I>
DG_DEVICE PagedRange<I> paged_divide(const PagedArgs &a, int u, int units, PagedSeq<I> &s,
                                     I (&bound)[kPagedBounds<ROWS>], void *sums)
{
    const int lane = threadIdx.x & 31;
    constexpr uint32_t all = 0xFFFFFFFFu;
    PagedRange<I> r{};
    r.units = units;
    int bad = 0;
    // this lane's sequences: cost, items, the dearest item
    I mine = 0, W = 0, items = 0, most = 0;
    PagedSeq<I> q{};
#pragma unroll 1
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        if (b0 + lane >= a.B) continue;
        int cut;
        q = paged_seq<ROWS, BKV, I>(a, b0 + lane, &cut);
        bad |= cut;
        mine = a.Hkv * paged_prefix(q, q.mt);
        W += mine;
        items += a.Hkv * q.mt;
        if (q.mt > 0) most = max(most, paged_prefix(q, q.mt) - paged_prefix(q, q.mt - 1));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        W += __shfl_xor_sync(all, W, o);
        items += __shfl_xor_sync(all, items, o);
        most = max(most, __shfl_xor_sync(all, most, o));
    }
    if (bad != 0 && u == 0) report_error(a.ws, DG_ERR_DEVICE, 911);
    // rows of several sequences may be longer than any line that was counted
    // on: nothing is computed
    if (__any_sync(all, bad & 2)) return r;
    if (W == 0) return r;
    if (paged_whole<ROWS>(a, W, items, most, units)) {
        if (u >= items) return r;
        r.waves = static_cast<int>(paged_div<I>(items - u + units - 1, units));
    } else {
        r.step = paged_step<ROWS>(a, W, units);
        r.begin = u * r.step;
        r.end = min(W, r.begin + r.step);
    }
    if constexpr (ROWS == 256) {
        const int rounds = paged_rounds<ROWS>(a, items, units);
        if (rounds > 0 && r.waves == 0 && paged_take_rounds<ROWS, BKV, I>(a, rounds, units, W, q, bound, sums)) {
            constexpr int K = kPagedBounds<ROWS>;
            r.begin = r.end = W;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const I begin = __shfl_sync(all, bound[k], u / K);
                if (k == u % K) r.begin = begin;
                const I end = __shfl_sync(all, bound[k], (u + 1) / K);
                if (k == (u + 1) % K && u + 1 < units) r.end = end;
            }
            r.step = 0;
            r.waves = rounds;
        }
    }
    if (r.waves == 0 && r.begin >= r.end) return r;
    // the first item: by its number, or by the place on the line
    const I x = r.waves > 0 ? u : r.begin;
    I base = 0;
    for (int b0 = 0;; b0 += 32) {
        if (a.B > 32) {
            q = paged_seq<ROWS, BKV, I>(a, min(b0 + lane, a.B - 1));
            if (b0 + lane >= a.B) q.mt = 0;
        }
        mine = a.Hkv * (r.waves > 0 ? q.mt : paged_prefix(q, q.mt));
        I incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I v = __shfl_up_sync(all, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t past = __ballot_sync(all, base + incl > x);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            base += __shfl_sync(all, incl - mine, at);
            s = q.from(at);
            r.b = b0 + at;
            r.at = x - base;
            if (r.waves == 0) paged_locate(s, r.b, base, x, r);
            return r;
        }
        base += __shfl_sync(all, incl, 31);
    }
}

// The unit whose stretch has place x of the line.  All lanes of the warp that
// divided it.
template <int ROWS, class I>
DG_DEVICE int paged_unit_of(const PagedRange<I> &r, const I (&bound)[kPagedBounds<ROWS>], I x)
{
    if (r.step > 0) return static_cast<int>(paged_div<I>(x, r.step));
    int n = 0;               // bounds that are not above
    for (int k = 0; k < kPagedBounds<ROWS>; ++k)
        n += __popc(__ballot_sync(0xFFFFFFFFu, (static_cast<int>(threadIdx.x) & 31) * kPagedBounds<ROWS> + k <
                                                       r.units && bound[k] <= x));
    return n - 1;
}

// One stretch's share of an item.
struct PagedPart {
    int s0, n, kv;       // the sequence
    int b, g;
    int frow0, rows;     // folded rows of the query tile
    int nkp;             // key tiles of the pages (further ones: the chunk's own keys)
    int lo;              // first visible key tile
    int t0, t1;          // this part's tiles, from lo
    int nt;              // the item's
    int last;            // first part of several: the unit with the last one, else -1
    bool whole;
};

// Walks a unit's whole items, then the parts of its stretch.
template <int ROWS, int BKV, class I>
struct PagedWalk {
    PagedSeq<I> s, ahead;   // this sequence, the next one's lengths (already loaded)
    int b, g, m;
    I at;                   // whole items: the next one's place in the sequence
    int waves;              // how many are left
    I item, begin, end;
    PagedRange<I> r;

    // first: the lengths of sequence r.b
    DG_BOTH void start(const PagedArgs &a, const PagedRange<I> &range, const PagedSeq<I> &first)
    {
        r = range;
        waves = r.waves;
        b = r.b;
        at = r.at;
        s = first;
        item = end = r.end;
        if (waves == 0 && r.begin < r.end) stretch(a);
    }

    // On to the sequence that item `at` is of.
    DG_BOTH void settle(const PagedArgs &a)
    {
        while (at >= static_cast<I>(a.Hkv) * s.mt && b + 1 < a.B) {
            at -= static_cast<I>(a.Hkv) * s.mt;
            s = paged_seq<ROWS, BKV, I>(a, ++b);
        }
    }

    DG_BOTH void stretch(const PagedArgs &a)
    {
        begin = r.begin;
        g = r.g;
        m = r.m;
        item = r.item;
        ahead = s;
        if (b + 1 < a.B) ahead = paged_seq<ROWS, BKV, I>(a, b + 1);
    }

    // To where the stretch begins.
    DG_BOTH void find(const PagedArgs &a)
    {
        I base = 0;
        for (b = 0;; ++b) {
            s = paged_seq<ROWS, BKV, I>(a, b);
            const I all = static_cast<I>(a.Hkv) * paged_prefix(s, s.mt);
            if (base + all > r.begin || b + 1 == a.B) break;
            base += all;
        }
        paged_locate(s, b, base, r.begin, r);
        stretch(a);
    }

    // What a part has of its item: all but its share of the tiles.
    DG_BOTH void fill(const PagedArgs &a, PagedPart &p) const
    {
        p.s0 = s.s0;
        p.n = s.n;
        p.kv = s.kv;
        p.b = b;
        p.g = g;
        p.frow0 = m * ROWS;
        p.rows = paged_min(ROWS, s.n * a.G - p.frow0);
        p.nkp = (s.kv + BKV - 1) / BKV;
        int hi, lo = 0;
        if (!a.causal) {
            hi = p.nkp + (a.has_new ? (s.n + BKV - 1) / BKV : 0);
        } else {
            const int i1 = (p.frow0 + p.rows - 1) / a.G;
            hi = a.has_new ? p.nkp + i1 / BKV + 1 : paged_max(0, (s.kv - s.n + i1 + BKV) / BKV);
        }
        if (a.window > 0) {
            const int i0 = p.frow0 / a.G;
            const int first = (a.has_new ? s.kv : s.kv - s.n) + i0 - a.window + 1;
            if (first > 0)
                lo = a.has_new && first >= s.kv ? p.nkp + (first - s.kv) / BKV : first / BKV;
        }
        p.lo = lo;
        p.nt = paged_max(0, hi - lo);
    }

    // The next part; false: there are no more.  unit_of(x): the unit whose
    // stretch has place x of the line.
    template <class UnitOf>
    DG_BOTH bool next(const PagedArgs &a, PagedPart &p, UnitOf unit_of)
    {
        if (waves > 0) {
            g = static_cast<int>(paged_div<I>(at, s.mt));
            m = static_cast<int>(at) - g * s.mt;
            fill(a, p);
            p.t0 = 0;
            p.t1 = p.nt;
            p.last = -1;
            p.whole = true;
            at += r.units;
            if (--waves > 0) settle(a);
            else if (r.begin < r.end) find(a);
            return true;
        }
        while (item < end) {
            const I cost = paged_prefix(s, m + 1) - paged_prefix(s, m);
            fill(a, p);
            // a tile is worth its keys: BKV x G of the cost after the fixed
            // part; what rounding leaves over goes with the last tile
            const I tile = static_cast<I>(a.G) * BKV;
            auto cut = [&](I x) -> int {   // tiles before cost x of the item
                if (x >= cost) return p.nt;
                if (x <= s.fixed) return 0;
                return static_cast<int>(paged_min<I>(paged_div<I>(x - s.fixed, tile), p.nt));
            };
            const I from = begin - item, to = end - item;
            p.t0 = cut(from);
            p.t1 = cut(to);
            p.whole = p.t0 == 0 && p.t1 == p.nt && (p.nt > 0 || from <= 0);
            p.last = -1;
            const bool any = p.t1 > p.t0 || (p.nt == 0 && from <= 0);
            if (any && p.t0 == 0 && !p.whole)
                p.last = unit_of(item + paged_min<I>(s.fixed + p.nt * tile, cost) - 1);
            item += cost;
            if (++m == s.mt) {
                m = 0;
                if (++g == a.Hkv) {
                    g = 0;
                    do {
                        if (++b >= a.B) {
                            item = end;
                            break;
                        }
                        s = ahead;
                        if (b + 1 < a.B) ahead = paged_seq<ROWS, BKV, I>(a, b + 1);
                    } while (s.n == 0);
                }
            }
            if (any) return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------- parts in shared memory
// One warp walks the stretch and hands the parts to the other roles through a
// small ring, so that the walk's arithmetic and its registers are paid once.
enum : int32_t { kPartWhole = 0, kPartFirst = 1, kPartLater = 2 };
struct __align__(16) PagedItem {
    int32_t b, g;
    int32_t s0, n, kv;       // the sequence: first token, tokens, cached keys
    int32_t frow0, rows;     // folded rows of the query tile (rows == 0: no more parts)
    int32_t tv0, tv1;        // key tiles of this part
    int32_t kind;            // kPart*
    int32_t last;            // kPartFirst: the unit with the item's last part
    int32_t pad;
};
constexpr int kPagedItems = 4;
constexpr int kPagedLoadSleep = 60;    // ns between a load warp's looks at a full ring
struct PagedRing {
    PagedItem item[kPagedItems];
    uint64_t full[kPagedItems], empty[kPagedItems];
};
// The walking warp waits for the slowest role, which may be a whole part
// behind: that takes as long as the part does.  (So does the odd CTA's warp that
// passes its queries on.  All other waits end after kWaitLimitNs.)
constexpr uint64_t kPagedWalkLimitNs = 20000000000ull;

// By one thread; `takers` arrivals free an entry.
DG_DEVICE void paged_ring_init(PagedRing &ring, int takers)
{
    for (int e = 0; e < kPagedItems; ++e) {
        mbar_init(&ring.full[e], 1);
        mbar_init(&ring.empty[e], takers);
    }
}

// The walking warp (all lanes), for unit u of `units`.  It divides the work
// while the rest of the CTA sets up; `ready` returns once the ring may be used.
template <class Gm, class I, class Ready>
DG_DEVICE void paged_walk_in(const PagedArgs &a, int u, int units, PagedRing &ring, int where,
                             void *sums, Ready ready)
{
    const bool lead = (threadIdx.x & 31) == 0;
    PagedWalk<Gm::Rows, Gm::BKV, I> walk;
    PagedSeq<I> first{};
    I bound[kPagedBounds<Gm::Rows>];
    const PagedRange<I> range = paged_divide<Gm::Rows, Gm::BKV, I>(a, u, units, first, bound, sums);
    if (range.waves > 0 || range.end > range.begin) {
        // the load warps will want the pages of the first keys next
        const I key = range.waves > 0 ? 0
                                      : paged_div<I>(paged_max<I>(range.begin - range.item, first.fixed) -
                                                         first.fixed, a.G);
        const int page = static_cast<int>(key) / a.page_size + (static_cast<int>(threadIdx.x) & 31) * 32;
        if (page < a.max_pages)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                a.page_table + static_cast<int64_t>(range.b) * a.max_pages + page));
    }
    walk.start(a, range, first);
    auto unit_of = [&](I x) -> int { return paged_unit_of<Gm::Rows>(range, bound, x); };
    PagedPart p;
    bool more = walk.next(a, p, unit_of);
    ready();
    for (uint32_t k = 0;; ++k) {
        const int e = static_cast<int>(k % kPagedItems);
        const bool ok = mbar_wait_poll<false, 400>(&ring.empty[e], ((k / kPagedItems) & 1u) ^ 1u, a.ws,
                                                   where, kPagedWalkLimitNs);
        if (!__all_sync(0xFFFFFFFFu, ok)) return;
        if (lead) {
            PagedItem it{};
            if (more) {
                it.b = p.b;
                it.g = p.g;
                it.s0 = p.s0;
                it.n = p.n;
                it.kv = p.kv;
                it.frow0 = p.frow0;
                it.rows = p.rows;
                it.tv0 = p.lo + p.t0;
                it.tv1 = p.lo + p.t1;
                it.kind = p.whole ? kPartWhole : p.last >= 0 ? kPartFirst : kPartLater;
                it.last = p.last;
            }
            ring.item[e] = it;
            mbar_arrive(&ring.full[e]);
        }
        if (!more) return;
        more = walk.next(a, p, unit_of);
    }
}

template <class Gm, class Ready>
DG_DEVICE void paged_walk(const PagedArgs &a, int u, int units, PagedRing &ring, int where, void *sums,
                          Ready ready)
{
    if (a.small) paged_walk_in<Gm, int32_t>(a, u, units, ring, where, sums, ready);
    else paged_walk_in<Gm, int64_t>(a, u, units, ring, where, sums, ready);
}

// The k-th part, by every thread of a role's warp (or one thread alone, which
// then passes alone = true).  False: no more parts, or a wait ran out.
DG_DEVICE bool paged_take(const PagedArgs &a, PagedRing &ring, uint32_t k, PagedItem &it, bool alone,
                          int where)
{
    const int e = static_cast<int>(k % kPagedItems);
    bool ok = mbar_wait_poll(&ring.full[e], (k / kPagedItems) & 1u, a.ws, where);
    if (!alone) ok = __all_sync(0xFFFFFFFFu, ok);
    if (!ok) return false;
    it = ring.item[e];
    if (!alone) __syncwarp();
    if (alone || (threadIdx.x & 31) == 0) mbar_arrive(&ring.empty[e]);
    return it.rows > 0;
}

// Keys of key tile tv that exist, and its first key's place among all keys.
template <int BKV>
DG_DEVICE int paged_valid(const PagedItem &p, int tv)
{
    const int nkp = (p.kv + BKV - 1) / BKV;
    return min(BKV, tv < nkp ? p.kv - tv * BKV : p.n - (tv - nkp) * BKV);
}
template <int BKV>
DG_DEVICE int paged_key0(const PagedItem &p, int tv)
{
    const int nkp = (p.kv + BKV - 1) / BKV;
    return tv < nkp ? tv * BKV : p.kv + (tv - nkp) * BKV;
}

// K steps of 16 keys that the last tile of n keys is multiplied with V in.
DG_DEVICE int paged_steps(int n, int bkv)
{
    return ((n - 1) % bkv + 16) / 16;
}

// One ring's loads (K or V) over all parts.  The whole warp: lane l loads the
// box (page piece l / NA, 64-dim atom l % NA) of a tile; the page ids of 32
// pieces ahead are held one per lane, the next 32 already on their way.
template <class Gm, int NS>
__device__ __forceinline__ void paged_ring_producer(uint8_t *buf, uint64_t *full, uint64_t *empty,
                                                    const CUtensorMap *map_c,
                                                    const CUtensorMap *map_n, const PagedArgs &a,
                                                    PagedRing &ring, int where)
{
    const int lane = threadIdx.x & 31;
    const uint64_t pol = policy_evict_first();
    const int R = a.box_rows, per_tile = Gm::BKV / R, batch = 32 / per_tile;
    const int box = lane / Gm::NA, at = lane % Gm::NA;
    uint32_t armed = 0, armed_par = 0;
    uint32_t it = 0;
    bool ok = true;
    PagedItem p;
    for (uint32_t k = 0; ok && paged_take(a, ring, k, p, false, where + 2); ++k) {
        const int32_t *table = a.page_table + static_cast<int64_t>(p.b) * a.max_pages;
        const int nkp = (p.kv + Gm::BKV - 1) / Gm::BKV;
        auto fetch = [&](int tile) -> int32_t {   // page of piece `lane` from this tile on
            const int key = tile * Gm::BKV + lane * R;
            return key < p.kv && tile < p.tv1 ? __ldg(table + key / a.page_size) : 0;
        };
        int32_t pages = fetch(p.tv0), ahead = fetch(p.tv0 + batch);
        int in = 0;
        for (int tv = p.tv0; tv < p.tv1; ++tv, ++it, ++in) {
            if (in == batch) {
                in = 0;
                pages = ahead;
                ahead = fetch(tv + batch);
            }
            const int s = static_cast<int>(it % NS);
            const uint32_t use = it / NS;
            ok = mbar_wait_poll<false, kPagedLoadSleep>(&empty[s], (use & 1u) ^ 1u, a.ws, where);
            if (!__all_sync(0xFFFFFFFFu, ok)) {
                ok = false;
                break;
            }
            uint8_t *dst = buf + s * Gm::KVBytes;
            if (tv < nkp) {
                const int key0 = tv * Gm::BKV;
                const int boxes = (min(Gm::BKV, p.kv - key0) + R - 1) / R;
                int32_t page = __shfl_sync(0xFFFFFFFFu, pages, in * per_tile + min(box, per_tile - 1));
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(boxes * R * Gm::Dim * 2));
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
                                p.s0 + (tv - nkp) * Gm::BKV, pol);
            }
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | ((use & 1u) << s);
        }
    }
    // every copy has landed before the CTA leaves
    for (int s = 0; s < NS; ++s)
        if (armed >> s & 1u) mbar_wait(&full[s], armed_par >> s & 1u, a.ws, where + 1);
}

// 16 values of an output row as bf16, 32 bytes (wide: one aligned store, which
// fills a memory sector; else two).
DG_DEVICE void store_bf16x16(uint16_t *dst, const float (&v)[16], float f, bool wide)
{
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[2 * e] * f, v[2 * e + 1] * f);
        w[e] = *reinterpret_cast<const uint32_t *>(&h2);
    }
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Where a part keeps 4 values (dims c .. c + 3, c a multiple of 4) of a row:
// [slot][D / 4][slot_rows][4], so that the threads of a warp, which hold
// neighbouring rows, store and load neighbouring addresses.
DG_DEVICE float4 *part_at(const PagedArgs &a, int slot, int row, int c)
{
    return reinterpret_cast<float4 *>(a.part_o) +
           (static_cast<int64_t>(slot) * (a.D / 4) + c / 4) * a.slot_rows + row;
}

// Dims [c0, c1) of a row of O from TMEM: the output row (times f), or the part
// slot as it is.  All lanes of the warp; only live rows store.
template <int N>
DG_DEVICE bool paged_store_row(const PagedArgs &a, uint32_t tmem_row, int c0, bool live, bool whole,
                               uint16_t *row_out, float f, int slot, int row)
{
    bool finite = true;
#pragma unroll 1
    for (int c = c0; c < c0 + N; c += 32) {
        uint32_t o[32];
        tmem_ld32_nowait(tmem_row + c, o);
        tmem_wait_ld();
        if (!live) continue;
        if (a.checks) {
#pragma unroll
            for (int e = 0; e < 32; ++e) finite &= isfinite(__uint_as_float(o[e])) != 0;
        }
        if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[16 * h + e]);
                store_bf16x16(row_out + c + 16 * h, v, f, a.out_wide != 0);
            }
        } else {
            float4 *dst = part_at(a, slot, row, c);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
                dst[static_cast<int64_t>(e / 4) * a.slot_rows] =
                    make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
        }
    }
    return finite;
}

// ---------------------------------------------------------------- values hidden from some rows
// A key that a mask hides from a row gets the weight 0 there, and 0 times an
// infinity or a NaN in its values would be a NaN in a row that must not know of
// it.  Only tiles with a key that some row of the query tile sees and another
// does not (those on a causal or window border) can hold one that matters:
// where a row sees all or nothing of a key, the products are right as they are.
// In those tiles the softmax threads look at a key's values each; a key with a
// value that is not finite has its values set to zero before the product, and
// the epilogue adds it to the rows that do see it (paged_add_hidden).

// First and last position of a part's rows, and whether some of them see a key
// of tile tv that others do not.
struct PagedEdge {
    int pos0, pos1;
};
DG_DEVICE PagedEdge paged_edge(const PagedArgs &a, const PagedItem &p)
{
    const int base = a.has_new ? p.kv : p.kv - p.n;
    return {base + p.frow0 / a.G, base + (p.frow0 + p.rows - 1) / a.G};
}
DG_DEVICE bool paged_border(const PagedArgs &a, const PagedEdge &e, int key0, int valid)
{
    return a.causal && (key0 + valid - 1 > e.pos0 || (a.window > 0 && key0 <= e.pos1 - a.window));
}

// The tiles of a part that are not whole and seen by all of its rows, by their
// index in the part: the first `lo` and those from `hi` on (borders), and the last
// of the pages and of the new tokens where it is not full (-1: none here).
struct PagedSpecial {
    int lo, hi, kv, fresh;
    DG_DEVICE bool at(int j) const { return j < lo || j >= hi || j == kv || j == fresh; }
    // Calls f with every such tile before tile `end`.
    template <class F>
    DG_DEVICE void each(int end, F f) const
    {
        for (int j = 0; j < min(lo, end); ++j) f(j);
        if (kv >= 0 && kv < end && kv >= lo && kv < hi) f(kv);
        if (fresh >= 0 && fresh < end && fresh >= lo && fresh < hi) f(fresh);
        for (int j = max(lo, hi); j < end; ++j) f(j);
    }
};
template <int BKV>
DG_DEVICE PagedSpecial paged_special(const PagedArgs &a, const PagedItem &p, const PagedEdge &e)
{
    const int nt = p.tv1 - p.tv0, nkp = (p.kv + BKV - 1) / BKV;
    PagedSpecial s;
    s.lo = 0;
    s.hi = nt;
    if (a.causal) {
        // what is hidden lies within a query tile's positions of either end
        if (a.window > 0)
            while (s.lo < nt && paged_key0<BKV>(p, p.tv0 + s.lo) <= e.pos1 - a.window) ++s.lo;
        while (s.hi > s.lo && paged_key0<BKV>(p, p.tv0 + s.hi - 1) +
                                      paged_valid<BKV>(p, p.tv0 + s.hi - 1) - 1 > e.pos0)
            --s.hi;
    }
    s.kv = p.kv % BKV ? nkp - 1 - p.tv0 : -1;
    s.fresh = a.has_new && p.n % BKV ? nkp + (p.n - 1) / BKV - p.tv0 : -1;
    if (s.kv >= nt) s.kv = -1;
    if (s.fresh >= nt) s.fresh = -1;
    return s;
}

// Whether any of 2 N bf16 values is infinite or NaN: the largest magnitude as
// integers.
DG_DEVICE uint32_t magnitude_max(uint32_t m, const uint4 &v)
{
    m = __vmaxu2(m, v.x & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.y & 0x7FFF7FFFu);
    m = __vmaxu2(m, v.z & 0x7FFF7FFFu);
    return __vmaxu2(m, v.w & 0x7FFF7FFFu);
}
DG_DEVICE bool not_finite(uint32_t m) { return (m & 0xFFFFu) >= 0x7F80u || (m >> 16) >= 0x7F80u; }

// Thread t's key of a landed V tile: true, and its values zeroed, if one of
// them is not finite.
template <class Gm>
DG_DEVICE bool paged_look(uint8_t *v_tile, int valid, int t)
{
    if (t >= valid) return false;
    uint32_t m = 0;
#pragma unroll
    for (int at = 0; at < Gm::NA; ++at) {
        const uint4 *row = reinterpret_cast<const uint4 *>(v_tile + at * Gm::KVAtomBytes + t * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) m = magnitude_max(m, row[(c + t) & 7]);   // (each piece; spread over banks)
    }
    if (!not_finite(m)) return false;
    for (int at = 0; at < Gm::NA; ++at)
        for (int c = 0; c < 8; ++c)
            reinterpret_cast<uint4 *>(v_tile + at * Gm::KVAtomBytes + t * 128)[c] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    return true;
}

// Where a part's key is: its offset in the pages or, from tile nkp on, among the
// new tokens (k, v: the arrays' own strides); false: its page does not exist.
struct PagedKey {
    const uint16_t *k, *v;
};
DG_DEVICE bool paged_key(const PagedArgs &a, const PagedItem &p, bool fresh, int key, PagedKey &at)
{
    if (fresh) {
        const int64_t row = p.s0 + key - p.kv;
        at = PagedKey{a.k_new + row * a.k_stride + p.g * a.D, a.v_new + row * a.v_stride + p.g * a.D};
        return true;
    }
    const int page = a.page_table[static_cast<int64_t>(p.b) * a.max_pages + key / a.page_size];
    if (page < 0 || page >= a.n_pages) return false;
    const int64_t off = page * a.page_stride +
                        static_cast<int64_t>(key % a.page_size) * a.Hkv * a.D + p.g * a.D;
    at = PagedKey{a.k_pages + off, a.v_pages + off};
    return true;
}
// The weight of a key for the row at q_off, whose reference is m_ref.
DG_DEVICE float paged_weight(const PagedArgs &a, const uint16_t *k, int64_t q_off, float m_ref)
{
    float s = 0.f;
#pragma unroll 1
    for (int d = 0; d < a.D; ++d)
        s = fmaf(__uint_as_float(static_cast<uint32_t>(a.q[q_off + d]) << 16),
                 __uint_as_float(static_cast<uint32_t>(k[d]) << 16), s);
    return fast_exp2(fmaf(s, a.scale_log2, -m_ref));
}
DG_DEVICE bool paged_sees(const PagedArgs &a, int pos, int key)
{
    return (!a.causal || key <= pos) && (a.window == 0 || key > pos - a.window);
}

// Adds to a row of O (dims [c0, c0 + N), in TMEM, with reference m_ref) the keys
// that paged_look zeroed and the row sees, those in columns [first, end) of their
// tiles.  The whole warp, lane = row (live: it exists); nothing here is fast, nor
// need it be.
template <int BKV, int N>
DG_DEVICE void paged_add_hidden(const PagedArgs &a, const PagedItem &p, uint32_t tmem_row, int c0,
                                bool live, int64_t q_off, int pos, float m_ref, int first = 0,
                                int end = BKV)
{
    const PagedEdge e = paged_edge(a, p);
    const int nkp = (p.kv + BKV - 1) / BKV;
#pragma unroll 1
    for (int tv = p.tv0; tv < p.tv1; ++tv) {
        const int valid = paged_valid<BKV>(p, tv), key0 = paged_key0<BKV>(p, tv);
        if (!paged_border(a, e, key0, valid)) continue;
#pragma unroll 1
        for (int c = first; c < min(valid, end); ++c) {
            PagedKey at;
            if (!paged_key(a, p, tv >= nkp, key0 + c, at)) continue;
            const uint16_t *v = at.v + c0;
            uint32_t m = 0;
#pragma unroll 1
            for (int d = 0; d < N; d += 8) m = magnitude_max(m, *reinterpret_cast<const uint4 *>(v + d));
            if (!not_finite(m)) continue;
            const bool sees = live && paged_sees(a, pos, key0 + c);
            const float w = sees ? paged_weight(a, at.k, q_off, m_ref) : 0.f;
#pragma unroll 1
            for (int d = 0; d < N; d += 16) {
                uint32_t o[16];
                tmem_ld16_issue(tmem_row + c0 + d, o);
                tmem_wait_ld16(o);
                if (sees) {
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        o[x] = __float_as_uint(
                            fmaf(w, __uint_as_float(static_cast<uint32_t>(v[d + x]) << 16),
                                 __uint_as_float(o[x])));
                }
                tmem_st16(tmem_row + c0 + d, o);
                tmem_wait_st();
            }
        }
    }
}

// Which of N dims (from c0 on; a bit each) have an infinity of either sign, or a
// NaN, in the value of a key of this part that token i of its rows sees.  A
// softmax's weights are positive, so that is all that such values bring to a sum;
// a key that is not finite itself has a score that is not, and makes NaN of them.
struct PagedMarks {
    uint64_t pos, neg, nan;
};
// The whole warp, a key a lane, so that a cache full of them (a sequence whose
// values have overflowed) does not hold up the other sequences: 2000 such keys of 16
// heads of 128 took 57 ms with each lane by itself and their weights worked out, so
// that 40000 outlasted the other warps' waits; they take 0.7.
template <int BKV, int N>
__device__ __noinline__ PagedMarks paged_marks(const PagedArgs &a, const PagedItem &p, int i, int c0)
{
    PagedMarks m{0, 0, 0};
    const int lane = threadIdx.x & 31;
    const int nkp = (p.kv + BKV - 1) / BKV;
    const int pos = (a.has_new ? p.kv : p.kv - p.n) + i;
#pragma unroll 1
    for (int tv = p.tv0; tv < p.tv1; ++tv) {
        const int valid = paged_valid<BKV>(p, tv), key0 = paged_key0<BKV>(p, tv);
#pragma unroll 1
        for (int c = lane; c < valid; c += 32) {
            PagedKey at;
            if (!paged_sees(a, pos, key0 + c) || !paged_key(a, p, tv >= nkp, key0 + c, at)) continue;
            uint32_t v = 0, k = 0;
#pragma unroll
            for (int d = 0; d < N; d += 8) v = magnitude_max(v, *reinterpret_cast<const uint4 *>(at.v + c0 + d));
            if (!not_finite(v)) continue;
#pragma unroll 1
            for (int d = 0; d < a.D; d += 8) k = magnitude_max(k, *reinterpret_cast<const uint4 *>(at.k + d));
            const bool no_weight = not_finite(k);
#pragma unroll 1
            for (int d = 0; d < N; ++d) {
                const uint32_t x = at.v[c0 + d];
                if ((x & 0x7F80u) != 0x7F80u) continue;
                const uint64_t bit = 1ull << d;
                if (no_weight || (x & 0x7Fu)) m.nan |= bit;
                else if (x >> 15) m.neg |= bit;
                else m.pos |= bit;
            }
        }
    }
    auto any = [](uint64_t x) -> uint64_t {
        return static_cast<uint64_t>(__reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(x >> 32))) << 32 |
               __reduce_or_sync(0xFFFFFFFFu, static_cast<uint32_t>(x));
    };
    m.pos = any(m.pos);
    m.neg = any(m.neg);
    m.nan = any(m.nan);
    return m;
}
// The sum's value in dim d (of those marked): else x.
DG_DEVICE float paged_marked(const PagedMarks &m, int d, float x)
{
    const bool pos = m.pos >> d & 1u, neg = m.neg >> d & 1u;
    if ((m.nan >> d & 1u) || (pos && neg)) return __int_as_float(0x7FC00000);
    return pos ? INFINITY : neg ? -INFINITY : x;
}

// The rows of a V tile between its last key and the next multiple of 16, up
// to which it is multiplied: zero, whatever the page holds there.  By the 128
// threads of a softmax group (t = 0 .. 127), after the tile has landed.
template <class Gm>
DG_DEVICE void paged_zero_tail(uint8_t *v_tile, int valid, int t)
{
    const int chunks = (((valid + 15) & ~15) - valid) * 8;   // 16-byte pieces of a 64-dim atom
    for (int c = t; c < chunks * Gm::NA; c += 128)
        *reinterpret_cast<uint4 *>(v_tile + c / chunks * Gm::KVAtomBytes + valid * 128 +
                                   c % chunks * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
}

}  // namespace dg
