// dg_paged.cuh -- how the paged attention kernels divide their work.
//
// The lengths of the sequences are device data, so the division is made on
// the device, by every CTA for itself, from the lengths alone.  An item is
// one query tile (ROWS folded rows = positions x heads of one kv head) of one
// kv head of one sequence; it costs a fixed part plus its visible keys.  The
// items in the order (sequence, kv head, query tile) lie end to end on a line
// of total cost W, CTA c takes the stretch [W c / n, W (c + 1) / n), and a cut
// inside an item falls between two of its key tiles.  So the CTAs' work is
// equal whatever the lengths are, a CTA leaves at most two unfinished parts
// (one at each end of its stretch), and the parts of an item are those of
// consecutive CTAs: they are merged in that order, whoever was first.
#pragma once

#include "dg_kernels.h"

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

constexpr int kPagedItemKeys = 256;    // an item's fixed cost, in keys
constexpr int kPagedMinKeys = 512;     // least cost of a CTA's stretch, in keys

struct PagedSeq {
    int s0, n, kv;      // first token, tokens, cached keys
    int mt;             // query tiles of a kv head
    int mc;             // tiles whose key count still grows with the tile index
    int64_t x0, slope, cap, fixed;
};

// Bounds every length by what the tensors hold, so that no later index can
// leave them; *bad is set when something had to be cut.
template <int ROWS, int BKV>
DG_BOTH PagedSeq paged_seq(const PagedArgs &a, int b, bool *bad = nullptr)
{
    PagedSeq s;
    const int r0 = paged_load(a.q_start + b), r1 = paged_load(a.q_start + b + 1);
    const int k0 = paged_load(a.kv_len + b);
    s.s0 = paged_min(paged_max(r0, 0), a.T);
    s.n = paged_min(paged_max(r1, s.s0), a.T) - s.s0;
    s.kv = paged_min(paged_max(k0, 0), a.max_pages * a.page_size);
    if (bad != nullptr) *bad = r0 != s.s0 || r1 != s.s0 + s.n || k0 != s.kv;
    s.mt = (s.n * a.G + ROWS - 1) / ROWS;
    const int64_t G = a.G;
    s.fixed = G * kPagedItemKeys + 1;
    s.cap = INT64_MAX / 4;
    if (!a.causal) {
        s.slope = 0;
        s.x0 = G * (static_cast<int64_t>(s.kv) + (a.has_new ? s.n : 0));
        s.mc = s.mt;
    } else {
        s.slope = ROWS;
        s.x0 = G * paged_max(0, a.has_new ? s.kv : s.kv - s.n);
        s.mc = s.mt;
        if (a.window > 0) {
            s.cap = G * (static_cast<int64_t>(a.window) + BKV) + ROWS;
            const int64_t k = s.cap < s.x0 ? 0 : (s.cap - s.x0) / ROWS;
            s.mc = static_cast<int>(paged_min(k, static_cast<int64_t>(s.mt)));
        }
    }
    return s;
}

// Cost of the first m query tiles of one kv head.
DG_BOTH int64_t paged_prefix(const PagedSeq &s, int m)
{
    const int64_t k = paged_min(m, s.mc);
    return m * s.fixed + k * s.x0 + s.slope * (k * (k + 1) / 2) + (m - k) * s.cap;
}

struct PagedRange {
    int64_t W, begin, end;   // the whole line, this CTA's stretch
    int n;                   // CTAs that have one
    int b;                   // sequence `begin` falls in
    int64_t base;            // where that sequence begins
};

DG_BOTH int64_t paged_bound(int64_t W, int n, int c)
{
    return W / n * c + W % n * c / n;
}

// The CTA whose stretch holds position x.
DG_BOTH int paged_owner(int64_t W, int n, int64_t x)
{
    int c = static_cast<int>(static_cast<float>(x) / static_cast<float>(W) * n);
    c = paged_min(paged_max(c, 0), n - 1);
    while (paged_bound(W, n, c) > x) --c;
    while (paged_bound(W, n, c + 1) <= x) ++c;
    return c;
}

// Units (CTAs, or pairs of them) that get a stretch of a line of cost W.
DG_BOTH int paged_units(const PagedArgs &a, int64_t W, int units)
{
    const int64_t least = static_cast<int64_t>(a.G) * kPagedMinKeys;
    return static_cast<int>(paged_min<int64_t>(units, paged_max<int64_t>(W / least, 1)));
}

struct PagedScan {
    int64_t warp_sum[32];
    PagedRange r;
};

// Unit u of `units` (a CTA, or a pair) of NT threads: its stretch, left in
// sc.r (end <= begin: nothing to do).  All threads of the CTA call it.
template <int ROWS, int BKV, int NT>
DG_DEVICE void paged_divide(const PagedArgs &a, int u, int units, PagedScan &sc)
{
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ch = (a.B + NT - 1) / NT;
    const int b0 = min(a.B, tid * ch), b1 = min(a.B, b0 + ch);
    int64_t mine = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        bool cut;
        const PagedSeq s = paged_seq<ROWS, BKV>(a, b, &cut);
        bad |= cut;
        mine += a.Hkv * paged_prefix(s, s.mt);
    }
    if (bad && u == 0) report_error(a.ws, DG_ERR_DEVICE, 911);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sc.warp_sum[warp] = incl;
    if (tid == 0) sc.r.begin = sc.r.end = 0;
    __syncthreads();
    int64_t W = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += sc.warp_sum[w];
        W += sc.warp_sum[w];
    }
    const int n = paged_units(a, W, units);
    if (W > 0 && u < n) {
        const int64_t x = paged_bound(W, n, u);
        if (x >= before && x < before + mine) {
            int64_t base = before;
            for (int b = b0; b < b1; ++b) {
                const PagedSeq s = paged_seq<ROWS, BKV>(a, b);
                const int64_t c = a.Hkv * paged_prefix(s, s.mt);
                if (x < base + c) {
                    sc.r.W = W;
                    sc.r.n = n;
                    sc.r.begin = x;
                    sc.r.end = paged_bound(W, n, u + 1);
                    sc.r.b = b;
                    sc.r.base = base;
                    break;
                }
                base += c;
            }
        }
    }
    __syncthreads();
}

// One stretch's share of an item.
struct PagedPart {
    PagedSeq s;
    int b, g;
    int frow0, rows;     // folded rows of the query tile
    int nkp;             // key tiles of the pages (further ones: the chunk's own keys)
    int lo;              // first visible key tile
    int t0, t1;          // this part's tiles, from lo
    int nt;              // the item's
    int last;            // first part of several: the unit with the last one, else -1
    bool whole;
};

// Walks the parts of a stretch.  Every role of the CTA walks its own copy, all
// the same.
template <int ROWS, int BKV>
struct PagedWalk {
    PagedSeq s, ahead;   // this sequence, the next one's lengths (already loaded)
    int b, g, m;
    int64_t item, begin, end, W;
    int n;

    DG_BOTH void start(const PagedArgs &a, const PagedRange &r)
    {
        begin = r.begin;
        item = end = r.end;
        if (end <= begin) return;
        W = r.W;
        n = r.n;
        b = r.b;
        s = paged_seq<ROWS, BKV>(a, b);
        ahead = s;
        if (b + 1 < a.B) ahead = paged_seq<ROWS, BKV>(a, b + 1);
        const int64_t head = paged_prefix(s, s.mt);
        int64_t y = begin - r.base;
        g = static_cast<int>(y / head);
        y -= g * head;
        int lo = 0, hi = s.mt - 1;   // the last tile that begins at or before y
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (paged_prefix(s, mid) <= y) lo = mid;
            else hi = mid - 1;
        }
        m = lo;
        item = r.base + g * head + paged_prefix(s, m);
    }

    // The next part; false: the stretch is done.
    DG_BOTH bool next(const PagedArgs &a, PagedPart &p)
    {
        while (item < end) {
            const int64_t cost = paged_prefix(s, m + 1) - paged_prefix(s, m);
            p.s = s;
            p.b = b;
            p.g = g;
            p.frow0 = m * ROWS;
            p.rows = paged_min(ROWS, s.n * a.G - p.frow0);
            const int i0 = p.frow0 / a.G, i1 = (p.frow0 + p.rows - 1) / a.G;
            p.nkp = (s.kv + BKV - 1) / BKV;
            int hi, lo = 0;
            if (!a.causal)
                hi = p.nkp + (a.has_new ? (s.n + BKV - 1) / BKV : 0);
            else if (a.has_new)
                hi = p.nkp + i1 / BKV + 1;
            else
                hi = paged_max(0, (s.kv - s.n + i1 + BKV) / BKV);
            if (a.window > 0) {
                const int first = (a.has_new ? s.kv : s.kv - s.n) + i0 - a.window + 1;
                if (first > 0)
                    lo = a.has_new && first >= s.kv ? p.nkp + (first - s.kv) / BKV : first / BKV;
            }
            p.lo = lo;
            p.nt = paged_max(0, hi - lo);
            const int64_t span = cost - s.fixed;
            auto cut = [&](int64_t x) -> int {   // tiles before cost x of the item
                if (x <= s.fixed) return 0;
                if (x >= cost) return p.nt;
                return static_cast<int>((x - s.fixed) * p.nt / span);
            };
            const int64_t from = begin - item, to = end - item;
            p.t0 = cut(from);
            p.t1 = cut(to);
            p.whole = p.t0 == 0 && p.t1 == p.nt && (p.nt > 0 || from <= 0);
            p.last = -1;
            const bool any = p.t1 > p.t0 || (p.nt == 0 && from <= 0);
            if (any && p.t0 == 0 && !p.whole) p.last = paged_owner(W, n, item + cost - 1);
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
                        if (b + 1 < a.B) ahead = paged_seq<ROWS, BKV>(a, b + 1);
                    } while (s.n == 0);
                }
            }
            if (any) return true;
        }
        return false;
    }
};

}  // namespace dg
