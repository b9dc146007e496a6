"""The division of the paged attention's work (csrc/dg_paged.cuh), run on the
host: over ragged batches, masks and CTA counts, every visible key tile of
every query tile is given to exactly one CTA, every row a CTA may leave in a
part slot has that slot to itself, and the last part named by an item's first
one is the part that holds its last key tile.  Lengths outside the tensors
are cut to them."""
import os
import random
import re
import subprocess

import pytest

from block_diffusion_decoding_gb300 import build as dgbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>
#include "dg_paged.cuh"
using namespace dg;
static long wholes = 0, rounds_n = 0;
static double worst = 0;

#define FAIL(...) do { printf(__VA_ARGS__); printf("\n"); return 1; } while (0)

template <int ROWS, int BKV, class I>
int check(const PagedArgs &a, int units)
{
    std::vector<I> base(a.B + 1, 0);
    I items_n = 0, most = 0;
    bool whole = false;
    for (int b = 0; b < a.B; ++b) {
        const PagedSeq<I> s = paged_seq<ROWS, BKV, I>(a, b);
        if (s.s0 < 0 || s.n < 0 || s.s0 + s.n > a.T || s.kv < 0 || s.kv > a.max_pages * a.page_size)
            FAIL("lengths not cut");
        base[b + 1] = base[b] + a.Hkv * paged_prefix(s, s.mt);
        items_n += a.Hkv * s.mt;
        for (int m = 0; m < s.mt; ++m) {
            const I c = paged_prefix(s, m + 1) - paged_prefix(s, m);
            if (c > most) most = c;
        }
    }
    const I W = base[a.B];
    if (W == 0) return 0;
    whole = paged_whole<ROWS>(a, W, items_n, most, units);
    const I step = paged_step<ROWS>(a, W, units);
    int n = units;
    std::vector<I> bound(units + 1, W), sum(units, 0);
    int waves = 0;
    if (whole) {
        ++wholes;
    } else {
        n = static_cast<int>((W + step - 1) / step);
        if (n > units) FAIL("%d units of %d", n, units);
        waves = paged_rounds<ROWS>(a, items_n, units);
        if (waves) {
            I i = 0, taken = 0, dearest = 0;
            for (int b = 0; b < a.B; ++b) {
                const PagedSeq<I> s = paged_seq<ROWS, BKV, I>(a, b);
                for (int e = 0; e < a.Hkv * s.mt; ++e, ++i)
                    if (i < static_cast<I>(waves) * units)
                        sum[i % units] += paged_prefix(s, e % s.mt + 1) - paged_prefix(s, e % s.mt);
            }
            for (I x : sum) taken += x, dearest = x > dearest ? x : dearest;
            if (!paged_even(W, units, dearest)) {
                waves = 0;
            } else {
                ++rounds_n;
                n = units;
                const I share = (W + units - 1) / units;
                I at = taken;
                for (int u = 0; u < units; ++u) {
                    bound[u] = at < W ? at : W;
                    at += share > sum[u] ? share - sum[u] : 0;
                    const double cost = static_cast<double>(sum[u] + (at < W ? at : W) - bound[u]) / share;
                    if (cost > worst) worst = cost;
                }
                if (at < W) FAIL("the line is not given out");
            }
        }
    }
    auto unit_of = [&](I x) -> int {
        if (!waves) return static_cast<int>(x / step);
        int k = 0;
        while (k < units && bound[k] <= x) ++k;
        return k - 1;
    };
    // per item: the tiles so far, the unit promised the last part
    std::map<std::tuple<int, int, int>, std::pair<int, int>> items;
    for (int u = 0; u < n; ++u) {
        PagedRange<I> r{};
        r.units = units;
        PagedSeq<I> first{};
        r.waves = waves;
        if (whole) {
            r.waves = u < items_n ? static_cast<int>((items_n - u + units - 1) / units) : 0;
        } else {
            r.begin = waves ? bound[u] : u * step;
            r.end = waves ? bound[u + 1] : r.begin + step < W ? r.begin + step : W;
            r.step = waves ? 0 : step;
        }
        if (r.waves) {
            I i = u;
            for (;; ++r.b) {
                first = paged_seq<ROWS, BKV, I>(a, r.b);
                if (i < a.Hkv * first.mt) break;
                i -= a.Hkv * first.mt;
            }
            r.at = i;
        } else if (r.begin < r.end) {
            while (base[r.b + 1] <= r.begin) ++r.b;
            first = paged_seq<ROWS, BKV, I>(a, r.b);
            paged_locate(first, r.b, base[r.b], r.begin, r);
        }
        PagedWalk<ROWS, BKV, I> walk;
        walk.start(a, r, first);
        PagedPart p;
        int slot0 = 0, slot1 = 0;
        while (walk.next(a, p, unit_of)) {
            // the definition, from the lengths alone
            int lo = 1 << 30, hi = 0;
            const int keys = p.kv + (a.has_new ? p.n : 0);
            for (int row = p.frow0; row < p.frow0 + p.rows; ++row) {
                const int pos = keys - p.n + row / a.G;
                const int last = a.causal ? pos : keys - 1;
                const int first = a.window ? (pos - a.window + 1 > 0 ? pos - a.window + 1 : 0) : 0;
                if (last < first) continue;
                auto tile = [&](int key) {
                    return key < p.kv ? key / BKV : p.nkp + (key - p.kv) / BKV;
                };
                if (tile(first) < lo) lo = tile(first);
                if (tile(last) + 1 > hi) hi = tile(last) + 1;
            }
            const int want = hi > lo ? hi - lo : 0;
            if (p.nt < want || (want && (p.lo > lo || p.lo + p.nt < hi))) FAIL("a visible tile is missing");
            if (p.nt > want + 1) FAIL("tiles nobody sees: %d of %d", p.nt - want, p.nt);
            if (p.t0 < 0 || p.t1 > p.nt || (p.t0 >= p.t1 && p.nt)) FAIL("bad part");
            auto it = items.emplace(std::make_tuple(p.b, p.g, p.frow0), std::make_pair(0, -1)).first;
            if (it->second.first != p.t0) FAIL("tiles not in order");
            if (p.t0 == 0 && it->second.second != -1) FAIL("an item twice");
            if (p.whole) {
                if (p.t0 != 0 || p.t1 != p.nt || p.last != -1) FAIL("whole");
                it->second = {p.nt, u};
            } else if (p.t0 == 0) {
                if (p.last <= u || p.last >= n) FAIL("last %d of %d", p.last, u);
                if (++slot1 > 1) FAIL("slot 1 twice");
                it->second = {p.t1, p.last};
            } else {
                if (p.last != -1) FAIL("last");
                if (++slot0 > 1) FAIL("slot 0 twice");
                if (u > it->second.second) FAIL("after the last part");
                if (p.t1 == p.nt && u != it->second.second) FAIL("the last part is %d's", u);
                it->second.first = p.t1;
            }
            if (p.t1 == p.nt) it->second.first = p.nt;
            if (p.rows < 1 || p.rows > ROWS) FAIL("rows");
            if (whole && !p.whole) FAIL("a whole item cut");
        }
    }
    for (int b = 0; b < a.B; ++b) {
        const PagedSeq<I> s = paged_seq<ROWS, BKV, I>(a, b);
        for (int g = 0; g < a.Hkv; ++g)
            for (int m = 0; m < s.mt; ++m)
                if (!items.count(std::make_tuple(b, g, m * ROWS))) FAIL("item (%d %d %d) missing", b, g, m);
    }
    return 0;
}

int main()
{
    int T, B, Hkv, G, page, width, fresh, causal, window, units, bkv, rows;
    long line = 0, small = 0;
    while (scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &T, &B, &Hkv, &G, &page, &width, &fresh, &causal,
                 &window, &units, &bkv, &rows) == 12) {
        std::vector<int32_t> start(B + 1), kv(B);
        for (auto &x : start) if (scanf("%d", &x) != 1) return 2;
        for (auto &x : kv) if (scanf("%d", &x) != 1) return 2;
        PagedArgs a{};
        a.T = T; a.B = B; a.Hkv = Hkv; a.G = G; a.page_size = page; a.max_pages = width;
        a.has_new = fresh; a.causal = causal; a.window = window;
        a.q_start = start.data(); a.kv_len = kv.data();
        int rc = rows == 256 ? check<256, 128, int64_t>(a, units)
                 : bkv == 128 ? check<128, 128, int64_t>(a, units) : check<128, 64, int64_t>(a, units);
        if (!rc && paged_small(T, B, Hkv, G, static_cast<int64_t>(width) * page)) {
            rc = rows == 256 ? check<256, 128, int32_t>(a, units)
                 : bkv == 128 ? check<128, 128, int32_t>(a, units) : check<128, 64, int32_t>(a, units);
            ++small;
        }
        if (rc) { printf("case %ld\n", line); return 1; }
        ++line;
    }
    printf("%ld cases, %ld of them also in 32 bits, %ld divisions left whole, %ld in rounds, %.0f at most\n", line, small,
           wholes, rounds_n, 1000 * worst);
    return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_division")
    src = d / "harness.cu"
    src.write_text(HARNESS)
    exe = str(d / "harness")
    r = subprocess.run([dgbuild.nvcc(), *dgbuild.ARCH, "-O1", "-std=c++17", "-I", dgbuild.CSRC, "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def _case(rng):
    B = rng.choice([1, 1, 2, 3, 7, 40, 300])
    top = 1 if rng.random() < 0.3 else rng.choice([3, 130, 900])
    n = [0 if rng.random() < 0.15 else rng.randint(1, top) for _ in range(B)]
    most = rng.choice([1, 60, 1000, 9000])
    causal = rng.random() < 0.6
    fresh = rng.random() < 0.5
    kv = [0 if rng.random() < 0.1 else rng.randint(0, most) for _ in range(B)]
    if causal and not fresh and rng.random() < 0.8:
        kv = [k + m for k, m in zip(kv, n)]
    start = [0]
    for m in n:
        start.append(start[-1] + m)
    T = start[-1] + rng.choice([0, 0, 5])
    page = rng.choice([16, 48, 64, 128])
    width = max(1, -(-max(kv) // page) + rng.choice([0, 3]))
    if rng.random() < 0.15:     # lengths that do not fit the tensors
        kv[rng.randrange(B)] = rng.choice([-5, 10 ** 9])
        start[rng.randrange(B + 1)] = rng.choice([-3, 10 ** 6, 0])
    window = rng.choice([0, 0, 1, 5, 64, 1024]) if causal else 0
    bkv, rows = rng.choice([(128, 128), (64, 128), (128, 256)])
    head = [T, B, rng.choice([1, 2, 8]), rng.choice([1, 2, 3, 4, 7, 16, 128]), page, width, int(fresh),
            int(causal), window, rng.choice([1, 2, 76, 152]), bkv, rows]
    return head + start + kv


def test_every_visible_tile_goes_to_one_cta(harness):
    rng = random.Random(11)
    cases = [_case(rng) for _ in range(1500)]
    text = "\n".join(" ".join(map(str, c)) for c in cases) + "\n"
    r = subprocess.run([harness], input=text, capture_output=True, text=True, timeout=600)
    where = int(r.stdout.split()[-1]) if "case " in r.stdout and r.returncode else None
    assert r.returncode == 0, (r.stdout[-300:], cases[where][:12] if where is not None else r.stderr[-300:])
    assert "1500 cases" in r.stdout
    # both integer widths, and both ways of dividing, are among them
    cases_, small, wholes, rounds, worst = (int(x) for x in re.findall(r"(\d+) (?:cases|of them|divisions|in|at)", r.stdout))
    assert 500 < small < 1500 and 200 < wholes < cases_ + small - 200 and rounds > 50, r.stdout
    # whole items first leave no unit with more than a sixteenth above its share (in thousandths)
    assert 900 < worst <= 1063, r.stdout
