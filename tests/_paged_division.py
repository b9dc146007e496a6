"""A program that divides ragged batches' paged attention work by csrc/dg_paged.cuh and checks that the parts are
all of it: on the host (walk alone, with the division's sums done over) or on the device (as the kernels do)."""
import os
import subprocess

from block_diffusion_decoding_gb300 import build as dgbuild

SOURCE = r"""
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <map>
#include <tuple>
#include <vector>
#include "dg_paged.cuh"
using namespace dg;

#define FAIL(...) do { printf(__VA_ARGS__); printf("\n"); return 1; } while (0)
#define CUDA(x) do { cudaError_t e_ = (x); if (e_ != cudaSuccess) { printf("%s\n", cudaGetErrorString(e_)); exit(3); } } while (0)
static long rounds_n = 0, cut_n = 0;

struct Given { PagedPart p; int unit, at; };   // a part, its unit, its place among the unit's

// what the parts have to be, from the lengths alone
template <int ROWS, int BKV, class I>
int check(const PagedArgs &a, int units, std::vector<Given> &parts)
{
    std::sort(parts.begin(), parts.end(), [](const Given &x, const Given &y) {
        return std::make_pair(x.unit, x.at) < std::make_pair(y.unit, y.at);
    });
    struct Item { int nt = -1, tiles = 0, last = -1, end = -1, n = 0; };
    std::map<std::tuple<int, int, int>, Item> items;
    std::vector<int> slot0(units, 0), slot1(units, 0);
    for (const Given &x : parts) {
        const PagedPart &p = x.p;
        if (x.unit < 0 || x.unit >= units) FAIL("unit %d", x.unit);
        if (p.rows < 1 || p.rows > ROWS || p.t0 < 0 || p.t1 > p.nt || (p.nt && p.t0 >= p.t1)) FAIL("bad part");
        Item &it = items[std::make_tuple(p.b, p.g, p.frow0)];
        if (it.n++ == 0) it.nt = p.nt;
        if (it.nt != p.nt) FAIL("the parts differ on their item");
        if (it.tiles != p.t0) FAIL("tile %d after %d", p.t0, it.tiles);
        it.tiles = p.t1;
        if (p.whole) {
            if (it.n > 1 || p.t1 != p.nt || p.last != -1) FAIL("not whole");
            it.end = it.last = x.unit;
        } else if (p.t0 == 0) {
            if (it.n > 1 || p.t1 == p.nt || p.last <= x.unit || p.last >= units || ++slot1[x.unit] > 1) FAIL("first part");
            it.last = p.last;
        } else {
            if (it.n < 2 || p.last != -1 || ++slot0[x.unit] > 1) FAIL("later part");
            if (p.t1 == p.nt) it.end = x.unit;
        }
    }
    size_t n = 0;
    for (int b = 0; b < a.B; ++b) {
        const PagedSeq<I> s = paged_seq<ROWS, BKV, I>(a, b);
        n += static_cast<size_t>(a.Hkv) * s.mt;
        for (int g = 0; g < a.Hkv; ++g)
            for (int m = 0; m < s.mt; ++m) {
                auto f = items.find(std::make_tuple(b, g, m * ROWS));
                if (f == items.end()) FAIL("item (%d %d %d) missing", b, g, m);
                const Item &it = f->second;
                // the tiles that hold a key that one of the rows sees
                const int frow0 = m * ROWS, rows = std::min(ROWS, s.n * a.G - frow0);
                const int keys = s.kv + (a.has_new ? s.n : 0), nkp = (s.kv + BKV - 1) / BKV;
                auto tile = [&](int key) { return key < s.kv ? key / BKV : nkp + (key - s.kv) / BKV; };
                int lo = 1 << 30, hi = 0;
                for (int i = frow0 / a.G; i <= (frow0 + rows - 1) / a.G; ++i) {
                    const int pos = keys - s.n + i, last = a.causal ? pos : keys - 1;
                    const int first = a.window ? std::max(0, pos - a.window + 1) : 0;
                    if (last < first) continue;
                    lo = std::min(lo, tile(first));
                    hi = std::max(hi, tile(last) + 1);
                }
                if (it.nt < (hi > lo ? hi - lo : 0)) FAIL("a visible tile is in no part's count");
                if (it.tiles != it.nt) FAIL("tiles %d of %d", it.tiles, it.nt);
                if (it.end < 0 || it.end != it.last) FAIL("the last part is %d's, promised to %d", it.end, it.last);
                cut_n += it.n > 1;
            }
    }
    if (items.size() != n) FAIL("%zu items of %zu", items.size(), n);
    return 0;
}

template <int ROWS, int BKV, class I>
int on_host(const PagedArgs &a, int units, std::vector<Given> &parts)
{
    std::vector<I> base(a.B + 1, 0);
    I items_n = 0, most = 0;
    for (int b = 0; b < a.B; ++b) {
        const PagedSeq<I> s = paged_seq<ROWS, BKV, I>(a, b);
        base[b + 1] = base[b] + a.Hkv * paged_prefix(s, s.mt);
        items_n += a.Hkv * s.mt;
        for (int m = 0; m < s.mt; ++m) most = std::max(most, paged_prefix(s, m + 1) - paged_prefix(s, m));
    }
    const I W = base[a.B];
    if (W == 0) return 0;
    const bool whole = paged_whole<ROWS>(a, W, items_n, most, units);
    const I step = paged_step<ROWS>(a, W, units);
    std::vector<I> bound(units + 1, W), sum(units, 0);
    int waves = whole ? 0 : paged_rounds<ROWS>(a, items_n, units);
    if (waves) {
        I i = 0, taken = 0;
        for (int b = 0; b < a.B; ++b) {
            const PagedSeq<I> s = paged_seq<ROWS, BKV, I>(a, b);
            for (int e = 0; e < a.Hkv * s.mt; ++e, ++i)
                if (i < static_cast<I>(waves) * units)
                    sum[i % units] += paged_prefix(s, e % s.mt + 1) - paged_prefix(s, e % s.mt);
        }
        for (I x : sum) taken += x;
        if (!paged_even(W, units, *std::max_element(sum.begin(), sum.end()))) {
            waves = 0;
        } else {
            ++rounds_n;
            I at = taken;
            for (int u = 0; u < units; ++u) {
                bound[u] = std::min(at, W);
                at += std::max<I>(0, (W + units - 1) / units - sum[u]);
            }
        }
    }
    auto unit_of = [&](I x) -> int {
        if (!waves) return static_cast<int>(x / step);
        int k = 0;
        while (k < units && bound[k] <= x) ++k;
        return k - 1;
    };
    for (int u = 0; u < units; ++u) {
        PagedRange<I> r{};
        r.units = units;
        r.waves = waves;
        PagedSeq<I> first{};
        if (whole) {
            r.waves = u < items_n ? static_cast<int>((items_n - u + units - 1) / units) : 0;
        } else {
            r.begin = waves ? bound[u] : std::min<I>(W, u * step);
            r.end = waves ? bound[u + 1] : std::min<I>(W, r.begin + step);
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
        Given x;
        x.unit = u;
        for (x.at = 0; walk.next(a, x.p, unit_of); ++x.at) parts.push_back(x);
    }
    return 0;
}

// As the walking warp of every CTA (or pair) does, into one list of parts.
template <int ROWS, int BKV, class I>
__global__ void divide_kernel(PagedArgs a, int units, Given *out, int *count, int cap)
{
    __shared__ alignas(8) unsigned char sums[kPagedUnits / 2 * sizeof(int64_t)];
    PagedSeq<I> first{};
    I bound[kPagedBounds<ROWS>];
    const PagedRange<I> range = paged_divide<ROWS, BKV, I>(a, blockIdx.x, units, first, bound, sums);
    PagedWalk<ROWS, BKV, I> walk;
    walk.start(a, range, first);
    auto unit_of = [&](I x) -> int { return paged_unit_of<ROWS>(range, bound, x); };
    Given x;
    x.unit = blockIdx.x;
    for (x.at = 0; x.at < cap && walk.next(a, x.p, unit_of); ++x.at)
        if (threadIdx.x == 0) {
            const int i = atomicAdd(count, 1);
            if (i < cap) out[i] = x;
        }
    if (threadIdx.x == 0 && range.waves > 0 && range.step == 0 && range.begin < range.end) atomicAdd(count + 1, 1);
}

template <int ROWS, int BKV, class I>
int on_device(PagedArgs a, int units, std::vector<Given> &parts)
{
    size_t items = 0;
    for (int b = 0; b < a.B; ++b) items += static_cast<size_t>(a.Hkv) * paged_seq<ROWS, BKV, I>(a, b).mt;
    const int cap = static_cast<int>(items) + 2 * units;
    int32_t *start, *kv, *count;
    Given *out;
    CUDA(cudaMalloc(&start, (a.B + 1) * 4));
    CUDA(cudaMalloc(&kv, a.B * 4));
    CUDA(cudaMalloc(&count, 8));
    CUDA(cudaMalloc(&out, cap * sizeof(Given)));
    CUDA(cudaMalloc(&a.ws, 256));
    CUDA(cudaMemset(a.ws, 0, 256));
    CUDA(cudaMemset(count, 0, 8));
    CUDA(cudaMemcpy(start, a.q_start, (a.B + 1) * 4, cudaMemcpyHostToDevice));
    CUDA(cudaMemcpy(kv, a.kv_len, a.B * 4, cudaMemcpyHostToDevice));
    PagedArgs d = a;
    d.q_start = start;
    d.kv_len = kv;
    divide_kernel<ROWS, BKV, I><<<units, 32>>>(d, units, out, count, cap);
    CUDA(cudaGetLastError());
    CUDA(cudaDeviceSynchronize());
    int n[2];
    CUDA(cudaMemcpy(n, count, 8, cudaMemcpyDeviceToHost));
    if (n[0] > cap) FAIL("%d parts of %zu items", n[0], items);
    rounds_n += n[1] > 0;
    parts.resize(n[0]);
    if (n[0]) CUDA(cudaMemcpy(parts.data(), out, n[0] * sizeof(Given), cudaMemcpyDeviceToHost));
    CUDA(cudaFree(start)); CUDA(cudaFree(kv)); CUDA(cudaFree(count)); CUDA(cudaFree(out)); CUDA(cudaFree(a.ws));
    return 0;
}

template <int ROWS, int BKV, class I>
int both(const PagedArgs &a, int units, bool device)
{
    std::vector<Given> parts;
    const int rc = device ? on_device<ROWS, BKV, I>(a, units, parts) : on_host<ROWS, BKV, I>(a, units, parts);
    if (rc) return rc;
    bool falls = false;
    for (int b = 0; b < a.B; ++b) falls |= a.q_start[b + 1] < a.q_start[b];
    if (device && falls) {
        if (!parts.empty()) FAIL("rows that decrease: %zu parts", parts.size());
        return 0;
    }
    return check<ROWS, BKV, I>(a, units, parts);
}

int main(int argc, char **argv)
{
    const bool device = argc > 1 && !std::strcmp(argv[1], "device");
    int T, B, Hkv, G, page, width, fresh, causal, window, units, bkv, rows;
    long line = 0;
    while (scanf("%d %d %d %d %d %d %d %d %d %d %d %d", &T, &B, &Hkv, &G, &page, &width, &fresh, &causal,
                 &window, &units, &bkv, &rows) == 12) {
        std::vector<int32_t> start(B + 1), kv(B);
        for (auto &x : start) if (scanf("%d", &x) != 1) return 2;
        for (auto &x : kv) if (scanf("%d", &x) != 1) return 2;
        PagedArgs a{};
        a.T = T; a.B = B; a.Hkv = Hkv; a.G = G; a.page_size = page; a.max_pages = width;
        a.has_new = fresh; a.causal = causal; a.window = window;
        a.q_start = start.data(); a.kv_len = kv.data();
        units = std::min(units, rows == 256 ? kPagedUnits / 2 : kPagedUnits);
        auto run = [&](auto i) -> int {
            using I = decltype(i);
            return rows == 256 ? both<256, 128, I>(a, units, device)
                   : bkv == 128 ? both<128, 128, I>(a, units, device) : both<128, 64, I>(a, units, device);
        };
        int rc = run(int64_t{});
        if (!rc && paged_small(T, B, Hkv, G, static_cast<int64_t>(width) * page)) rc = run(int32_t{});
        if (rc) { printf("case %ld\n", line); return 1; }
        ++line;
    }
    printf("%ld cases, %ld in rounds, %ld items cut\n", line, rounds_n, cut_n);
    return 0;
}
"""


def compile_to(folder):
    """The program, built in a folder."""
    src, exe = str(folder / "division.cu"), str(folder / "division")
    with open(src, "w") as f:
        f.write(SOURCE)
    r = subprocess.run([dgbuild.nvcc(), *dgbuild.ARCH, "-O1", "-std=c++17", "-I", dgbuild.CSRC, "-I",
                        os.path.join(dgbuild.ROOT, "include"), src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def run(exe, where, cases, timeout=600):
    """(cases, in rounds, items cut) after all of them passed."""
    text = "\n".join(" ".join(map(str, c)) for c in cases) + "\n"
    r = subprocess.run([exe, where], input=text, capture_output=True, text=True, timeout=timeout)
    if r.returncode:
        at = int(r.stdout.split()[-1]) if "case " in r.stdout else None
        raise AssertionError((r.stdout[-300:], r.stderr[-300:], cases[at][:12] if at is not None else None))
    return [int(w) for w in r.stdout.replace(",", "").split() if w.isdigit()]
