// dg_sample.cu -- draws a token from each row of logits: temperature, top-k, top-p
// and min-p, from given random numbers.
//
// What is kept of a row is a prefix of its tokens in the order (logit falling, index
// rising): all above a value, the cut, and the first few of those that equal it.  So
// nothing is sorted.  The cut is found by counting: the tokens fall into 1024 bins by
// their distance from the maximum, those of the bin it lies in into 1024 again, then
// by their bits.  For top-k the bins count tokens, for top-p their weights, rounded,
// and the exact sums decide afterwards whether the cut found so is the one, or its
// neighbour.
//
// A cluster of CTAs has the row in shared memory, so that the memory is read once,
// however many passes the row takes.  The exact weights exp((x - max) / T) are 64-bit
// fixed-point numbers with a relative error of about 2^-29 (see Weights): a token's
// place among the sums of a whole vocabulary would be lost in 32 bits, and sums of
// integers do not depend on their order.
#include "dg_paged_device.cuh"
#include "dg_serve_kernels.h"

namespace dg {

namespace {

constexpr int kBins = 1024;
constexpr float kBinsLog2 = 16.f;        // bins to a factor of 2 in weight
constexpr int kLaneBits = 54;            // a weight of 1 in a lane's sums; a lane has at most
                                         // 24 x 8 tokens
constexpr int kSumBits = 43;             // in all others: up to 2^19 tokens
constexpr int kDrop = kLaneBits - kSumBits;
constexpr unsigned kAll = 0xFFFFFFFFu;
// Neighbours that top-p's cut is moved over at most.  The rounded weights put it
// within 1e-5 of the row's weight, a few tokens of any vocabulary.
constexpr int kMoves = 1 << 14;

struct Found {
    int bin;                             // -1: the target lies past the last one
    uint32_t count, before;              // tokens in it, and above it
    float mass, target;                  // weight above it, and the weight that was looked for
};

struct alignas(16) SampleShared {
    uint32_t hist[2][kBins];
    uint64_t gather[2][kSampleCluster];
    uint64_t above[2][kSampleCluster * kSampleWarps];   // by segment: weight above the cut,
    uint64_t whole[2][kSampleCluster * kSampleWarps];   // above top-k's,
    uint32_t ties[2][kSampleCluster * kSampleWarps];    // tokens at the cut
    uint64_t red[kSampleWarps];
    uint64_t totals[3];
    uint64_t row_above[kSampleRows + 8];
    uint32_t row_ties[kSampleRows + 8];
    uint32_t table[32];
    float scan_f[kSampleWarps];
    uint32_t scan_u[kSampleWarps];
    Found found;
    int claim, last;
    int seg, tie_prefix;
    uint64_t rem;
};

// round(2^(30 + j / 32))
__constant__ uint32_t kExpTable[32] = {
    1073741824u, 1097253708u, 1121280436u, 1145833280u, 1170923762u, 1196563654u, 1222764986u, 1249540052u,
    1276901417u, 1304861917u, 1333434672u, 1362633090u, 1392470869u, 1422962010u, 1454120821u, 1485961921u,
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u, 1729250827u, 1767116489u,
    1805811301u, 1845353420u, 1885761398u, 1927054196u, 1969251188u, 2012372174u, 2056437387u, 2101467502u};

DG_DEVICE void st_cluster64(uint32_t addr, uint64_t v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
DG_DEVICE void st_cluster32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
DG_DEVICE uint2 ld_cluster2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// Floats as integers in the same order (no NaN; the zeros are one).
DG_DEVICE uint32_t order_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
DG_DEVICE float of_order(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <class T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    DG_DEVICE static void unpack(const uint4 &v, float (&x)[4])
    {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
};
template <>
struct Vec<uint16_t> {
    static constexpr int N = 8;
    DG_DEVICE static void unpack(const uint4 &v, float (&x)[8])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(w[e] << 16);
            x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
    }
};

// floor(f S) for f in [0, 1), a float's 24 bits times 64 (up: the next whole number
// instead, where it is not one).
DG_DEVICE uint64_t part_of(uint64_t S, float f, bool up)
{
    if (!(f > 0.f)) return 0;
    int e;
    const float m = frexpf(f, &e);                       // f = m 2^e, m in [0.5, 1)
    const uint64_t w = static_cast<uint64_t>(m * 16777216.f);
    const int s = 24 - e;                                // f S = w S / 2^s, s >= 24
    const uint64_t lo = w * S, hi = __umul64hi(w, S);
    uint64_t q, rest;
    if (s < 64) {
        q = lo >> s | hi << (64 - s);
        rest = lo & ((1ull << s) - 1);
    } else {
        q = s - 64 < 64 ? hi >> (s - 64) : 0;
        rest = lo | (s - 64 < 64 ? hi & ((1ull << (s - 64)) - 1) : hi);
    }
    return q + (up && rest != 0 ? 1 : 0);
}

// Weights 2^(c x - reference), c = log2 e / T, as 64-bit integers, 2^54 for 1.
// c x is taken in units of 1/32: P, its nearest whole number, comes out of one
// multiply-add with a large constant, exactly; what is left of it, |r| <= 1/64, of a
// second, rounded at 2^-31, and c's low half with it.  Then 2^(j / 32) from a table
// and 2^r = 1 + y by its series, y rounded at 2^-28.  The reference is the maximum's
// own P, so the largest weight lies within 2^(1/64) of 1 and a row of equal logits
// has equal ones, with nothing cut off.  Where |c x| is too large for that (2^16 and
// more), the same in 64-bit arithmetic.
struct Weights {
    float ch, cl, floor;
    int ref;
    bool wide;
    float m;
    double c;

    DG_DEVICE void init(float max, float t)
    {
        m = max;
        c = 1.4426950408889634 / static_cast<double>(t);
        ch = static_cast<float>(c);
        cl = static_cast<float>(c - static_cast<double>(ch));
        floor = max - 60.f / ch;
        ref = __float_as_int(fmaf(max, ch, 393216.f));   // 1.5 x 2^18: a unit in the last place is 1/32
        wide = !(fabsf(max) * ch < 65536.f);
    }
    // ln of what a weight of 2^54 stands for beside exp((x - max) / T) = 1
    DG_DEVICE double shift() const
    {
        if (wide) return 0.;
        const double at = static_cast<double>(__int_as_float(ref) - 393216.f);
        return (at - static_cast<double>(m) * c) * 0.6931471805599453;
    }
    DG_DEVICE uint64_t operator()(float x, const uint32_t *table) const
    {
        if (wide) return in_double(x);
        const float y = fmaxf(x, floor);
        const float P = fmaf(y, ch, 393216.f);
        const float Pf = P - 393216.f;
        float r = fmaf(y, ch, -Pf);
        r = fmaf(y, cl, r);
        const int i = __float_as_int(P) - ref;
        float s = fmaf(r, 0.0096181291f, 0.055504109f);  // ln2^4 / 24, ln2^3 / 6
        s = fmaf(r, s, 0.24022651f);                     // ln2^2 / 2
        s = fmaf(r, s, 0.69314718f);
        const float B = fmaf(r, s, 0.046875f);           // 1.5 x 2^-5: in units of 2^-28
        const uint32_t T = table[i & 31];
        const int yi = __float_as_int(B) - __float_as_int(0.046875f);
        const uint32_t w = T + static_cast<uint32_t>(__mulhi(static_cast<int>(T), yi << 4));
        return static_cast<uint64_t>(w) << 24 >> min(-(i >> 5), 63);
    }
    DG_DEVICE uint64_t in_double(float x) const
    {
        const double t = (static_cast<double>(x) - static_cast<double>(m)) * c;
        return t > -60. ? static_cast<uint64_t>(exp2(t) * 18014398509481984.) : 0;
    }
};

template <class T>
struct Sampler {
    static constexpr int E = Vec<T>::N;
    const SampleArgs &a;
    SampleShared &sh;
    const uint4 *data;
    const int warp, lane, rank, ctas;
    int turn = 0, hist_turn = 0;
    Weights weight;
    float m = 0.f;
    bool flat = false;                   // the maximum is infinite: those tokens alone, alike

    DG_DEVICE Sampler(const SampleArgs &args, SampleShared &s, const uint4 *d)
        : a(args), sh(s), data(d), warp(threadIdx.x >> 5), lane(threadIdx.x & 31),
          rank(static_cast<int>(cluster_ctarank())), ctas(0)
    {
        uint32_t n;
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
        const_cast<int &>(ctas) = static_cast<int>(n);
    }

    DG_DEVICE uint64_t w_of(float x) const
    {
        return flat ? (x == m ? 1ull << kLaneBits : 0) : weight(x, sh.table);
    }
    // n tokens of weight w in the units of the sums
    DG_DEVICE static uint64_t times(uint64_t w, uint64_t n)
    {
        return n * (w >> kDrop) + (n * (w & ((1u << kDrop) - 1)) >> kDrop);
    }

    // f(x) for each of this thread's tokens (places past the row hold -inf).
    template <class F>
    DG_DEVICE void each(F f) const
    {
        for (int r = 0; r < a.rows_warp; ++r) {
            float x[E];
            Vec<T>::unpack(data[(warp * a.rows_warp + r) * 32 + lane], x);
#pragma unroll
            for (int e = 0; e < E; ++e) f(x[e], r, e);
        }
    }
    // The place of a token in its row, `skew` places early.
    DG_DEVICE int place(int w, int r, int l, int e) const
    {
        return (((rank * kSampleWarps + w) * a.rows_warp + r) * 32 + l) * E + e;
    }

    // The largest of two values over the cluster.
    DG_DEVICE uint2 largest(uint32_t x, uint32_t y)
    {
        x = __reduce_max_sync(kAll, x);
        y = __reduce_max_sync(kAll, y);
        if (lane == 0) sh.red[warp] = static_cast<uint64_t>(y) << 32 | x;
        __syncthreads();
        const int buf = turn++ & 1;
        if (warp == 0) {
            const uint64_t v = sh.red[lane & (kSampleWarps - 1)];
            x = __reduce_max_sync(kAll, static_cast<uint32_t>(v));
            y = __reduce_max_sync(kAll, static_cast<uint32_t>(v >> 32));
            if (lane < ctas)
                st_cluster64(mapa_shared(smem_u32(&sh.gather[buf][rank]), lane),
                             static_cast<uint64_t>(y) << 32 | x);
        }
        cluster_sync_all();
        uint2 got = make_uint2(0, 0);
        for (int k = 0; k < ctas; ++k) {
            const uint64_t v = sh.gather[buf][k];
            got.x = max(got.x, static_cast<uint32_t>(v));
            got.y = max(got.y, static_cast<uint32_t>(v >> 32));
        }
        return got;
    }

    // ------------------------------------------------------------ a histogram over the cluster
    DG_DEVICE uint32_t *clear()
    {
        uint32_t *hist = sh.hist[hist_turn & 1];
        for (int k = threadIdx.x; k < kBins; k += kSampleThreads) hist[k] = 0;
        __syncthreads();
        return hist;
    }
    // The bin in which the tokens reach `target` in number, or with `mass` (counts
    // weighed by of_bin) want.target in weight, or that part of it all less `less`.
    // Where rounded sums stay short of that, the last one that is not empty.
    template <class F>
    DG_DEVICE Found find(bool mass, uint32_t target, float target_mass, float part, float less, F of_bin)
    {
        const int buf = hist_turn++ & 1;
        if (threadIdx.x == 0) {
            sh.claim = kSampleThreads;
            sh.last = -1;
        }
        cluster_sync_all();
        const int b = 2 * threadIdx.x;
        uint32_t n0 = 0, n1 = 0;
        for (int k = 0; k < ctas; ++k) {
            const uint2 v = ld_cluster2(mapa_shared(smem_u32(&sh.hist[buf][b]), k));
            n0 += v.x;
            n1 += v.y;
        }
        const float f0 = mass ? n0 * of_bin(b) : 0.f, f1 = mass ? n1 * of_bin(b + 1) : 0.f;
        uint32_t n = n0 + n1;
        float f = f0 + f1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t un = __shfl_up_sync(kAll, n, o);
            const float uf = __shfl_up_sync(kAll, f, o);
            if (lane >= o) {
                n += un;
                f += uf;
            }
        }
        if (lane == 31) {
            sh.scan_u[warp] = n;
            sh.scan_f[warp] = f;
        }
        __syncthreads();
        uint32_t n_all = 0;
        float f_all = 0.f;
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w == warp) {
                n += n_all;
                f += f_all;
            }
            n_all += sh.scan_u[w];
            f_all += sh.scan_f[w];
        }
        if (part > 0.f) target_mass = part * (f_all - less);
        if (n0 + n1 > 0) {
            if (mass ? f >= target_mass : n >= target) atomicMin(&sh.claim, static_cast<int>(threadIdx.x));
            atomicMax(&sh.last, static_cast<int>(threadIdx.x));
        }
        __syncthreads();
        const bool reached = sh.claim < kSampleThreads;
        if (static_cast<int>(threadIdx.x) == (reached ? sh.claim : max(sh.last, 0))) {
            bool second = n0 == 0;
            if (n0 > 0 && n1 > 0) second = !reached || (mass ? f - f1 < target_mass : n - n1 < target);
            sh.found = Found{reached || mass ? (second ? b + 1 : b) : -1, second ? n1 : n0,
                             second ? n - n1 : n - n0 - n1, second ? f - f1 : f - f0 - f1, target_mass};
            if (sh.last < 0) sh.found.bin = -1;
        }
        __syncthreads();
        return sh.found;
    }

    // ------------------------------------------------------------ the cut
    struct Cut {
        float v;                          // -inf: none
        uint32_t first;                   // how many of the tokens at v are kept
        uint32_t ties;                    // tokens at v
    };

    // Where the tokens reach k in number or, with `mass`, the part p of the weight of
    // those that `least` keeps.  Tokens of weight 0 do not count; none: there are too
    // few.  With `mass` it may be one of the cut's neighbours (the weights are rounded).
    DG_DEVICE Cut select(bool mass, uint32_t k, float p, const Cut &least)
    {
        const float s1 = weight.ch * kBinsLog2, floor_v = least.v;
        auto y_of = [&](float x) -> float { return (m - x) * s1; };
        uint32_t *hist = clear();
        each([&](float x, int, int) {
            const float y = y_of(x);
            if (!(x >= floor_v) || !(y < static_cast<float>(kBins))) return;
            const int b = static_cast<int>(y);
            uint32_t inc = 1;
            if (mass) {
                // its weight beside that of the bin's upper end, 2^(-f / 16)
                const float f = y - static_cast<float>(b);
                inc = static_cast<uint32_t>(fmaf(f, fmaf(f, 9.3838e-4f, -0.0433217f), 1.f) * 65536.f);
            }
            atomicAdd(hist + b, inc);
        });
        const float less = mass && floor_v > -INFINITY
                               ? static_cast<float>(least.ties - least.first) * exp2f(-y_of(floor_v) / kBinsLog2)
                               : 0.f;
        const Found f1 = find(mass, k, 0.f, p, less,
                              [&](int b) -> float { return exp2f(-b / kBinsLog2) * (1.f / 65536.f); });
        if (f1.bin < 0) return Cut{-INFINITY, 0, 0};
        // that bin's tokens by their place in it
        const float b1 = static_cast<float>(f1.bin);
        auto y2_of = [&](float y) -> int { return min(static_cast<int>((y - b1) * kBins), kBins - 1); };
        auto inside = [&](float x, float y) -> bool {
            return x >= floor_v && y < static_cast<float>(kBins) && static_cast<int>(y) == f1.bin;
        };
        hist = clear();
        each([&](float x, int, int) {
            const float y = y_of(x);
            if (inside(x, y)) atomicAdd(hist + y2_of(y), 1u);
        });
        uint32_t before = mass ? 0 : f1.before;
        float above = f1.mass;
        const Found f2 = find(mass, k - before, f1.target - above, 0.f, 0.f, [&](int b) -> float {
            return exp2f(-(b1 + (static_cast<float>(b) + 0.5f) * (1.f / kBins)) / kBinsLog2);
        });
        if (f2.bin < 0) return Cut{-INFINITY, 0, 0};
        // and by their bits
        before += f2.before;
        above += f2.mass;
        uint32_t hi = 0, lo = 0, ties = f2.count;
        each([&](float x, int, int) {
            const float y = y_of(x);
            if (inside(x, y) && y2_of(y) == f2.bin) {
                hi = max(hi, order_of(x));
                lo = max(lo, ~order_of(x));
            }
        });
        const uint2 ends = largest(hi, lo);
        hi = ends.x;
        lo = ~ends.y;
        while (hi > lo) {
            const int shift = max(0, 22 - __clz(hi - lo));
            hist = clear();
            each([&](float x, int, int) {
                if (!(x >= floor_v)) return;
                const uint32_t o = order_of(x);
                if (o <= hi && o >= lo) atomicAdd(hist + ((hi - o) >> shift), 1u);
            });
            const Found f3 = find(mass, k - before, f1.target - above, 0.f, 0.f, [&](int b) -> float {
                const uint64_t mid = (static_cast<uint64_t>(b) << shift) + (1u << shift >> 1);
                return exp2f(-y_of(of_order(mid < hi - lo ? hi - static_cast<uint32_t>(mid) : lo)) / kBinsLog2);
            });
            if (f3.bin < 0) return Cut{-INFINITY, 0, 0};
            before += f3.before;
            above += f3.mass;
            ties = f3.count;
            hi -= static_cast<uint32_t>(f3.bin) << shift;
            if (hi - lo > (1u << shift) - 1) lo = hi - ((1u << shift) - 1);
            if (shift == 0) break;
        }
        return Cut{of_order(hi), mass ? ties : k - before, ties};
    }

    // ------------------------------------------------------------ exact sums
    struct Sums {
        uint64_t above, whole;            // weight above the cut, above top-k's
        uint32_t ties;                    // tokens at the cut
        int buf;
    };
    int sum_turn = 0;
    DG_DEVICE Sums sums(float v, float floor_v, bool with_whole)
    {
        uint64_t above = 0, whole = 0;
        uint32_t ties = 0;
        const float least = with_whole ? fminf(v, floor_v) : v;
        for (int r = 0; r < a.rows_warp; ++r) {
            float x[E];
            Vec<T>::unpack(data[(warp * a.rows_warp + r) * 32 + lane], x);
            bool any = false;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                any |= x[e] > least;
                ties += x[e] == v ? 1u : 0u;
            }
            if (!__any_sync(kAll, any)) continue;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (!(x[e] > least)) continue;
                const uint64_t w = w_of(x[e]);
                if (x[e] > v) above += w;
                if (x[e] > floor_v) whole += w;
            }
        }
        above >>= kDrop;
        whole >>= kDrop;
        if (v == -INFINITY) ties = 0;     // (those past the row's end)
        ties = __reduce_add_sync(kAll, ties);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            above += __shfl_xor_sync(kAll, above, o);
            whole += __shfl_xor_sync(kAll, whole, o);
        }
        const int buf = sum_turn++ & 1;
        if (lane < ctas) {
            const int at = rank * kSampleWarps + warp;
            st_cluster64(mapa_shared(smem_u32(&sh.above[buf][at]), lane), above);
            st_cluster64(mapa_shared(smem_u32(&sh.whole[buf][at]), lane), whole);
            st_cluster32(mapa_shared(smem_u32(&sh.ties[buf][at]), lane), ties);
        }
        cluster_sync_all();
        if (warp == 0) {
            above = whole = 0;
            ties = 0;
            for (int k = lane; k < ctas * kSampleWarps; k += 32) {
                above += sh.above[buf][k];
                whole += sh.whole[buf][k];
                ties += sh.ties[buf][k];
            }
            ties = __reduce_add_sync(kAll, ties);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                above += __shfl_xor_sync(kAll, above, o);
                whole += __shfl_xor_sync(kAll, whole, o);
            }
            if (lane == 0) {
                sh.totals[0] = above;
                sh.totals[1] = whole;
                sh.totals[2] = ties;
            }
        }
        __syncthreads();
        const Sums s{sh.totals[0], sh.totals[1], static_cast<uint32_t>(sh.totals[2]), buf};
        __syncthreads();
        return s;
    }

    // The first of up to 32 parts, a lane's each (of weight `above` and `ties` tokens at
    // the cut, of which `kept` from the first part on count), in which `rem` falls: its
    // lane, what of rem lies in it and how many ties come before it.  By a warp.
    DG_DEVICE int locate(uint64_t above, uint32_t ties, uint64_t w, int64_t kept, uint64_t &rem, int &tie_prefix)
    {
        uint32_t before = ties;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += x;
        }
        before -= ties;
        const int64_t left = kept - tie_prefix - before;
        const uint64_t mine = above + times(w, left <= 0 ? 0 : left < ties ? left : ties);
        uint64_t end = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(kAll, end, o);
            if (lane >= o) end += x;
        }
        const uint32_t past = __ballot_sync(kAll, end > rem && mine > 0), any = __ballot_sync(kAll, mine > 0);
        int at = past != 0 ? __ffs(past) - 1 : any != 0 ? 31 - __clz(any) : 0;
        const uint64_t begin = __shfl_sync(kAll, end - mine, at), size = __shfl_sync(kAll, mine, at);
        rem = past != 0 ? rem - begin : size > 0 ? size - 1 : 0;     // (sums round off: the last one)
        tie_prefix += __shfl_sync(kAll, before, at);
        return at;
    }

    // The token in which `rem` of the kept weight falls, in the order of the vocabulary:
    // by the CTA that has it.
    DG_DEVICE void draw(float v, int64_t kept, const Sums &s, uint64_t rem, int row, int skew, double log_all)
    {
        const uint64_t wv = v > -INFINITY ? w_of(v) : 0;
        if (warp == 0) {
            // the segment: a lane takes `per` of them
            const int n = ctas * kSampleWarps, per = (n + 31) / 32;
            uint64_t above = 0;
            uint32_t ties = 0;
            for (int k = lane * per; k < min(n, (lane + 1) * per); ++k) {
                above += sh.above[s.buf][k];
                ties += sh.ties[s.buf][k];
            }
            int prefix = 0;
            const int at = locate(above, ties, wv, kept, rem, prefix);
            const int k = at * per + lane;
            const bool mine = lane < per && k < n;
            const int in = locate(mine ? sh.above[s.buf][k] : 0, mine ? sh.ties[s.buf][k] : 0, wv, kept, rem, prefix);
            if (lane == 0) {
                sh.seg = at * per + in;
                sh.rem = rem;
                sh.tie_prefix = prefix;
            }
        }
        __syncthreads();
        if (sh.seg / kSampleWarps != rank) return;
        const int seg = sh.seg % kSampleWarps;
        auto row_of = [&](int r, uint64_t &above, uint32_t &ties, float (&x)[E]) {
            Vec<T>::unpack(data[(seg * a.rows_warp + r) * 32 + lane], x);
            above = 0;
            ties = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (x[e] > v) above += w_of(x[e]);
                ties += x[e] == v && v > -INFINITY ? 1u : 0u;
            }
            above >>= kDrop;
        };
        for (int r = warp; r < a.rows_warp; r += kSampleWarps) {
            uint64_t above;
            uint32_t ties;
            float x[E];
            row_of(r, above, ties, x);
            ties = __reduce_add_sync(kAll, ties);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) above += __shfl_xor_sync(kAll, above, o);
            if (lane == 0) {
                sh.row_above[r] = above;
                sh.row_ties[r] = ties;
            }
        }
        __syncthreads();
        if (warp != 0) return;
        rem = sh.rem;
        int prefix = sh.tie_prefix;
        const bool mine = lane < a.rows_warp;
        const int r = locate(mine ? sh.row_above[lane] : 0, mine ? sh.row_ties[lane] : 0, wv, kept, rem, prefix);
        uint64_t above;
        uint32_t ties;
        float x[E];
        row_of(r, above, ties, x);
        const int l = locate(above, ties, wv, kept, rem, prefix);
        if (lane != l) return;
        uint64_t sum = 0;
        int token = -1;
        float value = 0.f;
        for (int e = 0; e < E; ++e) {
            const bool tie = x[e] == v && v > -INFINITY;
            const bool in = x[e] > v || (tie && prefix < kept);
            prefix += tie ? 1 : 0;
            const uint64_t w = in ? w_of(x[e]) : 0;
            if (w == 0) continue;
            token = place(seg, r, l, e) - skew;
            value = x[e];
            sum += w;
            if (sum > rem << kDrop) break;
        }
        if (token < 0) {
            // (parts too small to count beside the rest: the segment's last kept token)
            prefix = sh.tie_prefix;
            for (int k = 0; k < a.rows_warp * 32; ++k) {
                Vec<T>::unpack(data[seg * a.rows_warp * 32 + k], x);
                for (int e = 0; e < E; ++e) {
                    const bool tie = x[e] == v && v > -INFINITY;
                    if (x[e] > v || (tie && prefix < kept)) {
                        token = place(seg, k / 32, k % 32, e) - skew;
                        value = x[e];
                    }
                    prefix += tie ? 1 : 0;
                }
            }
        }
        say(row, token, value, log_all);
    }

    DG_DEVICE void say(int row, int token, float value, double log_all) const
    {
        a.token[row] = token;
        if (a.logprob != nullptr) {
            const double at = flat ? 0. : (static_cast<double>(value) - static_cast<double>(m)) * weight.c * 0.6931471805599453;
            a.logprob[row] = static_cast<float>(at - log_all);
        }
    }

    DG_DEVICE void row(int row, uint4 *keep)
    {
        constexpr uint32_t Low = E == 8 ? 0xFF80FF80u : 0xFF800000u;
        const int64_t at = row * a.stride;
        const int skew = static_cast<int>(at & (E - 1));     // the row begins inside 16 bytes
        const T *base = static_cast<const T *>(a.logits) + (at - skew);
        cluster_arrive_all();                                // (the others' shared memory: only once they run)
        m = -INFINITY;
#pragma unroll 4
        for (int r = 0; r < a.rows_warp; ++r) {
            const int first = place(warp, r, lane, 0);
            uint4 v = make_uint4(Low, Low, Low, Low);
            if (first >= skew && first + E <= a.V + skew) {
                v = __ldg(reinterpret_cast<const uint4 *>(base + first));
            } else if (first + E > skew && first < a.V + skew) {
                T x[E];
                *reinterpret_cast<uint4 *>(x) = v;
                for (int e = 0; e < E; ++e)
                    if (first + e >= skew && first + e < a.V + skew) x[e] = base[first + e];
                v = *reinterpret_cast<const uint4 *>(x);
            }
            keep[(warp * a.rows_warp + r) * 32 + lane] = v;
            float x[E];
            Vec<T>::unpack(v, x);
#pragma unroll
            for (int e = 0; e < E; ++e) m = fmaxf(m, x[e]);
        }
        if (threadIdx.x < 32) sh.table[threadIdx.x] = kExpTable[threadIdx.x];
        __syncwarp();
        cluster_wait_all();
        m = of_order(largest(order_of(m), 0).x);

        const bool lead = rank == 0 && threadIdx.x == 0;
        if (m == -INFINITY) {                                // no token
            if (lead) {
                a.token[row] = -1;
                if (a.logprob != nullptr) a.logprob[row] = -INFINITY;
            }
            return;
        }
        float t = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.f;
        const int k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
        const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
        const float low = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.f;
        if (!(t > 0.f) || k == 1 || p <= 0.f) {              // the first of the largest
            uint32_t best = 0;
            each([&](float x, int r, int e) {
                if (x == m) best = max(best, ~static_cast<uint32_t>(place(warp, r, lane, e)));
            });
            best = largest(best, 0).x;
            if (lead) {
                a.token[row] = static_cast<int>(~best) - skew;
                if (a.logprob != nullptr) a.logprob[row] = 0.f;
            }
            return;
        }
        flat = m == INFINITY;
        t = fminf(fmaxf(t, 7.8886091e-31f), 1.2676506e30f);  // 2^-100, 2^100
        if (!flat) weight.init(m, t);
        // top-k's cut, min-p's, top-p's: the highest is the one
        Cut by_k{-INFINITY, 0, 0};
        const bool some = k > 0 && k < a.V;
        if (flat) by_k = Cut{m, some ? static_cast<uint32_t>(k) : ~0u, 0};
        else if (some) by_k = select(false, k, 0.f, by_k);
        float least = by_k.v;
        if (low > 0.f && !flat)
            least = fmaxf(least, fminf(m, __double2float_ru(static_cast<double>(m) +
                                                            static_cast<double>(t) * log(static_cast<double>(low)))));
        const bool part = p < 1.f;
        float v = least;
        if (part && !flat) v = fmaxf(v, select(true, 0, p, by_k).v);
        Sums s = sums(v, by_k.v, part);
        int64_t kept;
        for (int moves = 0;; ++moves) {
            const uint64_t wv = v > -INFINITY ? w_of(v) : 0;
            kept = v == by_k.v ? min(by_k.first, s.ties) : s.ties;
            if (!part || moves == kMoves) break;
            uint64_t all = s.whole;
            if (by_k.v > -INFINITY) all += times(w_of(by_k.v), flat ? min(by_k.first, s.ties) : by_k.first);
            const uint64_t need = part_of(all, p, true);
            if (s.above >= need && s.above > 0) {            // reached before: one up
                uint32_t up = 0;
                each([&](float x, int, int) {
                    if (x > v) up = max(up, ~order_of(x));
                });
                v = of_order(~largest(up, 0).x);
            } else if (s.above + times(wv, kept) >= need || !(v > least)) {
                // the fewest at the cut that reach it
                const uint64_t short_of = need > s.above ? need - s.above : 0;
                int64_t n = 0;
                for (int64_t step = 1 << 20; step > 0; step >>= 1)
                    if (n + step <= kept && times(wv, n + step) < short_of) n += step;
                kept = min(kept, n + 1);
                break;
            } else {                                         // one down
                uint32_t down = 0;
                each([&](float x, int, int) {
                    if (x < v && x >= least) down = max(down, order_of(x));
                });
                down = largest(down, 0).x;
                if (down == 0 || of_order(down) == -INFINITY) break;
                v = of_order(down);
            }
            s = sums(v, by_k.v, part);
        }
        const uint64_t all = s.above + times(v > -INFINITY ? w_of(v) : 0, kept);
        const float u = __ldg(a.u + row);
        const uint64_t rem = u < 1.f ? part_of(all, u, false) : all - 1;
        const double log_all = log(static_cast<double>(all)) - kSumBits * 0.6931471805599453 +
                               (flat ? 0. : weight.shift());
        if (rem == 0) {                                      // the first that is kept, however light
            uint32_t best = 0;
            each([&](float x, int r, int e) {
                if (x > v || (x == v && kept > 0)) best = max(best, ~static_cast<uint32_t>(place(warp, r, lane, e)));
            });
            const uint32_t mine = best;
            best = largest(best, 0).x;
            if (mine == best && best != 0) {
                const int at = static_cast<int>(~best);      // (one thread has it)
                float x[E];
                Vec<T>::unpack(data[at / E - rank * kSampleWarps * a.rows_warp * 32], x);
                float value = x[0];
#pragma unroll
                for (int e = 1; e < E; ++e)
                    if (at % E == e) value = x[e];
                say(row, at - skew, value, log_all);
            }
            return;
        }
        draw(v, kept, s, min(rem, all - 1), row, skew, log_all);
    }
};

template <class T>
__device__ __forceinline__ void sample_body(const SampleArgs &a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    SampleShared &sh = *reinterpret_cast<SampleShared *>(smem);
    uint4 *keep = reinterpret_cast<uint4 *>(smem + sizeof(SampleShared));
    griddep_wait();
    griddep_launch_dependents();
    Sampler<T> s(a, sh, keep);
    s.row(static_cast<int>(cluster_id_x()), keep);
    __syncwarp();
    cluster_sync_all();                  // nobody leaves while its shared memory may be read
}

}  // namespace

int sample_smem_bytes(int rows_warp)
{
    return static_cast<int>(sizeof(SampleShared)) + rows_warp * kSampleThreads * 16;
}

__global__ void __launch_bounds__(kSampleThreads, 2) sample_bf16_kernel(SampleArgs a) { sample_body<uint16_t>(a); }
__global__ void __launch_bounds__(kSampleThreads, 2) sample_fp32_kernel(SampleArgs a) { sample_body<float>(a); }

}  // namespace dg
