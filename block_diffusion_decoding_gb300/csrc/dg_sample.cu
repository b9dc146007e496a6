// dg_sample.cu -- draws a token from each row of logits: temperature, top-k, top-p
// and min-p, from given random numbers.
//
// What is kept of a row is a prefix of its tokens in the order (logit falling, index
// rising): all above a value, the cut, and the first few of those that equal it.  So
// a vocabulary is not sorted.  Every way to the token begins with one pass over the
// row, in which a thread takes the maximum of each of its groups of tokens.
//   no filter    the weights are summed, a stretch of the row a warp; the token is
//                looked for in the stretch that the random number falls into;
//   few kept     (top-k of up to kListMost, what min-p leaves, a small nucleus) the
//                groups whose maximum reaches a value that the cut lies above are read
//                again for the tokens above it, which are sorted and summed by one CTA.
//                For top-k the value is the k-th largest of the groups' maxima;
//   top-p        the weights, rounded, are summed in bins of 1/8 of a factor of 2; the
//                tokens of the bin that holds the cut (or of a part of it) are sorted, as
//                above, beside the exact sums of the row and of what lies above them;
//   the rest     (a larger k, cuts that lie elsewhere) the cut is found by counting: the
//                tokens fall into 1024 bins by their distance from the maximum, those
//                of the bin it lies in into 1024 again, then by their bits; the exact
//                sums decide whether it is the one found or a neighbour.
// A row is a cluster's; its CTAs exchange maxima, bins and sums through each other's
// shared memory.
//
// What bounds it is not the one read of the logits that it cannot do without (the first
// pass; the later ones find much of the row in L2), but instructions and, where rows are
// few, barriers and latencies in a row.  On one GB300, us, beside that read at a copy's
// rate, normal logits times 3:
//                         floor  greedy  none  k 50  k 50, p 0.9  p 0.9  min-p 0.05  k 5000  p 0.99995
//   1 row of 16384 bf16     0.0     7     11    10       10         28        9         37       80
//   1 of 262144 fp32        0.2     6     15    15       15         40       13         50      375
//   64 of 262144 fp32       9.9    16     40    27       28         80       26        121     1031
//   1024 of 151643 bf16    45.8    71    206   100       99        462       98        585     1839
// (calls back to back, 6 us of which are the host's).  The last two are cut by counting.
// Without a filter a token takes 34 instructions in all, on 60% of the issue slots (512
// rows of 151643, in a profile); greedy rows wait for memory, and at a block's end for one
// another, with 44% of an SM's warps there (64 registers), on 38% of the slots.  Where the
// list is of one value, 1500 equal logits, its sort compares each with all: 1 row of 16384,
// k = 1000, 44 in place of 21.
// Tried and no better: the row a few pieces ahead through asynchronous copies to shared
// memory (the last line's none, then 225, -> 233; top-p on one row 46.4 -> 44.7), prefetches of the
// rows to come into L2 (its 122, then, -> 133), fewer CTAs an SM, to spread clusters (no
// change for few rows; top-p on 64 rows 109 with 4, 156 with 2), both policies for the
// clusters' places (no change).
//
// The exact weights exp((x - max) / T) are 64-bit fixed-point numbers with a relative
// error of about 2^-29 (see Weights): a token's place among the sums of a whole
// vocabulary would be lost in 32 bits, and sums of integers do not depend on their
// order, nor on the number of CTAs that share a row.
#include <cfloat>
#include <cstddef>

#include "dg_paged_device.cuh"
#include "dg_serve_kernels.h"

namespace dg {

namespace {

constexpr int kBins = 1024;
constexpr int kBinsThread = kBins / kSampleThreads;
constexpr float kBinsLog2 = 16.f;        // of the search by counting: bins to a factor of 2 in weight
constexpr float kMassOne = 8192.f;       // a weight where its bin stands for it, in sums of rounded ones
constexpr float kEighths = 1572864.f;    // 1.5 x 2^20: a unit in the last place is 1/8
constexpr int kMassBins = 256;           // of top-p's: 8 to a factor of 2
constexpr int kGroupBytes = 32;          // of the maxima of a thread's groups: 8, of bf16 tokens 16
constexpr int kList = 1536;              // tokens that are sorted at most
constexpr int kListMost = 1024;          // of which top-k's k
// A weight of 1, up to 393216 of which (and of 2^(1/64), see Weights) fit a sum.  Each one
// is cut off to this by itself: a sum is the same however its tokens are shared out.
constexpr int kWeightBits = 45;
constexpr unsigned kAll = 0xFFFFFFFFu;
// Tokens that top-p's cut of fp32 rows is moved over before it is looked for further off.
// The rounded weights put it within 1e-5 of the row's weight: mostly where it is or beside
// it, but where p is next to 1 that may be thousands of light tokens (2000 of 262144
// normal logits times 3, p = 0.99995: 20 ms token by token, 0.39 as it is).
constexpr int kNeighbours = 2;

struct Found {
    int bin;                             // -1: the target lies past the last one
    uint32_t count, before, total;       // tokens in it, above it, and in all bins
    float mass, all;                     // weight above it, and of all bins
    bool reached;                        // (with rounded weights: else the last one with a token)
};

struct Cut {
    float v;                             // -inf: none
    uint32_t first;                      // how many of the tokens at v are kept
    uint32_t ties;                       // tokens at v
};

constexpr int kSegments = kSampleCluster * kSampleWarps;
struct alignas(16) SampleShared {
    uint32_t hist[2][kBins];
    uint64_t list[kList];                 // (the first CTA's) tokens: falling value, index
    uint64_t mass[kList];                 // their weights in that order
    uint64_t gather[2][kSegments];
    union {
        struct {
            uint64_t above[2][kSegments];   // by segment: weight above the cut
            uint64_t whole[kSegments];      // (once a row)
            uint32_t ties[2][kSegments];    // and tokens at it
            uint64_t row_above[kSampleRows];
            uint32_t row_ties[kSampleRows];
            uint8_t group[kGroupBytes * kSampleThreads];   // maxima, as the tokens' type
        };
        uint64_t moved[kList];            // the list while it is sorted
    };
    uint64_t red[kSampleWarps];
    uint32_t table[32];
    float scan_f[kSampleWarps];
    uint32_t scan_u[kSampleWarps];
    Found found[2];
    Cut cut;
    int claim[2], last;
    int seg, tie_prefix;
    uint64_t rem, all;
    uint32_t listed, base, todo;
    float min_value;
};

// (what is written and read 64 and 128 bits wide through cluster addresses)
static_assert(offsetof(SampleShared, hist) % 16 == 0 && offsetof(SampleShared, list) % 8 == 0 &&
                  offsetof(SampleShared, gather) % 8 == 0 && offsetof(SampleShared, above) % 8 == 0 &&
                  offsetof(SampleShared, rem) % 8 == 0 && offsetof(SampleShared, all) % 8 == 0 &&
                  offsetof(SampleShared, cut) % 4 == 0 && offsetof(SampleShared, group) % 4 == 0,
              "alignment");

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
DG_DEVICE uint32_t ld_cluster32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
DG_DEVICE uint32_t add_cluster32(uint32_t addr, uint32_t v)
{
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
    return old;
}
DG_DEVICE uint4 ld_cluster4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
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
    using Most = float;
    DG_DEVICE static Most none() { return -INFINITY; }
    DG_DEVICE static void most(Most &m, const uint4 &v)
    {
        m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v.x)), __uint_as_float(v.y)),
                  fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    DG_DEVICE static float value(Most m) { return m; }
    DG_DEVICE static float at(const uint4 &v, int e)
    {
        return __uint_as_float(e < 2 ? (e < 1 ? v.x : v.y) : (e < 3 ? v.z : v.w));
    }
    DG_DEVICE static float widen(float x) { return x; }
    DG_DEVICE static float narrow(float x) { return x; }
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
    using Most = __nv_bfloat162;
    DG_DEVICE static Most none() { return __floats2bfloat162_rn(-INFINITY, -INFINITY); }
    DG_DEVICE static void most(Most &m, const uint4 &v)
    {
        const __nv_bfloat162 *x = reinterpret_cast<const __nv_bfloat162 *>(&v);
        m = __hmax2(__hmax2(m, x[0]), __hmax2(x[1], __hmax2(x[2], x[3])));
    }
    DG_DEVICE static float value(Most m) { return fmaxf(__low2float(m), __high2float(m)); }
    DG_DEVICE static float at(const uint4 &v, int e)
    {
        const uint32_t w = e < 4 ? (e < 2 ? v.x : v.y) : (e < 6 ? v.z : v.w);
        return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    }
    DG_DEVICE static float widen(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
    // (of what is a bf16 number)
    DG_DEVICE static uint16_t narrow(float x) { return static_cast<uint16_t>(__float_as_uint(x) >> 16); }
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

// A weight in 64-bit arithmetic (kept out of line: it is seldom called, and long).
__device__ __noinline__ uint64_t weight_in_double(float x, float m, float ch, float cl)
{
    const double t = (static_cast<double>(x) - static_cast<double>(m)) *
                     (static_cast<double>(ch) + static_cast<double>(cl));
    return t > -60. ? static_cast<uint64_t>(exp2(t) * 35184372088832.) : 0;   // 2^kWeightBits
}

// Weights 2^(c x - reference), c = log2 e / T, as 64-bit integers, 2^kWeightBits for 1.
// c x is taken in units of 1/32: P, its nearest whole number, comes out of one
// multiply-add with a large constant, exactly; what is left of it, |r| <= 1/64, of a
// second, rounded at 2^-31, and c's low half with it.  Then 2^(j / 32) from a table
// (turned so that P's own low bits find it) and 2^r = 1 + y by its series, to r^3 (the
// next term is below 2^-30), y rounded at 2^-28.  The reference is the maximum's own P,
// so the largest weight lies within 2^(1/64) of 1 and a row of equal logits has equal
// ones, with nothing cut off.  Where |c x| is too large for that (2^16 and more), the
// same in 64-bit arithmetic.
struct Weights {
    float ch, cl, floor;
    int ref;
    bool wide;
    float m;

    // (Arithmetic in 64 bits is slow here, and every thread goes through this: c, to
    // 2^-46 of itself, from two divisions in 32.)
    DG_DEVICE void init(float max, float t)
    {
        m = max;
        ch = 1.442695041f / t;
        cl = (fmaf(-ch, t, 1.442695041f) + 1.92596299e-8f) / t;   // log2 e in two parts
        floor = max - 48.f / ch;                         // (2^-45 is the last that counts)
        ref = __float_as_int(fmaf(max, ch, 393216.f));   // 1.5 x 2^18: a unit in the last place is 1/32
        wide = !(fabsf(max) * ch < 65536.f);
    }
    // What the table holds at place p.
    DG_DEVICE uint32_t turned(int p) const { return kExpTable[(p - ref) & 31]; }
    // log2 of what a weight of 2^kWeightBits stands for beside exp((x - max) / T) = 1, at most
    // 1/64 (what the multiply-add cuts off is below 2^-31)
    DG_DEVICE float shift() const
    {
        return wide ? 0.f : -fmaf(m, cl, fmaf(m, ch, 393216.f - __int_as_float(ref)));
    }
    DG_DEVICE uint64_t operator()(float x, const uint32_t *table) const
    {
        return wide ? in_double(x) : fast(x, table);
    }
    // c x to the nearest 1/8, in the last places of a number near 2^20.
    DG_DEVICE float eighths(float x) const { return fmaf(fmaxf(x, floor), ch, kEighths); }
    // Its weight beside that of its nearest eighth, in units of 1 / kMassOne: |r| <= 1/16,
    // the series to r^2 with r^3's nearest line, off by 4e-6 and the rounding.
    DG_DEVICE uint32_t beside(float x, float at) const
    {
        const float r = fmaf(fmaxf(x, floor), ch, kEighths - at);
        const float w = fmaf(r, fmaf(r, 0.24022651f * kMassOne, 0.69330979f * kMassOne), 12582912.f + kMassOne);
        return static_cast<uint32_t>(__float_as_int(w) - __float_as_int(12582912.f));   // (1.5 x 2^23: to a whole number)
    }
    DG_DEVICE uint64_t fast(float x, const uint32_t *table) const
    {
        const float y = fmaxf(x, floor);
        const float P = fmaf(y, ch, 393216.f);
        const int p = __float_as_int(P);
        float r = fmaf(y, ch, 393216.f - P);
        r = fmaf(y, cl, r);
        float s = fmaf(r, 0.055504109f, 0.24022651f);    // ln2^3 / 6, ln2^2 / 2
        s = fmaf(r, s, 0.69314718f);
        const float B = fmaf(r, s, 0.046875f);           // 1.5 x 2^-5: in units of 2^-28
        const uint32_t T = table[p & 31];
        const uint32_t Y = __float_as_uint(B) - (__float_as_uint(0.046875f) - (1u << 28));   // 2^28 (1 + y)
        return static_cast<uint64_t>(T) * Y >> (ref + 31 + 32 * (58 - kWeightBits) - p >> 5);  // (by 13 .. 62)
    }
    DG_DEVICE uint64_t in_double(float x) const { return weight_in_double(x, m, ch, cl); }
};

// a + b and what its rounding cut off
DG_DEVICE float2 two_sum(float a, float b)
{
    const float s = a + b, part = s - a;
    return make_float2(s, (a - (s - part)) + (b - part));
}
// n / d in two floats
DG_DEVICE float2 two_div(float n_hi, float n_lo, float d_hi, float d_lo)
{
    const float q = n_hi / d_hi;
    return make_float2(q, (fmaf(-q, d_lo, fmaf(-q, d_hi, n_hi)) + n_lo) / d_hi);
}

// A drawn token's logprob: (x - m) / t less ln of `all`, of which 2^kWeightBits stands for
// 2^shift of the largest weight.  One thread does this at the end of a row's way, so
// its latency counts: sums of two floats, off by less than 2^-28 beside the result's
// own rounding, in place of arithmetic in 64 bits (1.5 us of a row's 14).  With
// all = 2^n g, g about 1, ln g = 2 (s + s^3 / 3 + ...), s = (g - 1) / (g + 1), |s| < 0.172.
// Where its own weight w is nearly all, from what is left of that, whose rounding the
// result's size bounds: 0 for a token that is kept alone.
__device__ __noinline__ float logprob_of(float x, float m, float t, uint64_t w, uint64_t all, float shift)
{
    if (all - w <= w >> 4) return -log1pf(static_cast<float>(all - w) / static_cast<float>(w));
    constexpr float kLn2 = 0.693145752f, kLn2Low = 1.42860677e-6f;   // (the first: 16 bits)
    int n = 63 - __clzll(static_cast<long long>(all));
    const uint64_t top = all << (63 - n);                            // g 2^63
    float g = static_cast<float>(static_cast<uint32_t>(top >> 40)) * 1.1920929e-7f;
    float low = static_cast<float>(static_cast<uint32_t>(top >> 16) & 0xFFFFFFu) * 7.1054274e-15f;
    if (g > 1.41421354f) {
        g *= 0.5f;
        low *= 0.5f;
        ++n;
    }
    const float2 above = two_sum(g, 1.f);
    const float2 s = two_div(g - 1.f, low, above.x, above.y + low);
    const float q = s.x * s.x;
    const float series = fmaf(q, fmaf(q, fmaf(q, fmaf(q, 0.181818182f, 0.222222222f), 0.285714286f), 0.4f), 0.666666667f);
    // (halves: x - m may be past the largest number)
    const float2 d = two_sum(0.5f * x, -0.5f * m);
    const float2 at = two_div(d.x, d.y, t, 0.f);
    if (!(at.x > -1e37f)) return -INFINITY;
    const float e = static_cast<float>(n - kWeightBits);
    const float2 one = two_sum(2.f * at.x, -e * kLn2);
    const float2 two = two_sum(one.x, -2.f * s.x);
    return two.x + (two.y + one.y + 2.f * at.y - 2.f * s.y - fmaf(e, kLn2Low, fmaf(shift, 0.69314718f, series * q * s.x)));
}

// What a row's CTA hands on to the out-of-line end of its way to a token.
struct Row {
    int row;
    float m, t;                          // its maximum, its temperature within the range
    int turns;                           // parities of the exchange buffers
};
template <class T>
struct Sampler;
// The ends, out of line: a row takes one of them, and the passes of them all in one
// body are more than its registers hold.
template <class T>
__device__ __noinline__ void end_draw(const SampleArgs &a, SampleShared &sh, Row row, float v, int64_t kept,
                                      uint64_t above, uint32_t ties, int buf, float u)
{
    Sampler<T>(a, sh, row).draw_from(v, kept, {above, ties, buf}, u);
}
template <class T>
__device__ __noinline__ void end_listed(const SampleArgs &a, SampleShared &sh, Row row, int n, int k, float p,
                                        uint64_t all, float least, float u)
{
    Sampler<T>(a, sh, row).draw_listed(n, k, p, all, least, u);
}
template <class T>
__device__ __noinline__ void end_counted(const SampleArgs &a, SampleShared &sh, Row row, int k, float p,
                                         float min_value, float u)
{
    Sampler<T>(a, sh, row).draw_counted(k, p, min_value, u);
}
template <class T>
__device__ __noinline__ void end_nucleus(const SampleArgs &a, SampleShared &sh, Row row, float p, float u)
{
    Sampler<T> s(a, sh, row);
    if (!s.draw_nucleus(p, u)) end_counted<T>(a, sh, s.handed(), 0, p, -INFINITY, u);
}

template <class T>
struct Sampler {
    static constexpr int E = Vec<T>::N;
    static constexpr int kGroups = kGroupBytes / sizeof(T);
    static constexpr int kAhead = E == 4 ? 2 : 1;   // 16 bytes that a pass has on their way
    const SampleArgs &a;
    SampleShared &sh;
    const T *base;                       // the row, from the 16 bytes on that it begins in
    int skew;                            // where in them
    const int warp, lane, rank, ctas;
    int turn, hist_turn, sum_turn;
    Weights weight;
    const int row;
    float m, t;
    bool flat;                           // the maximum is infinite: those tokens alone, alike

    DG_DEVICE Sampler(const SampleArgs &args, SampleShared &s, const Row &r)
        : a(args), sh(s), warp(threadIdx.x >> 5), lane(threadIdx.x & 31),
          rank(static_cast<int>(cluster_ctarank())), ctas(args.ctas), turn(r.turns & 1), hist_turn(r.turns >> 1 & 1),
          sum_turn(r.turns >> 2 & 1), row(r.row), m(r.m), t(r.t)
    {
        const int64_t at = row * a.stride;
        skew = static_cast<int>(at & (E - 1));
        base = behind_waits(static_cast<const T *>(a.logits) + (at - skew));
        ready();
    }
    DG_DEVICE void ready()
    {
        flat = m == INFINITY;
        if (!flat) weight.init(m, t);
    }
    // The weights' table, once the maximum is known; before the next barrier.
    DG_DEVICE void lay_table()
    {
        if (threadIdx.x < 32) sh.table[threadIdx.x] = flat ? 0 : weight.turned(static_cast<int>(threadIdx.x));
    }
    DG_DEVICE Row handed() const { return Row{row, m, t, (turn & 1) | (hist_turn & 1) << 1 | (sum_turn & 1) << 2}; }

    DG_DEVICE uint64_t w_of(float x) const
    {
        return flat ? (x == m ? 1ull << kWeightBits : 0) : weight(x, sh.table);
    }
    // The least logit that is ever drawn: further down weights are zeros of 64-bit floats.
    DG_DEVICE float light() const { return flat ? m : fmaf(-745.13f, t, m); }

    // A barrier of the row's threads.
    DG_DEVICE void sync() const
    {
        if (ctas == 1) __syncthreads();
        else cluster_sync_all();
    }

    // 16 bytes of the row (-inf past its ends).  Stream: not to be kept in L1, of which
    // little is left beside the shared memory.  Top-p's passes gain from it (64 fp32 rows of
    // 262144, mixed: 83 -> 73 us; 256, top-p: 354 -> 294), those of fp32 rows do all (maxima
    // 56 -> 54, sums 146 -> 141); the maxima of bf16 rows do not (72 either way), and what
    // follows them is slower (sums 210 -> 220).  As a volatile load, in the order of all
    // other accesses, it costs top-p's passes 8 to 13% (64 fp32 rows of 262144, p = 0.9: 82
    // and 93): what it has to stay behind is the wait for the kernel that wrote the logits.
    template <bool Stream>
    DG_DEVICE static uint4 fetch(const T *p)
    {
        if (!Stream) return __ldg(reinterpret_cast<const uint4 *>(p));
        uint4 v;
        asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
            : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
            : "l"(p));                           // (an address that is known behind the wait alone)
        return v;
    }
    // ... that the row's first or last token is among, or none.
    DG_DEVICE uint4 edge(int first) const
    {
        constexpr uint32_t Low = E == 8 ? 0xFF80FF80u : 0xFF800000u;
        uint4 v = make_uint4(Low, Low, Low, Low);
        if (first + E > skew && first < a.V + skew) {
            alignas(16) T x[E];
            *reinterpret_cast<uint4 *>(x) = v;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (first + e >= skew && first + e < a.V + skew) x[e] = base[first + e];
            v = *reinterpret_cast<const uint4 *>(x);
        }
        return v;
    }
    template <bool Stream = false>
    DG_DEVICE uint4 load(int w, int r, int l) const
    {
        const int first = place(w, r, l, 0);
        return first >= skew && first + E <= a.V + skew ? fetch<Stream>(base + first) : edge(first);
    }
    // The 16 bytes of each row of this thread's warp that are its own: whole ones in rows
    // from .. to - 1.  Fewer instructions a load for more registers: top-p's passes gain
    // (484 -> 469 us on 1024 bf16 rows of 151643), the others lose (maxima 72 -> 74, sums
    // 210 -> 213).
    struct Own {
        const T *p;
        int first, from, to;
    };
    DG_DEVICE Own own() const
    {
        const int first = place(warp, 0, lane, 0), left = a.V + skew - E - first;
        return Own{base + first, first, first < skew ? 1 : 0, left >= 0 ? left / (32 * E) + 1 : 0};
    }
    DG_DEVICE uint4 load(const Own &o, int r) const
    {
        return r >= o.from && r < o.to ? fetch<true>(o.p + r * (32 * E)) : edge(o.first + r * (32 * E));
    }
    // The first token of 16 bytes, `skew` early.
    DG_DEVICE int place(int w, int r, int l, int e) const
    {
        return (((rank * kSampleWarps + w) * a.rows_warp + r) * 32 + l) * E + e;
    }
    DG_DEVICE int rows_group() const { return (a.rows_warp + kGroups - 1) / kGroups; }
    DG_DEVICE T &group(int g) const { return reinterpret_cast<T *>(sh.group)[g * kSampleThreads + threadIdx.x]; }

    // f(16 bytes, row of the warp) for rows r0 .. r1 - 1.
    template <int N, bool Stream, class F>
    DG_DEVICE void rows(int r0, int r1, F f) const
    {
#pragma unroll 1
        for (int r = r0; r < r1; r += N) {
            uint4 v[N];
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (r + e < r1) v[e] = load<Stream>(warp, r + e, lane);
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (r + e < r1) f(v[e], r + e);
        }
    }
    // The same for all rows, N ahead of those at work.
    template <int N, class F, class L>
    DG_DEVICE void rows_ahead(F f, L load_row) const
    {
        uint4 v[N];
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < a.rows_warp) v[e] = load_row(e);
#pragma unroll 1
        for (int r = 0; r < a.rows_warp; r += N) {
            uint4 now[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                now[e] = v[e];
                if (r + N + e < a.rows_warp) v[e] = load_row(r + N + e);
            }
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (r + e < a.rows_warp) f(now[e], r + e);
        }
    }
    // f(x, row of the warp, number in the 16 bytes) for each of this thread's tokens.
    template <class F>
    DG_DEVICE void each(F f) const
    {
        rows<2, false>(0, a.rows_warp, [&](const uint4 &v, int r) {
            float x[E];
            Vec<T>::unpack(v, x);
#pragma unroll
            for (int e = 0; e < E; ++e) f(x[e], r, e);
        });
    }
    // A place in a list for each of a lane's `n` tokens, the first of them; `count`: its
    // length.  By a warp.
    DG_DEVICE uint32_t places(uint32_t n, uint32_t *count) const
    {
        uint32_t end = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(kAll, end, o);
            if (lane >= o) end += x;
        }
        uint32_t first = 0;
        if (lane == 31 && end > 0) first = atomicAdd(count, end);
        return __shfl_sync(kAll, first, 31) + end - n;
    }
    // The 16 bytes of the groups whose maximum is wanted, listed; how many they are.  Once
    // a row.
    template <class W>
    DG_DEVICE int pick(W wanted)
    {
        uint16_t *todo = reinterpret_cast<uint16_t *>(sh.mass);
        static_assert(sizeof(sh.mass) >= kGroups * kSampleThreads * sizeof(uint16_t), "a place for every group");
        uint32_t want = 0;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) want |= wanted(Vec<T>::widen(group(g))) ? 1u << g : 0u;
        uint32_t slot = places(__popc(want), &sh.todo);
        for (; want != 0; want &= want - 1)
            todo[slot++] = static_cast<uint16_t>((__ffs(want) - 1) * kSampleThreads + threadIdx.x);
        __syncthreads();
        return static_cast<int>(sh.todo) * rows_group();
    }
    // f(N of those from place x0 on, a thread's, and where they are: warp, row, lane; where
    // there is none 16 bytes of -inf), shared out evenly; a warp's threads go together.
    template <int N, class F>
    DG_DEVICE void picked(int n, F f)
    {
        const uint16_t *todo = reinterpret_cast<const uint16_t *>(sh.mass);
        const int rg = rows_group();
#pragma unroll 1
        for (int x0 = warp * 32; x0 < n; x0 += N * kSampleThreads) {
            uint4 v[N];
            int w[N], r[N], l[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                constexpr uint32_t Low = E == 8 ? 0xFF80FF80u : 0xFF800000u;
                v[e] = make_uint4(Low, Low, Low, Low);
                const int x = x0 + lane + e * kSampleThreads;
                w[e] = r[e] = l[e] = 0;
                if (x >= n) continue;
                const int at = x / rg, id = todo[at];
                r[e] = id / kSampleThreads * rg + x - at * rg;
                w[e] = id % kSampleThreads / 32;
                l[e] = id % 32;
                if (r[e] < a.rows_warp) v[e] = load(w[e], r[e], l[e]);
            }
            f(v, w, r, l);
        }
    }
    // The tokens that are wanted, listed.
    template <class W>
    DG_DEVICE void list_of(W wanted)
    {
        constexpr int N = 4;
        picked<N>(pick(wanted), [&](const uint4 (&v)[N], const int (&w)[N], const int (&r)[N], const int (&l)[N]) {
            uint32_t hits = 0;                       // of N * E tokens
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float x[E];
                Vec<T>::unpack(v[i], x);
#pragma unroll
                for (int e = 0; e < E; ++e) hits |= wanted(x[e]) ? 1u << (i * E + e) : 0u;
            }
            if (!__any_sync(kAll, hits != 0)) return;
            uint32_t slot = places(__popc(hits), &sh.listed);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                for (uint32_t h = hits >> (i * E) & ((1u << E) - 1u); h != 0; h &= h - 1) {
                    const int e = __ffs(h) - 1;
                    if (slot < kList)
                        sh.list[slot] = static_cast<uint64_t>(~order_of(Vec<T>::at(v[i], e))) << 32 |
                                        static_cast<uint32_t>(place(w[i], r[i], l[i], e));
                    ++slot;
                }
            }
        });
    }

    // The largest of two values over the row's threads.
    DG_DEVICE uint2 largest(uint32_t x, uint32_t y)
    {
        x = __reduce_max_sync(kAll, x);
        y = __reduce_max_sync(kAll, y);
        uint64_t *got = sh.gather[turn++ & 1];
        const int at = rank * kSampleWarps + warp;
        const uint64_t both = static_cast<uint64_t>(y) << 32 | x;
        if (ctas == 1) {
            if (lane == 0) got[at] = both;
        } else if (lane < ctas) {
            st_cluster64(mapa_shared(smem_u32(got + at), lane), both);
        }
        sync();
        x = y = 0;
        for (int k = lane; k < ctas * kSampleWarps; k += 32) {
            x = max(x, static_cast<uint32_t>(got[k]));
            y = max(y, static_cast<uint32_t>(got[k] >> 32));
        }
        return make_uint2(__reduce_max_sync(kAll, x), __reduce_max_sync(kAll, y));
    }

    // ------------------------------------------------------------ a histogram over the row
    DG_DEVICE uint32_t *clear()
    {
        uint32_t *hist = sh.hist[hist_turn & 1];
        for (int k = threadIdx.x; k < kBins; k += kSampleThreads) hist[k] = 0;
        __syncthreads();
        return hist;
    }
    // The bin in which the tokens reach `target` in number, or with `Mass` (counts
    // weighed by of_bin) each of N weights, part[i] of `of` (of < 0: of all of theirs)
    // less `less`; where rounded sums stay short of that, the last one that is not empty.
    // Into sh.found[i].  Bins: of those that are in use.
    template <bool Mass, int Bins, int N, class F>
    DG_DEVICE void find_each(uint32_t target, const float (&part)[N], float of, float less, F of_bin)
    {
        const int buf = hist_turn++ & 1;
        if (threadIdx.x == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) sh.claim[i] = kSampleThreads;
            sh.last = -1;
        }
        sync();
        const int b = kBinsThread * threadIdx.x;
        uint32_t n[kBinsThread];
        float f[kBinsThread];
#pragma unroll
        for (int e = 0; e < kBinsThread; ++e) n[e] = 0;
        if (b >= Bins) {
        } else if (ctas == 1) {
            const uint4 v = *reinterpret_cast<const uint4 *>(&sh.hist[buf][b]);
            n[0] = v.x, n[1] = v.y, n[2] = v.z, n[3] = v.w;
        } else {
            constexpr int Ahead = 8;
            const uint32_t at = smem_u32(&sh.hist[buf][b]);
            for (int k0 = 0; k0 < ctas; k0 += Ahead) {
                uint4 v[Ahead];
#pragma unroll
                for (int k = 0; k < Ahead; ++k) {
                    v[k] = make_uint4(0, 0, 0, 0);
                    if (k0 + k < ctas) v[k] = ld_cluster4(mapa_shared(at, k0 + k));
                }
#pragma unroll
                for (int k = 0; k < Ahead; ++k) {
                    n[0] += v[k].x;
                    n[1] += v[k].y;
                    n[2] += v[k].z;
                    n[3] += v[k].w;
                }
            }
        }
        uint32_t n_sum = 0;
        float f_sum = 0.f;
#pragma unroll
        for (int e = 0; e < kBinsThread; ++e) {
            f[e] = Mass && n[e] > 0 ? n[e] * of_bin(b + e) : 0.f;
            n_sum += n[e];
            f_sum += f[e];
        }
        uint32_t n_end = n_sum;
        float f_end = f_sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t un = __shfl_up_sync(kAll, n_end, o);
            const float uf = __shfl_up_sync(kAll, f_end, o);
            if (lane >= o) {
                n_end += un;
                f_end += uf;
            }
        }
        if (lane == 31) {
            sh.scan_u[warp] = n_end;
            sh.scan_f[warp] = f_end;
        }
        __syncthreads();
        float f_all = 0.f;
        uint32_t n_all = 0;
#pragma unroll
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w < warp) {
                n_end += sh.scan_u[w];
                f_end += sh.scan_f[w];
            }
            f_all += sh.scan_f[w];
            n_all += sh.scan_u[w];
        }
        float aim[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            aim[i] = part[i] * (of < 0.f ? f_all : of) - less;
            if (n_sum > 0 && (Mass ? f_end >= aim[i] : n_end >= target))
                atomicMin(&sh.claim[i], static_cast<int>(threadIdx.x));
        }
        if (Mass && n_sum > 0) atomicMax(&sh.last, static_cast<int>(threadIdx.x));
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool reached = sh.claim[i] < kSampleThreads;
            if (static_cast<int>(threadIdx.x) != (reached ? sh.claim[i] : max(sh.last, 0))) continue;
            Found got{-1, 0, 0, n_all, 0.f, f_all, reached};
            uint32_t n_before = n_end - n_sum;
            float f_before = f_end - f_sum;
            bool stop = false;
#pragma unroll
            for (int e = 0; e < kBinsThread; ++e) {
                if (n[e] > 0 && !stop) {
                    got = Found{b + e, n[e], n_before, n_all, f_before, f_all, reached};
                    stop = reached && (Mass ? f_before + f[e] >= aim[i] : n_before + n[e] >= target);
                }
                n_before += n[e];
                f_before += f[e];
            }
            if (!reached && !Mass) got.bin = -1;
            sh.found[i] = got;
        }
        __syncthreads();
    }
    template <bool Mass, class F>
    DG_DEVICE Found find(uint32_t target, float target_mass, F of_bin)
    {
        const float part[1] = {target_mass};
        find_each<Mass, kBins>(target, part, 1.f, 0.f, of_bin);
        return sh.found[0];
    }

    // Where the tokens reach k in number or, with `Mass`, `target` in weight, of those
    // from `floor_v` on.  Tokens too light to be drawn do not count; none: there are too few.
    // With `Mass` it may be one of the cut's neighbours (the weights are rounded).
    template <bool Mass>
    DG_DEVICE Cut select(uint32_t k, float target, float floor_v)
    {
        const float s1 = weight.ch * kBinsLog2;
        auto y_of = [&](float x) -> float { return (m - x) * s1; };
        uint32_t *hist = clear();
        each([&](float x, int, int) {
            const float y = y_of(x);
            if (!(x >= floor_v) || !(y < static_cast<float>(kBins))) return;
            const int b = static_cast<int>(y);
            uint32_t inc = 1;
            if (Mass) {
                // its weight beside that of the bin's upper end, 2^(-f / 16)
                const float f = y - static_cast<float>(b);
                inc = static_cast<uint32_t>(fmaf(fmaf(f, fmaf(f, 9.3838e-4f, -0.0433217f), 1.f), kMassOne, 0.5f));
            }
            atomicAdd(hist + b, inc);
        });
        const Found f1 =
            find<Mass>(k, target, [&](int b) -> float { return exp2f(-b / kBinsLog2) * (1.f / kMassOne); });
        // Past the last bin, 64 factors of 2 below the largest, tokens add nothing to a sum of
        // weights, but they are of the first k: those are found by their bits alone.
        const bool past = !Mass && f1.bin < 0;
        if (f1.bin < 0 && !past) return Cut{-INFINITY, 0, 0};
        // else that bin's tokens by their place in it
        const float b1 = static_cast<float>(f1.bin);
        auto y2_of = [&](float y) -> int { return min(static_cast<int>((y - b1) * kBins), kBins - 1); };
        auto inside = [&](float x, float y) -> bool {
            return x >= floor_v && y < static_cast<float>(kBins) && static_cast<int>(y) == f1.bin;
        };
        uint32_t before = Mass ? 0 : f1.before;
        float above = f1.mass;
        Found f2{};
        if (past) {
            floor_v = fmaxf(floor_v, fmaxf(light(), -FLT_MAX));
            before = f1.total;
        } else {
            hist = clear();
            each([&](float x, int, int) {
                const float y = y_of(x);
                if (inside(x, y)) atomicAdd(hist + y2_of(y), 1u);
            });
            f2 = find<Mass>(k - before, target - above, [&](int b) -> float {
                return exp2f(-(b1 + (static_cast<float>(b) + 0.5f) * (1.f / kBins)) / kBinsLog2);
            });
            if (f2.bin < 0) return Cut{-INFINITY, 0, 0};
            before += f2.before;
            above += f2.mass;
        }
        // and by their bits
        uint32_t hi = 0, lo = 0, ties = f2.count;
        each([&](float x, int, int) {
            const float y = y_of(x);
            if (past ? x >= floor_v && !(y < static_cast<float>(kBins)) : inside(x, y) && y2_of(y) == f2.bin) {
                hi = max(hi, order_of(x));
                lo = max(lo, ~order_of(x));
            }
        });
        const uint2 ends = largest(hi, lo);
        hi = ends.x;
        lo = ~ends.y;
        if (hi < lo) return Cut{-INFINITY, 0, 0};            // (none past the last bin)
        while (hi > lo || past) {                            // (those have not been counted)
            const int shift = max(0, 22 - __clz(hi - lo));
            hist = clear();
            each([&](float x, int, int) {
                if (!(x >= floor_v)) return;
                const uint32_t o = order_of(x);
                if (o <= hi && o >= lo) atomicAdd(hist + ((hi - o) >> shift), 1u);
            });
            const Found f3 = find<Mass>(k - before, target - above, [&](int b) -> float {
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
        return Cut{of_order(hi), Mass ? ties : k - before, ties};
    }

    // ------------------------------------------------------------ exact sums
    struct Sums {
        uint64_t above;                   // weight above the cut
        uint32_t ties;                    // tokens at the cut
        int buf;
    };
    // Hands a lane's sums out by segment (a warp's stretch of the row) and adds them up;
    // with Whole another one, whose sum alone is wanted.
    template <bool Whole = false>
    DG_DEVICE Sums gather(uint64_t above, uint32_t ties, uint64_t *whole = nullptr, uint64_t more_above = 0)
    {
        above += more_above;
        ties = __reduce_add_sync(kAll, ties);
        uint64_t more = Whole ? *whole : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            above += __shfl_xor_sync(kAll, above, o);
            if (Whole) more += __shfl_xor_sync(kAll, more, o);
        }
        const int buf = sum_turn++ & 1;
        const int at = rank * kSampleWarps + warp;
        if (lane < ctas) {
            st_cluster64(mapa_shared(smem_u32(&sh.above[buf][at]), lane), above);
            if (Whole) st_cluster64(mapa_shared(smem_u32(&sh.whole[at]), lane), more);
            st_cluster32(mapa_shared(smem_u32(&sh.ties[buf][at]), lane), ties);
        }
        sync();
        above = more = 0;
        ties = 0;
        for (int k = lane; k < ctas * kSampleWarps; k += 32) {
            above += sh.above[buf][k];
            if (Whole) more += sh.whole[k];
            ties += sh.ties[buf][k];
        }
        ties = __reduce_add_sync(kAll, ties);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            above += __shfl_xor_sync(kAll, above, o);
            if (Whole) more += __shfl_xor_sync(kAll, more, o);
        }
        if (Whole) *whole = more;
        return Sums{above, ties, buf};
    }
    // Of the whole row.
    DG_DEVICE Sums sums_all()
    {
        uint64_t above = 0;
        if (flat || weight.wide) {
            each([&](float x, int, int) { above += w_of(x); });
        } else {
            rows_ahead<kAhead>([&](const uint4 &v, int) {
                float x[E];
                Vec<T>::unpack(v, x);
#pragma unroll
                for (int e = 0; e < E; ++e) above += weight.fast(x[e], sh.table);
            }, [&](int r) -> uint4 { return load<E == 4>(warp, r, lane); });
        }
        return gather(above, 0);
    }
    // Above v; and the tokens at v.
    DG_DEVICE Sums sums(float v)
    {
        uint64_t above = 0;
        uint32_t ties = 0;
        rows<2, false>(0, a.rows_warp, [&](const uint4 &raw, int) {
            float x[E];
            Vec<T>::unpack(raw, x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ties += x[e] == v ? 1u : 0u;
                if (x[e] > v) above += w_of(x[e]);
            }
        });
        if (v == -INFINITY) ties = 0;     // (those past the row's end)
        return gather(above, ties);
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
        const uint64_t mine = above + w * static_cast<uint64_t>(left <= 0 ? 0 : left < ties ? left : ties);
        uint64_t end = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(kAll, end, o);
            if (lane >= o) end += x;
        }
        // (all of them weigh more than rem: the parts' sums are exact)
        const int at = __ffs(__ballot_sync(kAll, end > rem) | 1u << 31) - 1;
        rem -= __shfl_sync(kAll, end - mine, at);
        tie_prefix += __shfl_sync(kAll, before, at);
        return at;
    }
    // The same of up to 1024 parts, a lane taking a stretch of them first.
    DG_DEVICE int locate_of(const uint64_t *aboves, const uint32_t *tie_counts, int n, uint64_t w, int64_t kept,
                            uint64_t &rem, int &tie_prefix)
    {
        const int per = (n + 31) / 32;
        uint64_t above = 0;
        uint32_t ties = 0;
        for (int k = lane * per; k < min(n, (lane + 1) * per); ++k) {
            above += aboves[k];
            ties += tie_counts[k];
        }
        const int at = per > 1 ? locate(above, ties, w, kept, rem, tie_prefix) : 0;
        const int k = at * per + lane;
        const bool mine = (per == 1 || lane < per) && k < n;
        return at * per + locate(mine ? aboves[k] : 0, mine ? tie_counts[k] : 0, w, kept, rem, tie_prefix);
    }

    // The token in which `rem` of the kept weight `all` falls, in the order of the
    // vocabulary: by the CTA that has it.  kept: how many of those at v are.
    DG_DEVICE void draw(float v, int64_t kept, const Sums &s, uint64_t rem, uint64_t all)
    {
        if (warp == 0) {
            const uint64_t wv = v > -INFINITY ? w_of(v) : 0;
            int prefix = 0;
            const int seg = locate_of(sh.above[s.buf], sh.ties[s.buf], ctas * kSampleWarps, wv, kept, rem, prefix);
            if (lane == 0) {
                sh.seg = seg;
                sh.rem = rem;
                sh.tie_prefix = prefix;
            }
        }
        __syncthreads();
        draw_segment(v, kept, all);
    }
    // The rest of it, once segment, remainder and ties before are in shared memory.
    DG_DEVICE void draw_segment(float v, int64_t kept, uint64_t all)
    {
        if (sh.seg / kSampleWarps != rank) return;
        const uint64_t wv = v > -INFINITY ? w_of(v) : 0;
        const int seg = sh.seg % kSampleWarps;
        auto row_of = [&](int r, uint64_t &above, uint32_t &ties, float (&x)[E]) {
            Vec<T>::unpack(load(seg, r, lane), x);
            above = 0;
            ties = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (x[e] > v) above += w_of(x[e]);
                ties += x[e] == v && v > -INFINITY ? 1u : 0u;
            }
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
        uint64_t rem = sh.rem;
        int prefix = sh.tie_prefix;
        const int r = locate_of(sh.row_above, sh.row_ties, a.rows_warp, wv, kept, rem, prefix);
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
            if (sum > rem) break;
        }
        say(token, value, w_of(value), all);
    }

    // The draw from all that lies above v and `kept` of the tokens at v, summed by s.
    DG_DEVICE void draw_from(float v, int64_t kept, const Sums &s, float u)
    {
        const uint64_t all = s.above + (v > -INFINITY ? w_of(v) : 0) * kept;
        const uint64_t rem = min(u < 1.f ? part_of(all, u, false) : all - 1, all - 1);
        if (rem > 0) {
            draw(v, kept, s, rem, all);
            return;
        }
        // the first that is kept and weighs anything
        uint32_t best = 0;
        float value = 0.f;
        each([&](float x, int r, int e) {
            const uint32_t at = ~static_cast<uint32_t>(place(warp, r, lane, e));
            if ((x > v || (x == v && kept > 0)) && x >= light() && at > best) {
                best = at;
                value = x;
            }
        });
        const uint32_t mine = best;
        best = largest(best, 0).x;
        if (mine == best && best != 0) say(static_cast<int>(~best) - skew, value, w_of(value), all);   // (one has it)
    }

    // w: its weight in the sums' units, as it is counted in `all`.
    DG_DEVICE void say(int token, float value, uint64_t w, uint64_t all) const
    {
        a.token[row] = token;
        if (a.logprob == nullptr) return;
        if (flat) a.logprob[row] = logprob_of(0.f, 0.f, 1.f, w, all, 0.f);
        else a.logprob[row] = logprob_of(value, m, t, w, all, weight.shift());
    }

    // ------------------------------------------------------------ few tokens
    // Sums up to and with each thread's, over the block; *all: of all threads.
    DG_DEVICE uint64_t scan(uint64_t v, uint64_t *all)
    {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t x = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += x;
        }
        __syncthreads();
        if (lane == 31) sh.red[warp] = v;
        __syncthreads();
        uint64_t sum = 0;
#pragma unroll
        for (int w = 0; w < kSampleWarps; ++w) {
            if (w == warp) v += sum;
            sum += sh.red[w];
        }
        *all = sum;
        return v;
    }

    // The n keys of the list in rising order: counted into bins (bin_of rises with the
    // key), put there, and each to its place among its bin's.
    template <class F>
    DG_DEVICE void sort(int n, F bin_of)
    {
        uint32_t *end = sh.hist[0];
        for (int k = threadIdx.x; k < kBins; k += kSampleThreads) end[k] = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < n; e += kSampleThreads) atomicAdd(end + bin_of(sh.list[e]), 1u);
        __syncthreads();
        uint32_t c[kBinsThread], sum = 0;
#pragma unroll
        for (int e = 0; e < kBinsThread; ++e) {
            c[e] = end[kBinsThread * threadIdx.x + e];
            sum += c[e];
        }
        uint64_t ignored;
        uint32_t at = static_cast<uint32_t>(scan(sum, &ignored)) - sum;
#pragma unroll
        for (int e = 0; e < kBinsThread; ++e) {
            end[kBinsThread * threadIdx.x + e] = at;
            at += c[e];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n; e += kSampleThreads) {
            const uint64_t key = sh.list[e];
            sh.moved[atomicAdd(end + bin_of(key), 1u)] = key;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n; e += kSampleThreads) {
            const uint64_t key = sh.moved[e];
            const int b = bin_of(key);
            const uint32_t first = b > 0 ? end[b - 1] : 0, last = end[b];
            uint32_t rank_in = first;
            for (uint32_t o = first; o < last; ++o) rank_in += sh.moved[o] < key ? 1 : 0;
            sh.list[rank_in] = key;
        }
        __syncthreads();
    }
    DG_DEVICE static float value_of(uint64_t key) { return of_order(~static_cast<uint32_t>(key >> 32)); }
    // ... of n listed tokens: falling value, rising index.
    DG_DEVICE void sort_values(int n)
    {
        uint32_t hi = 0, lo = 0;
        for (int e = threadIdx.x; e < n; e += kSampleThreads) {
            const uint32_t o = ~static_cast<uint32_t>(sh.list[e] >> 32);
            hi = max(hi, o);
            lo = max(lo, ~o);
        }
        hi = __reduce_max_sync(kAll, hi);
        lo = __reduce_max_sync(kAll, lo);
        if (lane == 0) sh.red[warp] = static_cast<uint64_t>(lo) << 32 | hi;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSampleWarps; ++w) {
            hi = max(hi, static_cast<uint32_t>(sh.red[w]));
            lo = max(lo, static_cast<uint32_t>(sh.red[w] >> 32));
        }
        const float top = of_order(hi), scale = static_cast<float>(kBins) / (top - of_order(~lo));
        sort(n, [&](uint64_t key) -> int {       // (equal ones only: 0 x infinity, the first bin)
            return min(max(static_cast<int>((top - value_of(key)) * scale), 0), kBins - 1);
        });
    }

    // The draw from the n listed tokens, which hold all that is kept, by one CTA: of the
    // first k (k > 0), top-p's part p of their weight or (k == 0) of `all`, and not below
    // `least`.
    DG_DEVICE void draw_listed(int n, int k, float p, uint64_t all, float least, float u)
    {
        least = fmaxf(least, light());
        if (n <= kSampleThreads) {
            draw_few(n, k, p, all, least, u);
            return;
        }
        sort_values(n);
        const int most = k > 0 ? min(k, n) : n;
        // the weights in that order and their sums; a thread has `per` neighbours
        int per = (most + kSampleThreads - 1) / kSampleThreads, first = threadIdx.x * per;
        uint64_t sum = 0, listed, part;
        for (int e = first; e < min(first + per, most); ++e) {
            const uint64_t w = w_of(value_of(sh.list[e]));
            sh.mass[e] = w;
            sum += w;
        }
        uint64_t before = scan(sum, &listed) - sum;
        const uint64_t need = p < 1.f ? part_of(k > 0 ? listed : all, p, true) : ~0ull;
        // how many of them are kept, and what those weigh
        uint64_t mine = 0, count = 0;
        for (int e = first; e < min(first + per, most); ++e) {
            if (e == 0 || (before < need && value_of(sh.list[e]) >= least)) {
                ++count;
                mine += sh.mass[e];
            }
            before += sh.mass[e];
        }
        scan(mine, &part);
        uint64_t number;
        scan(count, &number);
        const int kept = static_cast<int>(number);
        uint64_t rem = min(u < 1.f ? part_of(part, u, false) : part - 1, part - 1);
        // in the vocabulary's order: an index, the place in the first order beside it
        for (int e = threadIdx.x; e < kept; e += kSampleThreads)
            sh.list[e] = sh.list[e] << 32 | static_cast<uint32_t>(e);
        __syncthreads();
        const float per_bin = static_cast<float>(kBins) / static_cast<float>(a.V + E);
        sort(kept, [&](uint64_t key) -> int {
            return min(static_cast<int>(static_cast<float>(static_cast<uint32_t>(key >> 32)) * per_bin), kBins - 1);
        });
        per = (kept + kSampleThreads - 1) / kSampleThreads;
        first = threadIdx.x * per;
        sum = 0;
        for (int e = first; e < min(first + per, kept); ++e) sum += sh.mass[static_cast<uint32_t>(sh.list[e])];
        uint64_t at = scan(sum, &listed) - sum;
        for (int e = first; e < min(first + per, kept); ++e) {
            const uint64_t w = sh.mass[static_cast<uint32_t>(sh.list[e])];
            // (rem == 0: the first one, however light)
            if (rem == 0 ? e == 0 : at <= rem && rem < at + w) {
                const int place = static_cast<int>(sh.list[e] >> 32);
                say(place - skew, Vec<T>::widen(base[place]), w, part);
            }
            at += w;
        }
    }

    // The same for at most a token a thread: its place in either order is the number of
    // those before it, counted out.
    DG_DEVICE void draw_few(int n, int k, float p, uint64_t all, float least, float u)
    {
        const int e = threadIdx.x;
        uint64_t key = 0;
        if (e < n) {
            key = sh.list[e];
            int before = 0;
#pragma unroll 8
            for (int o = 0; o < n; ++o) before += sh.list[o] < key ? 1 : 0;
            sh.moved[before] = key;
            sh.mass[before] = w_of(value_of(key));
        }
        __syncthreads();
        const int most = k > 0 ? min(k, n) : n;
        uint64_t w = 0, listed;
        if (e < n) key = sh.moved[e];
        if (e < most) w = sh.mass[e];
        const uint64_t before = scan(w, &listed) - w;
        const uint64_t need = p < 1.f ? part_of(k > 0 ? listed : all, p, true) : ~0ull;
        const bool keeps = e < most && (e == 0 || (before < need && value_of(key) >= least));
        uint32_t *index = reinterpret_cast<uint32_t *>(sh.list);
        const uint32_t at = keeps ? static_cast<uint32_t>(key) : ~0u;
        index[e] = at;                           // (nobody looks at the list any more)
        const int kept = __syncthreads_count(keeps);
        if (e == kept - 1) sh.all = before + w;
        __syncthreads();
        if (!keeps) return;
        const uint64_t part = sh.all;
        const uint64_t rem = min(u < 1.f ? part_of(part, u, false) : part - 1, part - 1);
        uint64_t sum = 0;
        bool first = true;
#pragma unroll 8
        for (int o = 0; o < kept; ++o) {
            const bool lower = index[o] < at;
            sum += lower ? sh.mass[o] : 0;
            first &= !lower;
        }
        // (rem == 0: the first one, however light)
        if (rem == 0 ? first : sum <= rem && rem < sum + w) say(static_cast<int>(at) - skew, value_of(key), w, part);
    }

    // Lists a thread's hits among 16 bytes' tokens.
    DG_DEVICE void list(const float (&x)[E], uint32_t hits, int w, int r, int l)
    {
        if (hits == 0) return;
        uint32_t slot = atomicAdd(&sh.listed, static_cast<uint32_t>(__popc(hits)));
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (!(hits >> e & 1u)) continue;
            if (slot < kList)
                sh.list[slot] = static_cast<uint64_t>(~order_of(x[e])) << 32 | static_cast<uint32_t>(place(w, r, l, e));
            ++slot;
        }
    }
    // All that the row's CTAs have listed to the first one; how many that are (more than
    // kList: they are not all there).
    DG_DEVICE int join_lists()
    {
        __syncthreads();
        if (ctas == 1) return static_cast<int>(sh.listed);
        const uint32_t to_count = mapa_shared(smem_u32(&sh.listed), 0);
        if (rank != 0) {
            const uint32_t n = sh.listed;
            if (threadIdx.x == 0) sh.base = add_cluster32(to_count, n);
            __syncthreads();
            const uint32_t to_list = mapa_shared(smem_u32(sh.list), 0), at = sh.base;
            for (uint32_t e = threadIdx.x; e < min(n, static_cast<uint32_t>(kList)); e += kSampleThreads)
                if (at + e < kList) st_cluster64(to_list + 8 * (at + e), sh.list[e]);
        }
        __syncwarp();
        cluster_sync_all();
        return static_cast<int>(ld_cluster32(to_count));
    }

    // ------------------------------------------------------------ top-p alone
    DG_DEVICE int sub_bin(float x, float top, float scale) const
    {
        return min(max(static_cast<int>(fmaf(-x, weight.ch, top) * scale), 0), kBins - 1);
    }
    // The part p of the row's weight.  The weights, rounded, are summed in bins, by their
    // logarithm's nearest 1/8, a place a lane so that no two meet; then the whole weight
    // exactly, and of the tokens above the bins that the cut may lie in, which are listed
    // and sorted by the first CTA.  False: the row has to go the long way.
    DG_DEVICE bool draw_nucleus(float p, float u)
    {
        constexpr float kSlack = 2e-4f;          // (the bins' weights are off by less than 1e-4)
        if (weight.wide) return false;
        uint32_t *lanes = &sh.hist[0][0];        // [bin][lane]
        static_assert(offsetof(SampleShared, hist) == 0 && offsetof(SampleShared, gather) >= kMassBins * 32 * 4,
                      "hist, list and mass are the bins' room");
        static_assert(kMassBins == kSampleThreads, "a thread adds a bin up");
        for (int k = threadIdx.x; k < kMassBins * 32; k += kSampleThreads) lanes[k] = 0;
        __syncthreads();
        const float ref = weight.eighths(m);
        const Own mine_rows = own();
        auto load_row = [&](int r) -> uint4 { return load(mine_rows, r); };
        rows_ahead<kAhead>([&](const uint4 &v, int) {
            float x[E];
            Vec<T>::unpack(v, x);
#pragma unroll
            for (int e = 0; e < E; ++e) {        // (no branch: the tokens' latencies overlap)
                const float at = weight.eighths(x[e]);
                const int b = __float_as_int(ref) - __float_as_int(at);
                const uint32_t w = weight.beside(x[e], at);
                atomicAdd(lanes + min(b, kMassBins - 1) * 32 + lane, b < kMassBins ? w : 0);
            }
        }, load_row);
        __syncthreads();
        uint32_t mine = 0;
#pragma unroll 8
        for (int l = 0; l < 32; ++l) mine += lanes[threadIdx.x * 32 + ((l + lane) & 31)];   // (spread over the banks)
        __syncthreads();
        uint32_t *hist = sh.hist[hist_turn & 1];
        hist[threadIdx.x] = mine;
        auto of_bin = [](int b) -> float { return exp2f(-b / 8.f) * (1.f / kMassOne); };
        const float parts[2] = {p * (1.f + kSlack), p * (1.f - kSlack)};
        find_each<true, kMassBins>(0, parts, -1.f, 0.f, of_bin);
        const Found hi = sh.found[0];
        if (!hi.reached) return false;
        // (a token's rounded weight is at least 0.95 of kMassOne, at most 1.05)
        const bool all_listed = hi.before + hi.count < static_cast<uint32_t>(kMassOne * 0.85f * kList);
        int from = 0, first_sub = 0, last_sub = kBins - 1;
        float mass_from = 0.f;                   // (rounded, above bin `from`)
        float top = 0.f, scale = 0.f;            // bins of the bins: their upper end, how many to a factor of 2
        auto of_sub = [&](int b) -> float {
            return exp2f(top - (ref - kEighths) - (static_cast<float>(b) + 0.5f) / scale);
        };
        bool split = false;                      // the bins hold more than the CTAs can list
        const float last_at = ref - static_cast<float>(hi.bin) / 8.f;
        float first_at = INFINITY;               // (of the bins `from` and hi.bin)
        if (!all_listed) {
            const Found lo = sh.found[1];
            from = lo.bin;
            first_at = ref - static_cast<float>(from) / 8.f;
            mass_from = lo.mass;
            top = ref - kEighths - static_cast<float>(from) / 8.f + 0.0625f;
            scale = kBins * 8.f / static_cast<float>(hi.bin - from + 2);
            split = hi.before + hi.count - lo.before > static_cast<uint32_t>(kMassOne * 0.65f * kList) * ctas;
            if (split) {
                hist = clear();
                rows_ahead<kAhead>([&](const uint4 &v, int) {
                    float x[E];
                    Vec<T>::unpack(v, x);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float at = weight.eighths(x[e]);
                        if (at <= first_at && at >= last_at) atomicAdd(hist + sub_bin(x[e], top, scale), 1u);
                    }
                }, load_row);
                find_each<true, kBins>(0, parts, hi.all, mass_from, of_sub);
                const Found hi2 = sh.found[0], lo2 = sh.found[1];
                if (!hi2.reached || hi2.before + hi2.count - lo2.before > kList) return false;
                first_sub = lo2.bin;
                last_sub = hi2.bin;
            }
        }
        uint64_t above = 0, all = 0, listed_above = 0;
        rows_ahead<kAhead>([&](const uint4 &v, int r) {
            float x[E];
            Vec<T>::unpack(v, x);
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const uint64_t w = weight.fast(x[e], sh.table);
                all += w;
                const float at = weight.eighths(x[e]);
                above += at > first_at ? w : 0;
                hits |= at <= first_at && at >= last_at ? 1u << e : 0u;
            }
            if (split && hits != 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!(hits >> e & 1u)) continue;
                    const int sub = sub_bin(x[e], top, scale);
                    if (sub >= first_sub && sub <= last_sub) continue;
                    hits &= ~(1u << e);
                    if (sub < first_sub) above += weight.fast(x[e], sh.table);
                }
            }
            list(x, hits, warp, r, lane);
        }, load_row);
        if (!all_listed && !split) {
            // Each CTA has its part of the bins' tokens; those that the cut cannot be among
            // are told apart by bins of their own, and leave the list.
            hist = clear();
            const int n = static_cast<int>(min(sh.listed, static_cast<uint32_t>(kList)));
            const bool lost = sh.listed > kList;
            for (int e = threadIdx.x; e < n; e += kSampleThreads)
                atomicAdd(hist + sub_bin(value_of(sh.list[e]), top, scale), 1u);
            find_each<true, kBins>(0, parts, hi.all, mass_from, of_sub);
            const Found hi2 = sh.found[0], lo2 = sh.found[1];
            if (largest(lost ? 1 : 0, 0).x != 0 || !hi2.reached) return false;
            if (threadIdx.x < kSampleWarps) sh.mass[threadIdx.x] = 0;
            __syncthreads();
            const uint32_t size = E * 32 * a.rows_warp;
            uint64_t key[kList / kSampleThreads];
#pragma unroll
            for (int e = 0; e < kList / kSampleThreads; ++e) {
                const int at = e * kSampleThreads + threadIdx.x;
                key[e] = at < n ? sh.list[at] : 0;
                if (at >= n) continue;
                const float x = value_of(key[e]);
                const int b = sub_bin(x, top, scale);
                if (b >= lo2.bin && b <= hi2.bin) continue;
                if (b < lo2.bin)                 // above them after all
                    atomicAdd(reinterpret_cast<unsigned long long *>(sh.mass) +
                                  (static_cast<uint32_t>(key[e]) / size - rank * kSampleWarps),
                              static_cast<unsigned long long>(w_of(x)));
                key[e] = 0;
            }
            __syncthreads();
            if (threadIdx.x == 0) sh.listed = 0;
            if (lane == 0) listed_above = sh.mass[warp];
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kList / kSampleThreads; ++e)
                if (key[e] != 0) sh.list[atomicAdd(&sh.listed, 1u)] = key[e];
        }
        const Sums s = gather<true>(above, 0, &all, listed_above);
        const int n = join_lists();
        if (n <= kList && n > 0 && all_listed) {
            if (rank == 0) end_listed<T>(a, sh, handed(), n, 0, p, all, -INFINITY, u);
            return true;
        }
        if (n > kList || n == 0) return false;
        const uint64_t need = part_of(all, p, true);
        if (rank == 0) {
            // the segments' weights are kept where the sort leaves them
            uint64_t *segment = sh.gather[0];
            for (int k = threadIdx.x; k < ctas * kSampleWarps; k += kSampleThreads) segment[k] = sh.above[s.buf][k];
            if (threadIdx.x == 0) sh.cut = Cut{-INFINITY, 0, 0};
            sort_values(n);
            const int per = (n + kSampleThreads - 1) / kSampleThreads, first = threadIdx.x * per;
            uint64_t sum = 0, listed;
            for (int e = first; e < min(first + per, n); ++e) sum += w_of(value_of(sh.list[e]));
            uint64_t before = s.above + scan(sum, &listed) - sum;
            for (int e = first; e < min(first + per, n); ++e) {
                const float x = value_of(sh.list[e]);
                const uint64_t w = w_of(x);
                if (before < need && before + w >= need) {
                    uint32_t ties = 1;
                    for (int o = e - 1; o >= 0 && value_of(sh.list[o]) == x; --o) ++ties;
                    sh.cut = Cut{x, ties, static_cast<uint32_t>(e + 1)};   // (and how many of the list are kept)
                    sh.all = before + w;
                }
                before += w;
            }
            __syncthreads();
            const Cut cut = sh.cut;
            const int kept = static_cast<int>(cut.ties), size = E * 32 * a.rows_warp;
            for (int e = threadIdx.x; e < kept; e += kSampleThreads)
                atomicAdd(reinterpret_cast<unsigned long long *>(segment) + static_cast<uint32_t>(sh.list[e]) / size,
                          static_cast<unsigned long long>(w_of(value_of(sh.list[e]))));
            __syncthreads();
            if (warp == 0 && kept > 0) {
                const uint64_t kept_all = sh.all;
                uint64_t rem = min(u < 1.f ? part_of(kept_all, u, false) : kept_all - 1, kept_all - 1);
                const bool light = rem == 0;     // (the first that is kept, however light: looked for below)
                int prefix = 0;
                const int seg = locate_of(segment, sh.ties[0], ctas * kSampleWarps, 0, 0, rem, prefix);
                // tokens at the cut before that segment
                prefix = 0;
                for (int e = kept - static_cast<int>(cut.first);; e += 32) {
                    const bool tie = e + lane < n && value_of(sh.list[min(e + lane, n - 1)]) == cut.v;
                    prefix += __popc(__ballot_sync(kAll, tie && static_cast<uint32_t>(sh.list[min(e + lane, n - 1)]) <
                                                                    static_cast<uint32_t>(seg * size)));
                    if (!__all_sync(kAll, tie)) break;
                }
                if (lane < ctas) {
                    const uint32_t to = mapa_shared(smem_u32(&sh.cut), lane);
                    st_cluster32(to, __float_as_uint(cut.v));            // (a Cut is 4-byte aligned)
                    st_cluster32(to + 4, cut.first);
                    st_cluster32(to + 8, light ? 2u : 1u);
                    st_cluster32(mapa_shared(smem_u32(&sh.seg), lane), seg);
                    st_cluster32(mapa_shared(smem_u32(&sh.tie_prefix), lane), prefix);
                    st_cluster64(mapa_shared(smem_u32(&sh.rem), lane), rem);
                    st_cluster64(mapa_shared(smem_u32(&sh.all), lane), kept_all);
                }
            } else if (warp == 0 && lane < ctas) {
                st_cluster32(mapa_shared(smem_u32(&sh.cut), lane) + 8, 0);
            }
        }
        __syncwarp();
        sync();
        const Cut cut = sh.cut;
        if (cut.ties == 0) return false;
        if (cut.ties == 2) {
            const Sums all_of = sums(cut.v);
            end_draw<T>(a, sh, handed(), cut.v, cut.first, all_of.above, all_of.ties, all_of.buf, u);
        } else {
            draw_segment(cut.v, cut.first, sh.all);
        }
        return true;
    }

    // ------------------------------------------------------------ a row
    // False: this CTA has nothing left to do for its row, and nobody looks at its
    // shared memory again.
    DG_DEVICE bool run()
    {
        t = a.temperature != nullptr ? __ldg(a.temperature + row) : 1.f;
        const int k = a.top_k != nullptr ? __ldg(a.top_k + row) : 0;
        const float p = a.top_p != nullptr ? __ldg(a.top_p + row) : 1.f;
        const float low = a.min_p != nullptr ? __ldg(a.min_p + row) : 0.f;
        const float u = __ldg(a.u + row);
        if (threadIdx.x == 0) sh.listed = sh.todo = 0;
        for (int k = threadIdx.x; k < kBins; k += kSampleThreads) sh.hist[0][k] = 0;
        __syncwarp();
        if (ctas > 1) cluster_arrive_all();                  // (the others' shared memory: only once they run)
        uint32_t hi = 0, lo = 0;
        typename Vec<T>::Most most = Vec<T>::none();
        int g = 0, left = rows_group();
        rows<8, E == 4>(0, a.rows_warp, [&](const uint4 &v, int r) {
            Vec<T>::most(most, v);
            if (--left > 0 && r + 1 < a.rows_warp) return;
            const float x = Vec<T>::value(most);
            group(g++) = Vec<T>::narrow(x);
            hi = max(hi, order_of(x));
            if (x > -INFINITY) lo = max(lo, ~order_of(x));
            most = Vec<T>::none();
            left = rows_group();
        });
        const int groups = g;
        for (; g < kGroups; ++g) group(g) = Vec<T>::narrow(-INFINITY);
        __syncwarp();
        if (ctas > 1) cluster_wait_all();
        const uint2 ends = largest(hi, lo);
        m = of_order(ends.x);

        const bool lead = rank == 0 && threadIdx.x == 0;
        if (m == -INFINITY) {                                // no token
            if (lead) {
                a.token[row] = -1;
                if (a.logprob != nullptr) a.logprob[row] = -INFINITY;
            }
            return true;
        }
        if (!(t > 0.f) || k == 1 || p <= 0.f) {              // the first of the largest
            uint32_t best = 0;
            constexpr int N = 4;
            picked<N>(pick([&](float x) -> bool { return x == m; }),
                      [&](const uint4 (&v)[N], const int (&w)[N], const int (&r)[N], const int (&l)[N]) {
#pragma unroll
                          for (int i = 0; i < N; ++i) {
                              float x[E];
                              Vec<T>::unpack(v[i], x);
#pragma unroll
                              for (int e = 0; e < E; ++e)
                                  if (x[e] == m) best = max(best, ~static_cast<uint32_t>(place(w[i], r[i], l[i], e)));
                          }
                      });
            __syncwarp();
            best = largest(best, 0).x;
            if (lead) {
                a.token[row] = static_cast<int>(~best) - skew;
                if (a.logprob != nullptr) a.logprob[row] = 0.f;
            }
            return true;
        }
        t = fminf(fmaxf(t, 7.8886091e-31f), 1.2676506e30f);  // 2^-100, 2^100
        ready();
        lay_table();
        const bool some = k > 0 && k < a.V, part = p < 1.f;
        if (!some && !part && !(low > 0.f)) {
            __syncthreads();
            const Sums s = sums_all();
            end_draw<T>(a, sh, handed(), -INFINITY, 0, s.above, s.ties, s.buf, u);
            return true;
        }
        float min_value = -INFINITY;
        if (low > 0.f && !flat) {
            if (threadIdx.x == 0)
                sh.min_value = fminf(m, __double2float_ru(static_cast<double>(m) +
                                                          static_cast<double>(t) * log(static_cast<double>(low))));
            __syncthreads();
            min_value = sh.min_value;
        }
        // few tokens: above the k-th largest of the groups' maxima, or above min-p's value
        const bool list_k = some && k <= kListMost;
        const bool list_min = !list_k && low > 0.f && !(part && some);
        if (!flat && (list_k || list_min)) {
            uint64_t all = 0;
            if (part && !some) all = sums_all().above;
            float scale = 0.f, limit = INFINITY, from = min_value;
            if (list_k) {
                // What a mask of finite values leaves aside: weights below e^-750.  It may
                // not widen the bins, nor count as groups that hold a token.
                const float masked = m - fmaxf(1000.f, 750.f * t);
                uint32_t lo = ends.y;
                if (of_order(~lo) < masked) {
                    lo = 0;
                    for (int g = 0; g < groups; ++g) {
                        const float x = Vec<T>::widen(group(g));
                        if (x >= masked && x > -INFINITY) lo = max(lo, ~order_of(x));
                    }
                    lo = largest(lo, 0).x;
                }
                from = masked;
                scale = static_cast<float>(kBins) / (m - of_order(~lo));
                uint32_t *hist = sh.hist[0];
                auto count = [&](float x) {
                    if (x >= masked && x > -INFINITY)
                        atomicAdd(hist + max(0, min(static_cast<int>((m - x) * scale), kBins - 1)), 1u);
                };
                auto found = [&]() -> Found { return find<false>(k, 0.f, [](int) -> float { return 0.f; }); };
                // (below half of the maxima there are many more tokens than maxima)
                Found f;
                f.total = 0;
                if (2 * k <= ctas * kSampleThreads * (a.rows_warp / rows_group())) {
#pragma unroll 1
                    for (int g = 0; g < groups; ++g) count(Vec<T>::widen(group(g)));
                    f = found();
                }
                if (f.total < 2u * static_cast<uint32_t>(k)) {
                    hist = clear();
                    each([&](float x, int, int) { count(x); });
                    f = found();
                }
                if (f.bin >= 0 && f.bin < kBins - 1) limit = static_cast<float>(f.bin + 1);
                else scale = 0.f;                            // (all of them)
            }
            auto wanted = [&](float x) -> bool {
                return x >= from && x > -INFINITY && !((m - x) * scale >= limit);
            };
            list_of(wanted);
            const int n = join_lists();
            if (n <= kList) {
                if (rank != 0) return false;
                end_listed<T>(a, sh, handed(), n, some ? k : 0, p, all, min_value, u);
                return true;
            }
        }
        __syncthreads();
        if (!flat && part && !some && !(low > 0.f)) {
            end_nucleus<T>(a, sh, handed(), p, u);
            return true;
        }
        end_counted<T>(a, sh, handed(), some ? k : 0, p, min_value, u);
        return true;
    }

    // The values that a token may have by their place in the order, which the lower bits of a
    // bf16 number's order do not change.
    static constexpr int kUnused = E == 8 ? 16 : 0;
    DG_DEVICE static uint32_t place_in_order(float v) { return order_of(v) >> kUnused; }
    DG_DEVICE static float value_in_order(uint32_t at)
    {
        return of_order(E == 8 ? at << 16 | (at >> 15 ? 0u : 0xFFFFu) : at);
    }
    // The least of them that is not below x.
    DG_DEVICE static float value_from(float x)
    {
        const uint32_t o = order_of(x);
        if (E == 4) return x;
        return of_order(o >> 31 ? (o + 0xFFFFu) & ~0xFFFFu : o | 0xFFFFu);
    }
    // The cuts by counting: top-k's, min-p's, top-p's; the highest is the one.
    DG_DEVICE void draw_counted(int k, float p, float min_value, float u)
    {
        const bool part = p < 1.f;
        Cut by_k{-INFINITY, 0, 0};
        if (flat) by_k = Cut{m, k > 0 ? static_cast<uint32_t>(k) : ~0u, 0};
        else if (k > 0) by_k = select<false>(k, 0.f, -INFINITY);
        const float least = value_from(fmaxf(by_k.v, min_value));
        float v = least;
        uint64_t whole = 0;                                  // what top-p is the part of
        if (part) {
            const Sums s = sums(by_k.v);
            whole = s.above;
            if (by_k.v > -INFINITY) whole += w_of(by_k.v) * min(by_k.first, s.ties);
            if (!flat)
                v = fmaxf(v, select<true>(0, p * (static_cast<float>(whole) * (1.f / 35184372088832.f) * exp2f(weight.shift())),
                                          by_k.v).v);
        }
        // Top-p's cut by exact sums, from v on.  By its place in the order it is one of lo .. hi,
        // which each sum narrows: by steps that grow (in fp32 rows, whose tokens are far apart
        // there, after a few neighbours), then by halves, 45 sums at most.
        uint32_t at = place_in_order(v), lo = place_in_order(least), hi = place_in_order(m);
        uint32_t step = E == 8 ? 1 : 1 << 12;
        Sums s = sums(v);
        int64_t kept;
        for (int moves = 0;; ++moves) {
            const uint64_t wv = v > -INFINITY ? w_of(v) : 0;
            kept = v == by_k.v ? min(by_k.first, s.ties) : s.ties;
            if (!part) break;
            const uint64_t need = part_of(whole, p, true);
            const bool up = s.above >= need;                 // reached before
            if (lo >= hi || (!up && (s.above + wv * kept >= need || !(v > least)))) {
                // the fewest at the cut that reach it
                const uint64_t short_of = need > s.above ? need - s.above : 0;
                int64_t n = 0;
                for (int64_t step = 1 << 20; step > 0; step >>= 1)
                    if (n + step <= kept && wv * (n + step) < short_of) n += step;
                kept = min(kept, n + 1);
                break;
            }
            if (up) lo = at + 1;
            else hi = at - 1;
            if (E == 4 && moves < kNeighbours) {
                uint32_t near = 0;
                each([&](float x, int, int) {
                    if (up ? x > v : x < v && x >= least) near = max(near, up ? ~order_of(x) : order_of(x));
                });
                near = largest(near, 0).x;
                at = (up ? ~near : near) >> kUnused;
            } else {
                const uint32_t half = hi > lo ? (hi - lo) / 2 : 0;
                at = up ? lo + min(half, step) : hi - min(half, step);
                step = min(step, 1u << 28) * 4;
            }
            at = min(max(at, lo), max(lo, hi));
            v = value_in_order(at);
            s = sums(v);
        }
        end_draw<T>(a, sh, handed(), v, kept, s.above, s.ties, s.buf, u);
    }
};

template <class T>
__device__ __forceinline__ void sample_body(const SampleArgs &a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    griddep_wait();
    griddep_launch_dependents();
    const bool stays = Sampler<T>(a, *reinterpret_cast<SampleShared *>(smem),
                                  Row{static_cast<int>(blockIdx.x) / a.ctas, 0.f, 1.f, 0}).run();
    if (a.ctas == 1) return;
    // nobody leaves while its shared memory may be read
    __syncwarp();
    cluster_arrive_all();
    if (stays) cluster_wait_all();
}

}  // namespace

int sample_smem_bytes() { return static_cast<int>(sizeof(SampleShared)); }

__global__ void __launch_bounds__(kSampleThreads, kSampleCtas) sample_bf16_kernel(const __grid_constant__ SampleArgs a)
{
    sample_body<uint16_t>(a);
}
__global__ void __launch_bounds__(kSampleThreads, kSampleCtas) sample_fp32_kernel(const __grid_constant__ SampleArgs a)
{
    sample_body<float>(a);
}

}  // namespace dg
