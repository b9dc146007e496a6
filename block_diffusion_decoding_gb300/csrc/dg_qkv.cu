// dg_qkv.cu -- the per-head RMS norm of queries and keys with the position
// rotation, into dense rows (dg_qk_norm_rope) or, with the values, into the
// pages of a paged KV cache (dg_paged_append).
//
// Both are one read and one write of every value, so what is left to decide
// is how few instructions a value costs.  A head of D values is held by a
// group of D / 8 lanes (rounded up to a power of two) as two runs of 4 values
// a lane, placed so that a rotated pair never leaves its lane:
//   pairs (m, m + rot / 2)   runs at 4 l and rot / 2 + 4 l for l < rot / 8,
//                            then the values that are not rotated, 8 a lane;
//   pairs (2m, 2m + 1)       runs at 8 l and 8 l + 4.
// So a lane needs 4 angles, computed once for all the heads it works on, and
// the only shuffles are the norm's sum.
//   norm      r = 1 / sqrt(mean x^2 + eps) by a shuffle tree of the group,
//             y = x r (offset + w);
//   rotation  the angle, position x frequency, is kept as a fraction of a
//             turn in 64-bit fixed point: the step of a frequency f is
//             2^64 f / 2 pi, so position x step wraps modulo one turn exactly
//             and the angle of position 262143 is as accurate as that of
//             position 1; its top 32 bits give an angle in [-pi, pi) for the
//             fast sine and cosine (absolute error about 2^-21, far below the
//             half step 2^-8 of the bf16 result).
// Everything is fp32 until the one rounding to bf16 at the store.
//
// Bound by HBM where there are many tokens: 32768 tokens' 16 + 8 heads of 256
// (0.8 GB read and written) take 127.8 us, 93% of a plain copy's rate; the append
// of thirteen prompts' keys and values, 42185 tokens of 8 heads of 128, 55.1 us
// (93%); of 16 blocks of 256 with their queries, 134 MB, 25.6 us.  Issue slots come
// second: with a value's pair in another lane, and sines by shuffles, the first of
// these took 265 us, and with a position, a row and angles for every four heads
// instead of eight 133 (the blocks 29.4).  Twelve heads a group, or four batches of
// four or two, were slower, as were blocks of 256 and 512 threads, and the loads
// behind the staging of q_start.  A few tokens are bound by the launch: 1.9 us on the
// GPU, 7.0-7.6 for the call through the Python binding.
#include "dg_paged_kernels.h"

namespace dg {

namespace {

// 4 bf16 values.  Not the read-only path: q_out may be q itself.
DG_DEVICE uint2 ld_stream(const uint16_t *p)
{
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "l"(p)
                 : "memory");
    return v;
}

DG_DEVICE float2 unpack2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

DG_DEVICE uint32_t pack2(float2 v)
{
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&h2);
}

// cos and sin of position x step (turns in 64-bit fixed point).
DG_DEVICE void turn(int pos, uint64_t step, float &c, float &s)
{
    const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
    const float ang = static_cast<float>(static_cast<int32_t>(ph >> 32)) *
                      1.4629180792671596e-9f;   // 2 pi / 2^32
    __sincosf(ang, &s, &c);
}

// The last b with start[b] <= t (-1: none), start non-decreasing, [n].
DG_DEVICE int last_not_above(const int32_t *start, int n, int t)
{
    int lo = 0, hi = n;   // answer + 1 in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

}  // namespace

// A group takes up to HPG x BATCH consecutive heads of one kind (q, k or v):
// they share the lane's addresses, weights, sines and cosines, and the loads of
// HPG of them are in flight together; without pages, those of the next HPG
// behind them (into pages that took 15% longer where nothing is normed).
template <bool PAGED, int HPG, int BATCH>
__device__ __forceinline__ void qkv_body(const QkvArgs &a)
{
    __shared__ int32_t s_start[PAGED ? kQkvSeqSmem : 1];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int lg = a.lanes;                       // lanes of a group, a power of two
    const int sub = tid & (lg - 1);

    if (PAGED) {
        if (a.B < kQkvSeqSmem) {
            for (int b = tid; b <= a.B; b += kQkvThreads) s_start[b] = a.q_start[b];
            __syncthreads();
        }
        // the batch's new lengths, and a look at the given ones
        for (int64_t b = static_cast<int64_t>(blockIdx.x) * kQkvThreads + tid; b < a.B;
             b += static_cast<int64_t>(gridDim.x) * kQkvThreads) {
            const int r0 = a.q_start[b], r1 = a.q_start[b + 1], kv = a.kv_len[b];
            // its rows as the attention counts them: those that the batch has
            const int first = min(max(r0, 0), a.T), n = max(min(r1, a.T) - first, 0);
            if (a.kv_len_out != nullptr) a.kv_len_out[b] = kv < 0 ? kv : kv + min(n, 0x7FFFFFFF - kv);
            if (r0 < 0 || r1 < r0 || r1 > a.T || kv < 0) report_error(a.ws, DG_ERR_DEVICE, 902);
        }
    }

    // the groups of a warp have the same heads of neighbouring tokens, so that
    // all of it norms and rotates, or none
    const uint32_t warp = (blockIdx.x * static_cast<uint32_t>(kQkvThreads) + tid) >> 5;
    const uint32_t tw = warp / static_cast<uint32_t>(a.chunks);
    const uint32_t tu = (tw << (5 - a.lanes_log2)) + ((tid & 31u) >> a.lanes_log2);
    const bool live = tu < static_cast<uint32_t>(a.T);
    const int t = live ? static_cast<int>(tu) : 0;
    int c = static_cast<int>(warp - tw * a.chunks);
    const bool is_q = c < a.q_chunks, is_v = c >= a.q_chunks + a.k_chunks;
    c -= is_q ? 0 : is_v ? a.q_chunks + a.k_chunks : a.q_chunks;
    const int h0 = c * (HPG * BATCH);
    const int count = live ? min(HPG * BATCH, (is_q ? a.nq : a.nk) - h0) : 0;   // heads of this group

    // ---- the two runs of this lane: value offsets, angles of its pairs
    const int rl = a.interleaved ? 0 : a.rot >> 3;    // lanes with split runs
    const bool split = sub < rl;
    const int e0 = split ? 4 * sub : a.interleaved ? 8 * sub : a.rot + 8 * (sub - rl);
    const int gap = split ? (a.rot >> 1) : 4;         // from the first run to the second
    const bool in_head = sub * 8 < a.D;
    const bool turns = !is_v && (a.interleaved ? e0 < a.rot : split);

    uint2 lo[HPG], hi[HPG];
    const uint16_t *src = (is_q ? a.q + t * a.q_stride : is_v ? a.v + t * a.v_stride
                                                              : a.k + t * a.k_stride) +
                          (h0 * a.D + e0);
    auto load = [&](int first, uint2 (&l)[HPG], uint2 (&h)[HPG]) {
#pragma unroll
        for (int j = 0; j < HPG; ++j, src += a.D) {
            l[j] = h[j] = make_uint2(0, 0);
            if (in_head && first + j < count) {
                l[j] = ld_stream(src);
                h[j] = ld_stream(src + gap);
            }
        }
    };
    load(0, lo, hi);

    // ---- position, and the row of the cache that takes the token
    int pos = 0;
    int64_t row = -1;             // row of the cache's pages (k and v), -1: none
    bool token = live;            // the token belongs to a sequence
    if (PAGED) {
        if (live) {
            const int32_t *start = a.B < kQkvSeqSmem ? s_start : a.q_start;
            const int b = last_not_above(start, a.B + 1, t);
            token = b >= 0 && b < a.B && t >= start[b] && t < start[b + 1];
            if (token) {
                const int kv = a.kv_len[b];
                const int64_t at = static_cast<int64_t>(kv) + (t - max(start[b], 0));
                pos = a.positions != nullptr ? a.positions[t] : static_cast<int>(at);
                if (kv >= 0 && at < static_cast<int64_t>(a.max_pages) * a.page_size) {
                    const uint32_t pg = static_cast<uint32_t>(at) / static_cast<uint32_t>(a.page_size);
                    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pg];
                    if (page >= 0 && page < a.n_pages)
                        row = page * a.page_stride +
                              (at - static_cast<int64_t>(pg) * a.page_size) * a.nk * a.D;
                }
                if (row < 0) report_error(a.ws, DG_ERR_DEVICE, 901);
            }
        }
    } else if (live && a.rot > 0) {
        pos = a.positions[t];
    }
    float2 cs[2], sn[2], ns[2];   // of the lane's four pairs; ns = -sn
#pragma unroll
    for (int e = 0; e < 2; ++e) cs[e] = make_float2(1.f, 1.f), sn[e] = make_float2(0.f, 0.f);
    if (turns) {
        // pairs m .. m + 3 either way
        const ulonglong2 *steps = reinterpret_cast<const ulonglong2 *>(a.steps + 4 * sub);
        const ulonglong2 s0 = __ldg(steps), s1 = __ldg(steps + 1);
        turn(pos, s0.x, cs[0].x, sn[0].x);
        turn(pos, s0.y, cs[0].y, sn[0].y);
        turn(pos, s1.x, cs[1].x, sn[1].x);
        turn(pos, s1.y, cs[1].y, sn[1].y);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) ns[e] = make_float2(-sn[e].x, -sn[e].y);

    const uint16_t *wp = is_v ? nullptr : is_q ? a.q_weight : a.k_weight;
    float2 w[4];                  // offset + weight of the lane's values
    if (wp != nullptr && in_head) {
        const uint2 wa = __ldg(reinterpret_cast<const uint2 *>(wp + e0));
        const uint2 wb = __ldg(reinterpret_cast<const uint2 *>(wp + e0 + gap));
        const float2 off = make_float2(a.weight_offset, a.weight_offset);
        w[0] = add2(unpack2(wa.x), off);
        w[1] = add2(unpack2(wa.y), off);
        w[2] = add2(unpack2(wb.x), off);
        w[3] = add2(unpack2(wb.y), off);
    }

    uint16_t *dst;
    if (is_q)
        dst = a.q_out + t * a.qo_stride;
    else if (!PAGED)
        dst = a.k_out + t * a.ko_stride;
    else
        dst = (is_v ? a.v_cache : a.k_cache) + row;
    dst += h0 * a.D + e0;
    const int stores = token && in_head && (is_q || !PAGED || row >= 0) ? count : 0;
    const bool normed = wp != nullptr;
#pragma unroll
    for (int b = 0; b < BATCH; ++b) {
        uint2 next_lo[HPG], next_hi[HPG];
        if (!PAGED && b + 1 < BATCH) load((b + 1) * HPG, next_lo, next_hi);
        // ---- norms of all the group's heads together, so that their shuffles
        // overlap; every lane of the warp takes part in them
        float rn[HPG];
        if (__any_sync(0xFFFFFFFFu, normed)) {
#pragma unroll
            for (int j = 0; j < HPG; ++j) {
                float2 x = unpack2(lo[j].x);
                float2 s2 = mul2(x, x);
                x = unpack2(lo[j].y);
                s2 = fma2(x, x, s2);
                x = unpack2(hi[j].x);
                s2 = fma2(x, x, s2);
                x = unpack2(hi[j].y);
                s2 = fma2(x, x, s2);
                rn[j] = s2.x + s2.y;
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                if (o < lg) {
#pragma unroll
                    for (int j = 0; j < HPG; ++j) rn[j] += __shfl_xor_sync(0xFFFFFFFFu, rn[j], o);
                }
            }
#pragma unroll
            for (int j = 0; j < HPG; ++j) rn[j] = rsqrtf(rn[j] * a.inv_d + a.eps);
        }
        if (normed || turns) {        // else the bits go as they are
#pragma unroll
            for (int j = 0; j < HPG; ++j) {
                // x[0], x[1]: the first run, x[2], x[3]: the second
                float2 x[4] = {unpack2(lo[j].x), unpack2(lo[j].y), unpack2(hi[j].x), unpack2(hi[j].y)};
                if (normed) {
                    const float2 r2 = make_float2(rn[j], rn[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = mul2(mul2(x[e], r2), w[e]);
                }
                if (!turns) {
                    // (also where a value is infinite: no product with a zero sine)
                } else if (a.interleaved) {
                    // (x.x, x.y) is a pair
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float co = (e & 1) ? cs[e >> 1].y : cs[e >> 1].x;
                        const float si = (e & 1) ? sn[e >> 1].y : sn[e >> 1].x;
                        const float2 p = x[e];
                        x[e] = make_float2(p.x * co - p.y * si, p.y * co + p.x * si);
                    }
                } else {
                    // x[e] pairs with x[e + 2], component by component
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 p = x[e], q = x[e + 2];
                        x[e] = fma2(q, ns[e], mul2(p, cs[e]));
                        x[e + 2] = fma2(p, sn[e], mul2(q, cs[e]));
                    }
                }
                lo[j] = make_uint2(pack2(x[0]), pack2(x[1]));
                hi[j] = make_uint2(pack2(x[2]), pack2(x[3]));
            }
        }
#pragma unroll
        for (int j = 0; j < HPG; ++j, dst += a.D) {
            if (b * HPG + j < stores) {
                *reinterpret_cast<uint2 *>(dst) = lo[j];
                *reinterpret_cast<uint2 *>(dst + gap) = hi[j];
            }
        }
        if (PAGED && b + 1 < BATCH) load((b + 1) * HPG, lo, hi);
#pragma unroll
        for (int j = 0; j < HPG; ++j) {
            if (!PAGED && b + 1 < BATCH) {
                lo[j] = next_lo[j];
                hi[j] = next_hi[j];
            }
        }
    }
}

__global__ void __launch_bounds__(kQkvThreads) qk_norm_rope_kernel_1(QkvArgs a)
{
    qkv_body<false, 1, 1>(a);
}
__global__ void __launch_bounds__(kQkvThreads) qk_norm_rope_kernel_4(QkvArgs a)
{
    qkv_body<false, 4, 1>(a);
}
__global__ void __launch_bounds__(kQkvThreads) qk_norm_rope_kernel_8(QkvArgs a)
{
    qkv_body<false, 4, 2>(a);
}
__global__ void __launch_bounds__(kQkvThreads) paged_append_kernel_1(QkvArgs a)
{
    qkv_body<true, 1, 1>(a);
}
__global__ void __launch_bounds__(kQkvThreads) paged_append_kernel_4(QkvArgs a)
{
    qkv_body<true, 4, 1>(a);
}
__global__ void __launch_bounds__(kQkvThreads, 8) paged_append_kernel_8(QkvArgs a)
{
    qkv_body<true, 4, 2>(a);
}

}  // namespace dg
