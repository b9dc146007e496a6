// dg_qkv.cu -- the per-head RMS norm of queries and keys with the position
// rotation, into dense rows (dg_qk_norm_rope) or, with the values, into the
// pages of a paged KV cache (dg_paged_append).
//
// Both are one read and one write of every value.  A head of D values is
// held by a group of D / 8 lanes (rounded up to a power of two), 8 values
// (one 16-byte load) per lane:
//   norm      r = 1 / sqrt(mean x^2 + eps) by a shuffle tree of the group,
//             y = x r (offset + w);
//   rotation  of the first `rot` values by position x frequency.  The angle
//             is kept as a fraction of a turn in 64-bit fixed point: the
//             frequency step is round(2^64 f / 2 pi), so position x step
//             wraps modulo one turn exactly, and the angle of position
//             262143 is as accurate as that of position 1; its top 32 bits
//             give an angle in [-pi, pi) for the fast sine and cosine
//             (absolute error about 2^-21, far below the half step 2^-9 of
//             the bf16 result).  Pairs (m, m + rot / 2) exchange values by a
//             shuffle, pairs (2m, 2m + 1) sit in one lane.
// Everything is fp32 until the one rounding to bf16 at the store.
#include "dg_kernels.h"

namespace dg {

namespace {

// Not the read-only path: q_out may be q itself.
DG_DEVICE uint4 ld_stream(const uint16_t *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

DG_DEVICE void unpack8(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}

DG_DEVICE uint4 pack8(const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t *>(&h2);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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

// HPG heads per group: their loads are in flight together and share one set
// of sines and cosines.
template <bool PAGED, int HPG>
__device__ __forceinline__ void qkv_body(const QkvArgs &a)
{
    __shared__ int32_t s_start[kQkvSeqSmem];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x;
    const int lg = a.lanes;                       // lanes of a group, a power of two
    const int sub = tid & (lg - 1);
    const int e0 = sub * 8;                       // first value this lane holds
    const bool in_head = e0 < a.D;

    if (PAGED) {
        const bool staged = a.B < kQkvSeqSmem;
        if (staged) {
            for (int b = tid; b <= a.B; b += kQkvThreads) s_start[b] = a.q_start[b];
            __syncthreads();
        }
        // the batch's new lengths, and a look at the given ones
        for (int64_t b = static_cast<int64_t>(blockIdx.x) * kQkvThreads + tid; b < a.B;
             b += static_cast<int64_t>(gridDim.x) * kQkvThreads) {
            const int r0 = a.q_start[b], r1 = a.q_start[b + 1], kv = a.kv_len[b];
            if (a.kv_len_out != nullptr) a.kv_len_out[b] = kv + r1 - r0;
            if (r0 < 0 || r1 < r0 || r1 > a.T || kv < 0) report_error(a.ws, DG_ERR_DEVICE, 902);
        }
    }

    const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kQkvThreads + tid) / lg;
    const int64_t t64 = unit / a.chunks;
    const int chunk = static_cast<int>(unit - t64 * a.chunks);
    const bool live = t64 < a.T;
    const int t = live ? static_cast<int>(t64) : 0;

    // ---- this group's heads: chunk, chunk + chunks, ...; q, then k, then v
    uint4 raw[HPG];
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = chunk + j * a.chunks;
        raw[j] = make_uint4(0, 0, 0, 0);
        if (live && in_head && h < a.heads) {
            const uint16_t *src =
                h < a.nq            ? a.q + static_cast<int64_t>(t) * a.q_stride + h * a.D
                : h < a.nq + a.nk   ? a.k + static_cast<int64_t>(t) * a.k_stride + (h - a.nq) * a.D
                                    : a.v + static_cast<int64_t>(t) * a.v_stride +
                                          (h - a.nq - a.nk) * a.D;
            raw[j] = ld_stream(src + e0);
        }
    }

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
                const int64_t at = static_cast<int64_t>(a.kv_len[b]) + (t - start[b]);
                pos = a.positions != nullptr ? a.positions[t] : static_cast<int>(at);
                const int64_t pg = at / a.page_size;
                if (at >= 0 && pg < a.max_pages) {
                    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pg];
                    if (page >= 0 && page < a.n_pages)
                        row = static_cast<int64_t>(page) * a.page_stride +
                              (at - pg * a.page_size) * a.nk * a.D;
                }
                if (row < 0) report_error(a.ws, DG_ERR_DEVICE, 901);
            }
        }
    } else if (live && a.rot > 0) {
        pos = a.positions[t];
    }

    // ---- sines and cosines of this lane's values
    float cs[8], sn[8];
    const int half = a.rot >> 1;
    const bool turns = e0 < a.rot;
    if (a.rot > 0) {
        const int m0 = a.interleaved ? e0 >> 1 : (e0 < half ? e0 : e0 - half);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cs[e] = 1.f;
            sn[e] = 0.f;
            if (turns) {
                const int m = a.interleaved ? m0 + (e >> 1) : m0 + e;
                if (!a.interleaved || (e & 1) == 0) {
                    const uint64_t ph =
                        static_cast<uint64_t>(static_cast<int64_t>(pos)) * __ldg(a.steps + m);
                    const float ang = static_cast<float>(static_cast<int32_t>(ph >> 32)) *
                                      1.4629180792671596e-9f;   // 2 pi / 2^32
                    __sincosf(ang, &sn[e], &cs[e]);
                } else {
                    sn[e] = sn[e - 1];
                    cs[e] = cs[e - 1];
                }
            }
        }
    }

#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = chunk + j * a.chunks;
        const bool have = h < a.heads;
        const bool is_q = h < a.nq, is_v = h >= a.nq + a.nk;
        uint4 res = raw[j];
        float x[8];
        unpack8(raw[j], x);
        const uint16_t *w = is_q ? a.q_weight : a.k_weight;
        // every lane of the warp takes part in the shuffles
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
        for (int o = lg >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
        if (w != nullptr && !is_v) {
            const float r = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
            float wv[8];
            unpack8(in_head ? __ldg(reinterpret_cast<const uint4 *>(w + e0)) : make_uint4(0, 0, 0, 0),
                    wv);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (a.weight_offset + wv[e]);
        }
        if (a.rot > 0) {
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float p = x[e], q = x[e + 1];
                    x[e] = p * cs[e] - q * sn[e];
                    x[e + 1] = q * cs[e] + p * sn[e];
                }
            } else {
                // the pair's other value sits rot / 16 lanes away
                const int hop = a.rot >> 4;
                const int other = !turns ? sub : e0 < half ? sub + hop : sub - hop;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = __shfl_sync(0xFFFFFFFFu, x[e], other, lg);
                    x[e] = e0 < half ? x[e] * cs[e] - p * sn[e] : x[e] * cs[e] + p * sn[e];
                }
            }
        }
        if (!is_v && (w != nullptr || turns)) res = pack8(x);   // else the bits as they are
        if (have && in_head && token) {
            if (is_q) {
                *reinterpret_cast<uint4 *>(a.q_out + static_cast<int64_t>(t) * a.qo_stride +
                                           h * a.D + e0) = res;
            } else if (PAGED) {
                if (row >= 0) {
                    uint16_t *base = is_v ? a.v_cache : a.k_cache;
                    const int hk = h - a.nq - (is_v ? a.nk : 0);
                    *reinterpret_cast<uint4 *>(base + row + hk * a.D + e0) = res;
                }
            } else {
                *reinterpret_cast<uint4 *>(a.k_out + static_cast<int64_t>(t) * a.ko_stride +
                                           (h - a.nq) * a.D + e0) = res;
            }
        }
    }
}

__global__ void __launch_bounds__(kQkvThreads) qk_norm_rope_kernel_1(QkvArgs a)
{
    qkv_body<false, 1>(a);
}
__global__ void __launch_bounds__(kQkvThreads) qk_norm_rope_kernel_4(QkvArgs a)
{
    qkv_body<false, 4>(a);
}
__global__ void __launch_bounds__(kQkvThreads) paged_append_kernel_1(QkvArgs a)
{
    qkv_body<true, 1>(a);
}
__global__ void __launch_bounds__(kQkvThreads) paged_append_kernel_4(QkvArgs a)
{
    qkv_body<true, 4>(a);
}

}  // namespace dg
