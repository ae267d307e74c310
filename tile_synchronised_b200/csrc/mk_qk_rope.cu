// mk_qk_rope.cu -- the pass between the QKV projection and the attention of
// new tokens: per-head RMSNorm of q and k, rotation by each token's position,
// q out in the cache's type, K and V into the pages.
//
//   x' = x * rsqrt(mean(x^2) + eps) * gain          (q and k heads, with gains)
//   (a, b) = (x'_i, x'_{i + d/2}) -> (a cos - b sin, b cos + a sin),
//   angle = (length + depth) * theta^(-2i/d)
//
// The angle is kept in turns in 64 bits (position * theta^(-2i/d) / 2 pi,
// reduced by its nearest integer), so that far positions lose nothing; sine
// and cosine then are of a number within half a turn, in 32 bits.  One CTA
// per token: its d/2 sines and cosines are computed once for all heads.
// A warp takes a head at a time, each lane the same d/64 values of both
// halves, so a rotation needs no exchange and the norm one warp sum.
// Bound by HBM: each input value is read once (4 or 2 bytes), each output
// written once (2 bytes).
#include <atomic>
#include <cmath>

#include "mk_kernel.h"
#include "mk_pages.h"

namespace mk {

constexpr int kRopeThreads = 256;

struct RopeArgs {
    mk_pages p;
    const void *qkv;
    const int *seqs, *n_new, *depth;
    const uint16_t *q_gain, *k_gain;
    uint16_t *q;
    long long qkv_stride, q_stride;
    size_t k_off, v_off;  // of this layer's pages
    int n, T, nq;
    float eps;
    double log2_theta;
};

// E consecutive values of 32 or 16 bits, widened.
template <int E, bool F32, bool BF16>
__device__ __forceinline__ void load_values(const void *base, size_t at, float *v) {
    if constexpr (F32) {
        const float *s = static_cast<const float *>(base) + at;
        if constexpr (E == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(s);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        } else if constexpr (E == 2) {
            const float2 x = *reinterpret_cast<const float2 *>(s);
            v[0] = x.x, v[1] = x.y;
        } else {
            v[0] = s[0];
        }
    } else {
        const uint16_t *s = static_cast<const uint16_t *>(base) + at;
        if constexpr (E == 4) {
            const uint2 x = *reinterpret_cast<const uint2 *>(s);
            v[0] = from16<BF16>(x.x & 0xFFFF), v[1] = from16<BF16>(x.x >> 16);
            v[2] = from16<BF16>(x.y & 0xFFFF), v[3] = from16<BF16>(x.y >> 16);
        } else if constexpr (E == 2) {
            const uint32_t x = *reinterpret_cast<const uint32_t *>(s);
            v[0] = from16<BF16>(x & 0xFFFF), v[1] = from16<BF16>(x >> 16);
        } else {
            v[0] = from16<BF16>(s[0]);
        }
    }
}

template <int E, bool BF16>
__device__ __forceinline__ void store_values(uint16_t *to, const float *v) {
    if constexpr (E == 4)
        *reinterpret_cast<uint2 *>(to) = make_uint2(pack16<BF16>(v[0], v[1]), pack16<BF16>(v[2], v[3]));
    else if constexpr (E == 2)
        *reinterpret_cast<uint32_t *>(to) = pack16<BF16>(v[0], v[1]);
    else
        to[0] = to16<BF16>(v[0]);
}

template <int D, bool F32, bool BF16>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const RopeArgs a) {
    constexpr int E = D / 64;  // values of each half per lane
    __shared__ float s_cos[D / 2], s_sin[D / 2];
    const int tok = blockIdx.x, i = tok / a.T, t = tok - i * a.T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, i, a.T);
    int twice = 0;
    for (int k = threadIdx.x; k < a.n; k += kRopeThreads) twice |= k != i && a.seqs[k] == e.seq;
    if (t >= e.fresh) {  // padding, or an entry that is out of range
        if (e.err && t == 0 && threadIdx.x == 0) pages_fail(a.p.state, e.err, i, e.seq);
        return;
    }
    const long long pos = (long long)e.len + (a.depth ? a.depth[tok] : t);
    if (threadIdx.x < D / 2) {
        const double turns = (double)pos * exp2(a.log2_theta * (-2.0 * threadIdx.x / D) - 2.6514961294723188);
        sincospif((float)(2.0 * (turns - rint(turns))), &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
    }
    twice = __syncthreads_or(twice);
    // the slot of the new token, and whether it may be written
    const int slot = e.len + t;
    const int page = a.p.table[(size_t)e.seq * a.p.max_pages + slot / a.p.page_size];
    int err = 0;
    if (twice)
        err = kPgSeq;
    else if (page < 0 || page >= a.p.n_pages)
        err = kPgPosition;
    else if (a.p.refs[page] != 1)
        err = kPgShared;
    if (err && threadIdx.x == 0) pages_fail(a.p.state, err, i, err == kPgSeq ? e.seq : page);
    const int nkv = a.p.n_kv_heads;
    const size_t row = ((size_t)(err ? 0 : page) * nkv * a.p.page_size + slot % a.p.page_size) * D;
    float c[E], s[E], gq[2][E], gk[2][E];
#pragma unroll
    for (int x = 0; x < E; ++x) {
        c[x] = s_cos[lane * E + x];
        s[x] = s_sin[lane * E + x];
    }
    if (a.q_gain) {
        load_values<E, false, true>(a.q_gain, lane * E, gq[0]);
        load_values<E, false, true>(a.q_gain, D / 2 + lane * E, gq[1]);
    }
    if (a.k_gain) {
        load_values<E, false, true>(a.k_gain, lane * E, gk[0]);
        load_values<E, false, true>(a.k_gain, D / 2 + lane * E, gk[1]);
    }
    const int heads = err ? a.nq : a.nq + 2 * nkv;
    for (int h = warp; h < heads; h += kRopeThreads / 32) {
        const size_t at = (size_t)tok * a.qkv_stride + (size_t)h * D + lane * E;
        float lo[E], hi[E];
        load_values<E, F32, BF16>(a.qkv, at, lo);
        load_values<E, F32, BF16>(a.qkv, at + D / 2, hi);
        uint16_t *to;
        if (h < a.nq + nkv) {
            const bool is_q = h < a.nq;
            if (is_q ? a.q_gain != nullptr : a.k_gain != nullptr) {
                float ss = 0.f;
#pragma unroll
                for (int x = 0; x < E; ++x) ss = fmaf(lo[x], lo[x], fmaf(hi[x], hi[x], ss));
                const float r = rsqrtf(warp_sum(ss) * (1.f / D) + a.eps);
#pragma unroll
                for (int x = 0; x < E; ++x) {
                    lo[x] *= r * (is_q ? gq[0][x] : gk[0][x]);
                    hi[x] *= r * (is_q ? gq[1][x] : gk[1][x]);
                }
            }
#pragma unroll
            for (int x = 0; x < E; ++x) {
                const float u = lo[x], w = hi[x];
                lo[x] = u * c[x] - w * s[x];
                hi[x] = w * c[x] + u * s[x];
            }
            to = is_q ? a.q + (size_t)tok * a.q_stride + (size_t)h * D
                      : static_cast<uint16_t *>(a.p.kv) + a.k_off + row + (size_t)(h - a.nq) * a.p.page_size * D;
        } else {
            to = static_cast<uint16_t *>(a.p.kv) + a.v_off + row + (size_t)(h - a.nq - nkv) * a.p.page_size * D;
        }
        store_values<E, BF16>(to + lane * E, lo);
        store_values<E, BF16>(to + D / 2 + lane * E, hi);
    }
}

template <int D>
static cudaError_t launch_rope(const RopeArgs &a, bool f32, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.n * a.T);
    const bool bf16 = a.p.dtype == MK_BF16;
    if (f32 && bf16) qk_rope_kernel<D, true, true><<<grid, kRopeThreads, 0, s>>>(a);
    if (f32 && !bf16) qk_rope_kernel<D, true, false><<<grid, kRopeThreads, 0, s>>>(a);
    if (!f32 && bf16) qk_rope_kernel<D, false, true><<<grid, kRopeThreads, 0, s>>>(a);
    if (!f32 && !bf16) qk_rope_kernel<D, false, false><<<grid, kRopeThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mk

using namespace mk;

extern "C" mk_status mk_qk_norm_rope(const mk_pages *p, int layer, const void *qkv, int qkv_dtype,
                                     long long qkv_stride, int n, int T, int n_heads, const int32_t *seqs,
                                     const int32_t *n_new, const int32_t *depth, const void *q_gain,
                                     const void *k_gain, float eps, double theta, void *q, long long q_stride,
                                     void *stream) {
    const char *who = "qk_norm_rope";
    const mk_status st = pages_check(p, layer < 0 ? 1 << 30 : layer, who);
    if (st != MK_OK) return st;
    if (n < 0 || n > p->max_seqs || T < 1 || (long long)n * T > (1 << 30) || n_heads < 1 || n_heads > 65535)
        return pages_refuse(who, "bad sizes: 0 <= n <= max_seqs, T >= 1, n_heads >= 1");
    if (n == 0) return MK_OK;
    if (!qkv || !q || !seqs) return pages_refuse(who, "null pointer");
    if (qkv_dtype != MK_FP32 && qkv_dtype != p->dtype)
        return pages_refuse(who, "qkv must be fp32 or of the cache's type", MK_ERR_UNSUPPORTED);
    if (((uintptr_t)qkv | (uintptr_t)q | (uintptr_t)q_gain | (uintptr_t)k_gain) & 15)
        return pages_refuse(who, "qkv, q and the gains must be 16-byte aligned");
    const int d = p->head_dim;
    if (qkv_stride < (long long)(n_heads + 2 * p->n_kv_heads) * d || qkv_stride % 8 ||
        q_stride < (long long)n_heads * d || q_stride % 8)
        return pages_refuse(who, "a stride is shorter than a row or not a multiple of 8");
    if (!(theta > 0.0) || !(eps >= 0.f)) return pages_refuse(who, "theta must be positive and eps not negative");
    RopeArgs a{*p, qkv, seqs, n_new, depth, static_cast<const uint16_t *>(q_gain),
               static_cast<const uint16_t *>(k_gain), static_cast<uint16_t *>(q), qkv_stride, q_stride,
               pages_offset(*p, 0, layer, 0), pages_offset(*p, 1, layer, 0), n, T, n_heads, eps, std::log2(theta)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool f32 = qkv_dtype == MK_FP32;
    return pages_launched(d == 64 ? launch_rope<64>(a, f32, s)
                                  : d == 128 ? launch_rope<128>(a, f32, s) : launch_rope<256>(a, f32, s),
                          who);
}
