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
// and cosine then are of a number within half a turn, in 32 bits.  A CTA takes
// kRopeTokens tokens of a sequence (one where there are too few to fill the
// SMs): their sines and cosines are computed once for all heads.  D / 8 lanes
// take a head, 4 values of both halves each, so that a rotation needs no
// exchange, the norm one sum over those lanes, and loads are of 16 bytes; they
// go through the heads kRopeRows at a time.  The first loads go out before the
// chain sequence -> length -> page -> holders is followed.
// Bound by HBM: each input value is read once (4 or 2 bytes), each output
// written once (2 bytes).  8 x 1024 prompt tokens of 32 + 2 x 8 heads of 128 from
// fp32 (768 live on average): 44 us, 5.2 TB/s, 0.80 of the measured copy; a step
// of 16 tokens: 4.2 us, the latency of its chain of loads.
#include <atomic>
#include <cmath>

#include "mk_kernel.h"
#include "mk_pages.h"

namespace mk {

constexpr int kRopeThreads = 256, kRopeTokens = 4, kRopeRows = 3;

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

// 4 consecutive values of 32 or 16 bits, widened.
template <bool F32, bool BF16>
__device__ __forceinline__ float4 load4(const void *base, size_t at) {
    if constexpr (F32) {
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
        return make_float4(from16<BF16>(x.x & 0xFFFF), from16<BF16>(x.x >> 16), from16<BF16>(x.y & 0xFFFF),
                           from16<BF16>(x.y >> 16));
    }
}
template <bool BF16>
__device__ __forceinline__ void store4(uint16_t *to, const float4 &v) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(pack16<BF16>(v.x, v.y), pack16<BF16>(v.z, v.w));
}
__device__ __forceinline__ float dot4(const float4 &x, const float4 &y) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
}
__device__ __forceinline__ float4 mul4(const float4 &x, const float4 &y) {
    return make_float4(x.x * y.x, x.y * y.y, x.z * y.z, x.w * y.w);
}
__device__ __forceinline__ float4 scale4(const float4 &x, float s) {
    return make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
}

template <int D, bool F32, bool BF16, int TOK>
__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int LR = D / 8, kSubs = kRopeThreads / LR;  // lanes of a head, heads at a time
    __shared__ __align__(16) float s_cos[TOK][D / 2], s_sin[TOK][D / 2];  // read 4 at a time
    __shared__ size_t s_row[TOK];  // offset of the token's slot in its layer's K or V
    __shared__ int s_write[TOK];
    const int chunks = (a.T + TOK - 1) / TOK, i = blockIdx.x / chunks, t0 = (blockIdx.x - i * chunks) * TOK;
    const int sub = threadIdx.x / LR, at = threadIdx.x % LR * 4;  // first head, values at, at + D / 2 of each
    const int nkv = a.p.n_kv_heads, heads = a.nq + 2 * nkv;
    float4 lo[kRopeRows], hi[kRopeRows];
    auto load = [&](int t, int h0) {  // heads h0 + sub, ... of token t
        const size_t row = (size_t)(i * a.T + t0 + t) * a.qkv_stride + at;
#pragma unroll
        for (int x = 0; x < kRopeRows; ++x) {
            const int h = h0 + sub + x * kSubs;
            if (h < heads) {
                lo[x] = load4<F32, BF16>(a.qkv, row + (size_t)h * D);
                hi[x] = load4<F32, BF16>(a.qkv, row + (size_t)h * D + D / 2);
            }
        }
    };
    load(0, 0);

    const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, i, a.T);
    const int tokens = min(TOK, e.fresh - t0);  // the others are padding, or the entry is out of range
    if (tokens <= 0) {
        if (e.err && t0 == 0 && threadIdx.x == 0) pages_fail(a.p.state, e.err, i, e.seq);
        return;
    }
    int twice = 0;
    for (int k = threadIdx.x; k < a.n; k += kRopeThreads) twice |= k != i && a.seqs[k] == e.seq;
    twice = __syncthreads_or(twice);
    if (threadIdx.x < tokens) {  // the slot of the new token, and whether it may be written
        const int slot = e.len + t0 + threadIdx.x;
        const int page = a.p.table[(size_t)e.seq * a.p.max_pages + slot / a.p.page_size];
        int err = 0;
        if (twice)
            err = kPgSeq;
        else if (page < 0 || page >= a.p.n_pages)
            err = kPgPosition;
        else if (a.p.refs[page] != 1)
            err = kPgShared;
        if (err) pages_fail(a.p.state, err, i, err == kPgSeq ? e.seq : page);
        s_write[threadIdx.x] = !err;
        s_row[threadIdx.x] = ((size_t)(err ? 0 : page) * nkv * a.p.page_size + slot % a.p.page_size) * D;
    }
    for (int x = threadIdx.x; x < tokens * (D / 2); x += kRopeThreads) {
        const int t = x / (D / 2), j = x - t * (D / 2);
        const long long pos = (long long)e.len + (a.depth ? a.depth[i * a.T + t0 + t] : t0 + t);
        // theta^(-2j/d) / 2 pi
        const double turns = (double)pos * exp2(a.log2_theta * (-2.0 * j / D) - 2.6514961294723188);
        sincospif((float)(2.0 * (turns - rint(turns))), &s_sin[t][j], &s_cos[t][j]);
    }
    __syncthreads();
    uint16_t *const kv = static_cast<uint16_t *>(a.p.kv);
#pragma unroll 1
    for (int t = 0; t < tokens; ++t) {
        const float4 c = *reinterpret_cast<const float4 *>(&s_cos[t][at]);
        const float4 s = *reinterpret_cast<const float4 *>(&s_sin[t][at]);
#pragma unroll 1
        for (int h0 = 0; h0 < heads; h0 += kRopeRows * kSubs) {
            if (t || h0) load(t, h0);
#pragma unroll
            for (int x = 0; x < kRopeRows; ++x) {
                const int h = h0 + sub + x * kSubs;
                const bool is_q = h < a.nq, is_v = h >= a.nq + nkv;
                const uint16_t *gain = is_q ? a.q_gain : a.k_gain;
                float4 l = lo[x], u = hi[x];
                if (a.q_gain || a.k_gain) {  // every lane of the warp: the sum needs them all
                    float ss = h < heads && !is_v ? dot4(l, l) + dot4(u, u) : 0.f;
#pragma unroll
                    for (int o = LR / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float n = rsqrtf(ss * (1.f / D) + a.eps);
                    if (gain && !is_v) {
                        l = mul4(scale4(l, n), load4<false, true>(gain, at));
                        u = mul4(scale4(u, n), load4<false, true>(gain, at + D / 2));
                    }
                }
                if (h >= heads || (!is_q && !s_write[t])) continue;
                if (!is_v) {
                    const float4 v = l;
                    l = make_float4(v.x * c.x - u.x * s.x, v.y * c.y - u.y * s.y, v.z * c.z - u.z * s.z,
                                    v.w * c.w - u.w * s.w);
                    u = make_float4(u.x * c.x + v.x * s.x, u.y * c.y + v.y * s.y, u.z * c.z + v.z * s.z,
                                    u.w * c.w + v.w * s.w);
                }
                uint16_t *to = is_q ? a.q + (size_t)(i * a.T + t0 + t) * a.q_stride + (size_t)h * D
                                    : kv + (is_v ? a.v_off : a.k_off) + s_row[t] +
                                          (size_t)(h - a.nq - (is_v ? nkv : 0)) * a.p.page_size * D;
                store4<BF16>(to + at, l);
                store4<BF16>(to + at + D / 2, u);
            }
        }
    }
}

template <int D, bool F32, bool BF16>
static void launch_rope_as(const RopeArgs &a, cudaStream_t s) {
    // 4 tokens a CTA once that still gives every SM two
    if ((long long)a.n * a.T >= 2 * kRopeTokens * pages_sms())
        qk_rope_kernel<D, F32, BF16, kRopeTokens>
            <<<(unsigned)(a.n * ((a.T + kRopeTokens - 1) / kRopeTokens)), kRopeThreads, 0, s>>>(a);
    else
        qk_rope_kernel<D, F32, BF16, 1><<<(unsigned)(a.n * a.T), kRopeThreads, 0, s>>>(a);
}

template <int D>
static cudaError_t launch_rope(const RopeArgs &a, bool f32, cudaStream_t s) {
    const bool bf16 = a.p.dtype == MK_BF16;
    if (f32 && bf16) launch_rope_as<D, true, true>(a, s);
    if (f32 && !bf16) launch_rope_as<D, true, false>(a, s);
    if (!f32 && bf16) launch_rope_as<D, false, true>(a, s);
    if (!f32 && !bf16) launch_rope_as<D, false, false>(a, s);
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
    // q in place of qkv's own q heads is fine: the lanes that write a value are those that read it, before
    const bool in_place = q == qkv && qkv_dtype == p->dtype && q_stride == qkv_stride;
    const size_t wide = qkv_dtype == MK_FP32 ? 4 : 2;
    if (!in_place && pages_rows_meet(qkv, (size_t)(n_heads + 2 * p->n_kv_heads) * d * wide, (size_t)qkv_stride * wide, q,
                                     (size_t)n_heads * d * 2, (size_t)q_stride * 2, (size_t)n * T))
        return pages_refuse(who, "q must not overlap qkv, other than in place of its q heads");
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
