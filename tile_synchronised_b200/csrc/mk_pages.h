// mk_pages.h -- what the kernels over a paged KV cache share: the device view
// of mk_pages, its sticky error word, and the lookup of a listed sequence.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/mk.h"
#include "mk_device.cuh"

namespace mk {

constexpr int kPagesMaxSeqs = 1024;     // rows of the table: one thread each in the management kernels
constexpr int kPagesMaxPages = 1 << 19; // pages of a pool: two bits each in shared memory (pages_copy_kernel)

// Words of mk_pages.state: the first error (code, entry, value); the pages
// that a reserve has to copy (count, then source and destination of each);
// one ticket per listed sequence for the last CTA of a compact (zero between
// launches).
constexpr int kStErr = 0, kStEntry = 1, kStValue = 2, kStCopies = 4, kStList = 8;
constexpr int kStTickets = kStList + 2 * kPagesMaxSeqs;
constexpr int kPagesStateInts = kStTickets + kPagesMaxSeqs;

// Error codes of the state's first word (see pages_message).
enum PagesError {
    kPgSeq = 1,       // a sequence index out of range, or listed twice
    kPgCount = 2,     // a count, length or kept index out of range
    kPgPosition = 3,  // a position past the table's width, or without a page
    kPgFull = 4,      // not enough free pages
    kPgShared = 5,    // a write to a page that another sequence holds too
    kPgPage = 6,      // a page index out of range, or written twice
    kPgBusy = 7,      // the destination of a fork is not empty
    kPgTimeout = 8    // a bounded device-side wait ran out
};

__device__ __forceinline__ void pages_fail(int *state, int code, int entry, int value) {
    if (atomicCAS(state + kStErr, 0, code) == 0) {
        state[kStEntry] = entry;
        state[kStValue] = value;
    }
}

// Offset in 16-bit elements of page `page` of one layer's K (kv = 0) or V (1).
__host__ __device__ inline size_t pages_offset(const mk_pages &p, int kv, int layer, int page) {
    return (((size_t)kv * p.n_layers + layer) * p.n_pages + page) * p.n_kv_heads * (size_t)p.page_size * p.head_dim;
}

// A listed sequence: its row, committed length and new tokens; `fresh` is 0
// for an entry that is out of range, which `err` then names.
struct PagesEntry {
    int seq, len, fresh, err;
};
__device__ __forceinline__ PagesEntry pages_entry(const mk_pages &p, const int *seqs, const int *n_new, int i, int T) {
    PagesEntry e{seqs[i], 0, 0, 0};
    if (e.seq < 0 || e.seq >= p.max_seqs) {
        e.err = kPgSeq;
        return e;
    }
    const int fresh = n_new ? n_new[i] : T;
    e.len = p.lengths[e.seq];
    if (fresh < 0 || fresh > T || e.len < 0)
        e.err = kPgCount;
    else if ((long long)e.len + fresh > (long long)p.max_pages * p.page_size)
        e.err = kPgPosition;
    else
        e.fresh = fresh;
    return e;
}

// 16-bit storage types of the cache.
template <bool BF16>
__device__ __forceinline__ uint16_t to16(float v) {
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    return __half_as_ushort(__float2half_rn(v));
}
template <bool BF16>
__device__ __forceinline__ float from16(uint16_t v) {
    if constexpr (BF16) return bf2f(v);
    return __half2float(__ushort_as_half(v));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Host: checks of a cache's geometry and pointers and of `layer` (-1: none);
// a refusal with its reason in the op error; a launch's result; the SM count.
mk_status pages_check(const mk_pages *p, int layer, const char *who);
mk_status pages_refuse(const char *who, const char *why, mk_status st = MK_ERR_INVALID);
mk_status pages_launched(cudaError_t e, const char *who);
// `rows` rows of width_a bytes, stride_a bytes apart from a on, and as many from
// b on: can they have a byte in common?  Exact where the strides are the same;
// else rows that lie between each other's count as common.
bool pages_rows_meet(const void *a, size_t width_a, size_t stride_a, const void *b, size_t width_b, size_t stride_b,
                     size_t rows);
int pages_sms();

}  // namespace mk
