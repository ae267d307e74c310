// mk_pages.cu -- managing the pages of a KV cache: reserving them (with copy
// on write of a shared last page), forking, compacting and freeing
// sequences, and copying pages.
//
// A page belongs to refs[page] sequences and is free at 0, so the reference
// counts are the whole allocator state: a free page is found by scanning
// them, lowest index first, which keeps every result deterministic (no free
// list whose order depends on history).  The scan costs 4 bytes a page, read
// by one CTA: all of them once, to know that the free ones suffice, and from
// the first page on until enough are found.  16 reserves of a page each, us, with
// the free pages in front and at the end: 4000 pages 7 and 7, 50000 13 and 37,
// 200000 35 and 139, 2^19 80 and 353.
//
// The bookkeeping kernels run as one CTA of 1024 threads, one per listed
// sequence (a table has at most 1024 rows): what they have to order (which
// sequence gets which page, which of several sharers of a page copies it) is
// a prefix sum over the list.  The data kernels (copies of whole pages, moves
// of positions) run on all SMs and are bound by HBM.  Freeing, forking and
// reserving 24 sequences with a copy of every last page (16 layers, 99 MB read
// and written): 23.5 us; cutting, reserving, copying and compacting 16 drafts (32
// layers, 249 MB): 46 us, 0.84 of the measured copy; with hardly any data: 10 us,
// the four launches.
#include <atomic>
#include <cstdio>

#include "mk_kernel.h"
#include "mk_pages.h"
#include "mk_tc.cuh"

namespace mk {

constexpr int kMgThreads = 1024;
constexpr int kCpThreads = 256;
constexpr int kCpLoads = 4;                                // 16-byte loads in flight per thread
constexpr int kCpUnit = kCpThreads * kCpLoads * 16;        // bytes of one CTA step of a page copy
constexpr int kCmBlock = 256;                              // kept positions whose offsets a CTA holds at a time
constexpr int kCmLoads = 8;                                // positions a thread reads before it writes any

// Exclusive prefix sum over the CTA's 1024 threads; `total` is their sum.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // an earlier call's sums have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    total = warp_sums[31];
    return x - v + (warp ? warp_sums[warp - 1] : 0);
}

__device__ __forceinline__ int pages_of(long long positions, int ps) { return (int)((positions + ps - 1) / ps); }

// Is entry i the only one of its value in the list?
__device__ __forceinline__ bool only_one(const int *list, int n, int i) {
    bool ok = true;
    for (int k = 0; k < n; ++k) ok = ok && (k == i || list[k] != list[i]);
    return ok;
}

// Thread i makes sure that positions len .. len + counts[i] - 1 of sequence
// seqs[i] lie in pages that it holds alone.  It takes one page for every table
// entry of that range that has none, and one in place of its partly filled
// last page while another sequence holds that too (of several listed sharers
// of a page each copies as long as another holder is left, in list order).
// The k-th taken entry, in list order, gets the k-th lowest free page.  The
// pages to copy go to the list in `state` for pages_cow_kernel.
__global__ void __launch_bounds__(kMgThreads, 1)
    pages_reserve_kernel(mk_pages p, const int *seqs, const int *counts, int n) {
    __shared__ int sums[32];
    __shared__ int s_seq[kPagesMaxSeqs], s_page[kPagesMaxSeqs], s_at[kPagesMaxSeqs], s_cow_at[kPagesMaxSeqs];
    __shared__ int s_first[kPagesMaxSeqs], s_miss[kPagesMaxSeqs];
    pdl_launch_dependents();
    const int i = threadIdx.x, ps = p.page_size;
    if (i < n) s_seq[i] = seqs[i];
    __syncthreads();
    int shared = -1, need = 0;
    if (i < n) {
        PagesEntry e = pages_entry(p, seqs, counts, i, 0x7fffffff);
        if (!e.err && !only_one(s_seq, n, i)) e.err = kPgSeq;
        if (e.err) {
            pages_fail(p.state, e.err, i, s_seq[i]);
        } else if (e.fresh) {
            const int first = e.len / ps, last = pages_of((long long)e.len + e.fresh, ps);
            const int *row = p.table + (size_t)e.seq * p.max_pages;
            // a row's pages are a prefix of it: the first entry of the range without one
            int lo = first, hi = last;
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (row[mid] < 0)
                    hi = mid;
                else
                    lo = mid + 1;
            }
            need = last - lo;
            if (e.len % ps && lo > first) {
                const int page = row[first];
                if (page < p.n_pages) {
                    shared = page;
                } else {  // the committed positions on it are lost: no new ones behind them
                    pages_fail(p.state, kPgPage, i, page);
                    need = 0;
                }
            }
            s_first[i] = first;
            s_miss[i] = lo;
        }
        s_page[i] = shared;
    }
    __syncthreads();
    bool cow = false;
    if (shared >= 0) {
        int earlier = 0;
        for (int k = 0; k < i; ++k) earlier += s_page[k] == shared;
        cow = p.refs[shared] - earlier > 1;
        need += cow;
    }
    need = min(need, p.n_pages + 1);  // more than there are: the sum stays within 32 bits
    int total, n_free, n_cow;
    const int at = block_scan(need, sums, total);
    int have = 0;
    for (int g = i; g < p.n_pages; g += kMgThreads) have += p.refs[g] == 0;
    block_scan(have, sums, n_free);
    const int cow_at = block_scan(cow, sums, n_cow);
    const bool fits = total <= n_free;  // enough free pages for everyone, or nobody gets any
    if (i == 0) {
        p.state[kStCopies] = fits ? n_cow : 0;
        if (!fits) pages_fail(p.state, kPgFull, total, n_free);
    }
    if (!fits || total == 0) return;
    if (i < n) {
        s_at[i] = at;
        s_cow_at[i] = cow ? cow_at : -1;
        if (cow) atomicSub(&p.refs[shared], 1);  // another holder is left: not free after it
    }
    for (int base = 0, found = 0; base < p.n_pages && found < total; base += kMgThreads) {
        const int g = base + i;
        const int is_free = g < p.n_pages && p.refs[g] == 0;
        int here;
        const int k = found + block_scan(is_free, sums, here);
        if (is_free && k < total) {
            int lo = 0, hi = n - 1;  // the last entry whose taken pages start at or before k
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_at[mid] <= k)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int t = k - s_at[lo], c = s_cow_at[lo];
            int col = s_miss[lo] + t;
            if (c >= 0) {
                col -= 1;
                if (t == 0) {
                    col = s_first[lo];
                    p.state[kStList + 2 * c] = s_page[lo];
                    p.state[kStList + 2 * c + 1] = g;
                }
            }
            p.refs[g] = 1;
            p.table[(size_t)s_seq[lo] * p.max_pages + col] = g;
        }
        found += here;
    }
}

// One CTA step of a page copy: the `unit`-th kCpUnit bytes of a slab (the K or
// V of one layer) of page a of `src` to page b of `dst`.
__device__ __forceinline__ void copy_unit(const mk_pages &dst, const mk_pages &src, int slab, int a, int b,
                                          size_t bytes, int unit) {
    const int kv = slab / dst.n_layers, layer = slab - kv * dst.n_layers;
    const char *from = static_cast<const char *>(src.kv) + pages_offset(src, kv, layer, a) * 2;
    char *to = static_cast<char *>(dst.kv) + pages_offset(dst, kv, layer, b) * 2;
    uint4 v[kCpLoads];
    size_t off = (size_t)unit * kCpUnit + threadIdx.x * 16;
#pragma unroll
    for (int k = 0; k < kCpLoads; ++k)
        if (off + (size_t)k * kCpThreads * 16 < bytes)
            v[k] = *reinterpret_cast<const uint4 *>(from + off + (size_t)k * kCpThreads * 16);
#pragma unroll
    for (int k = 0; k < kCpLoads; ++k)
        if (off + (size_t)k * kCpThreads * 16 < bytes)
            *reinterpret_cast<uint4 *>(to + off + (size_t)k * kCpThreads * 16) = v[k];
}

__device__ __forceinline__ size_t slab_bytes(const mk_pages &p) {
    return (size_t)p.n_kv_heads * p.page_size * p.head_dim * 2;
}

// The copies that a reserve listed in `state`.
__global__ void __launch_bounds__(kCpThreads) pages_cow_kernel(mk_pages p) {
    pdl_wait();
    const int count = p.state[kStCopies];
    const size_t bytes = slab_bytes(p);
    const int per = (int)((bytes + kCpUnit - 1) / kCpUnit), each = 2 * p.n_layers * per;
    for (long long u = blockIdx.x; u < (long long)count * each; u += gridDim.x) {
        const int c = (int)(u / each), r = (int)(u - (long long)c * each);
        copy_unit(p, p, r / per, p.state[kStList + 2 * c], p.state[kStList + 2 * c + 1], bytes, r % per);
    }
}

// dst page dst_pages[k] = src page src_pages[k], k < n, in every layer.  Each
// CTA marks the written pages in a bitmap of its own, so that a pair whose
// destination is written twice, or whose source is written by another pair of
// the same pool, is left out without any order between CTAs.
__global__ void __launch_bounds__(kCpThreads)
    pages_copy_kernel(mk_pages dst, mk_pages src, const int *src_pages, const int *dst_pages, int n) {
    extern __shared__ uint32_t bits[];  // written once, then written twice
    const int words = (dst.n_pages + 31) / 32;
    uint32_t *twice = bits + words;
    for (int k = threadIdx.x; k < 2 * words; k += kCpThreads) bits[k] = 0;
    __syncthreads();
    for (int k = threadIdx.x; k < n; k += kCpThreads) {
        const int b = dst_pages[k];
        if (b < 0 || b >= dst.n_pages) continue;
        const uint32_t bit = 1u << (b & 31);
        if (atomicOr(&bits[b >> 5], bit) & bit) atomicOr(&twice[b >> 5], bit);
    }
    __syncthreads();
    const bool same = src.kv == dst.kv;
    const size_t bytes = slab_bytes(dst);
    const int per = (int)((bytes + kCpUnit - 1) / kCpUnit), each = 2 * dst.n_layers * per;
    auto good = [&](int a, int b) {
        if (a < 0 || a >= src.n_pages || b < 0 || b >= dst.n_pages) return false;
        if (twice[b >> 5] >> (b & 31) & 1u) return false;
        return !(same && (bits[a >> 5] >> (a & 31) & 1u));
    };
    if (blockIdx.x == 0)
        for (int k = threadIdx.x; k < n; k += kCpThreads)
            if (!good(src_pages[k], dst_pages[k])) pages_fail(dst.state, kPgPage, k, dst_pages[k]);
    for (long long u = blockIdx.x; u < (long long)n * each; u += gridDim.x) {
        const int c = (int)(u / each), r = (int)(u - (long long)c * each);
        const int a = src_pages[c], b = dst_pages[c];
        if (good(a, b)) copy_unit(dst, src, r / per, a, b, bytes, r % per);
    }
}

// Sequence dst[i] becomes another holder of the pages of src[i]'s committed
// positions.
__global__ void __launch_bounds__(kMgThreads, 1)
    pages_fork_kernel(mk_pages p, const int *src, const int *dst, int n) {
    __shared__ int s_src[kPagesMaxSeqs], s_dst[kPagesMaxSeqs], s_held[kPagesMaxSeqs];
    const int i = threadIdx.x;
    if (i < n) {
        s_src[i] = src[i];
        s_dst[i] = dst[i];
    }
    __syncthreads();
    if (i < n) {
        const int a = s_src[i], b = s_dst[i];
        int err = 0;
        if (a < 0 || a >= p.max_seqs || b < 0 || b >= p.max_seqs || !only_one(s_dst, n, i)) err = kPgSeq;
        for (int k = 0; k < n; ++k)
            if (s_src[k] == b) err = kPgSeq;
        int held = -1;
        if (!err) {
            const int len = p.lengths[a];
            if (p.lengths[b] != 0 || p.table[(size_t)b * p.max_pages] >= 0)
                err = kPgBusy;
            else if (len < 0 || len > (long long)p.max_pages * p.page_size)
                err = kPgCount;
            else
                held = pages_of(len, p.page_size);
        }
        if (err) pages_fail(p.state, err, i, b);
        s_held[i] = held;
    }
    __syncthreads();
    for (int k = threadIdx.x >> 5; k < n; k += kMgThreads / 32) {
        if (s_held[k] < 0) continue;
        const int *from = p.table + (size_t)s_src[k] * p.max_pages;
        bool ok = true;
        for (int j = threadIdx.x & 31; j < s_held[k]; j += 32) {
            const int page = from[j];
            if (page >= 0 && page < p.n_pages) continue;
            pages_fail(p.state, kPgPosition, k, page);
            ok = false;
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) continue;  // a hole in the source's row
        for (int j = threadIdx.x & 31; j < s_held[k]; j += 32) {
            p.table[(size_t)s_dst[k] * p.max_pages + j] = from[j];
            atomicAdd(&p.refs[from[j]], 1);
        }
        if ((threadIdx.x & 31) == 0) p.lengths[s_dst[k]] = p.lengths[s_src[k]];
    }
}

// Sequence seqs[i] is cut to lengths[i] positions (0 without `lengths`), and
// the pages behind them lose a holder.
__global__ void __launch_bounds__(kMgThreads, 1)
    pages_free_kernel(mk_pages p, const int *seqs, const int *lengths, int n) {
    __shared__ int s_seq[kPagesMaxSeqs], s_keep[kPagesMaxSeqs];
    const int i = threadIdx.x;
    if (i < n) s_seq[i] = seqs[i];
    __syncthreads();
    if (i < n) {
        const int s = s_seq[i], len = lengths ? lengths[i] : 0;
        int err = 0;
        if (s < 0 || s >= p.max_seqs || !only_one(s_seq, n, i))
            err = kPgSeq;
        else if (len < 0 || len > p.lengths[s])
            err = kPgCount;
        if (err)
            pages_fail(p.state, err, i, s);
        else
            p.lengths[s] = len;
        s_keep[i] = err ? p.max_pages : pages_of(len, p.page_size);
    }
    __syncthreads();
    for (int k = threadIdx.x >> 5; k < n; k += kMgThreads / 32) {
        if (s_keep[k] >= p.max_pages) continue;
        int *row = p.table + (size_t)s_seq[k] * p.max_pages;
        for (int base = s_keep[k]; base < p.max_pages; base += 32) {
            const int j = base + (threadIdx.x & 31);
            const int page = j < p.max_pages ? row[j] : -1;
            if (page >= 0) {
                row[j] = -1;
                if (page >= p.n_pages || atomicSub(&p.refs[page], 1) <= 0) {
                    if (page < p.n_pages) atomicAdd(&p.refs[page], 1);
                    pages_fail(p.state, kPgPage, k, page);
                }
            }
            if (__any_sync(0xFFFFFFFFu, page < 0)) break;  // a row's pages are a prefix of it
        }
    }
}

// The kept new tokens of sequence seqs[i] move together: position len + j
// gets what position len + keep[i][j] holds, j < n_keep[i], in every layer,
// and the sequence grows by n_keep[i].  keep is ascending, so position len + j
// is never a source of a later j: a thread that owns 16 bytes of a head's row
// moves them in order, reading kCmLoads positions before it writes them, and
// no thread waits for another.  The last CTA of a sequence updates its length.
__global__ void __launch_bounds__(kCpThreads)
    pages_compact_kernel(mk_pages p, const int *seqs, const int *n_keep, const int *keep, int width, int n) {
    __shared__ long long s_from[kCmBlock], s_to[kCmBlock];  // element offsets within a slab
    const int i = blockIdx.y, ps = p.page_size, d = p.head_dim;
    const int s = seqs[i], count = n_keep[i];
    int err = 0, value = s;
    if (s < 0 || s >= p.max_seqs) err = kPgSeq;
    for (int k = threadIdx.x; k < n; k += kCpThreads)
        if (k != i && seqs[k] == s) err = kPgSeq;
    const int len = err == kPgSeq && (s < 0 || s >= p.max_seqs) ? 0 : p.lengths[s];
    if (!err && (count < 0 || (keep && count > width) || len < 0)) err = kPgCount;
    if (!err && (long long)len + count > (long long)p.max_pages * ps) err = kPgPosition;
    const int *row = p.table + (size_t)(s < 0 || s >= p.max_seqs ? 0 : s) * p.max_pages;
    const int *kept = keep ? keep + (size_t)i * width : nullptr;
    int moved = count;  // the first j that moves
    if (__syncthreads_or(err) == 0) {
        for (int j = threadIdx.x; j < count; j += kCpThreads) {
            const int from = kept ? kept[j] : j;
            if (from < 0 || (j > 0 && kept && kept[j - 1] >= from)) {
                err = kPgCount;
                value = from;
                break;
            }
            if ((long long)len + from >= (long long)p.max_pages * ps) {
                err = kPgPosition;
                value = from;
                break;
            }
            const int a = row[(len + from) / ps], b = row[(len + j) / ps];
            if (a < 0 || a >= p.n_pages || b < 0 || b >= p.n_pages) {
                err = kPgPosition;
                value = from;
                break;
            }
            if (from != j) {
                moved = min(moved, j);
                if (p.refs[b] != 1) {
                    err = kPgShared;
                    value = b;
                    break;
                }
            }
        }
    }
    if (err && blockIdx.x == 0) pages_fail(p.state, err, i, value);
    const bool bad = __syncthreads_or(err);
    // moves start at the first of all threads' `moved`
    __shared__ int s_moved;
    if (threadIdx.x == 0) s_moved = count;
    __syncthreads();
    atomicMin(&s_moved, moved);
    __syncthreads();
    if (!bad) {
        const int per_row = d / 8, cols = 2 * p.n_layers * p.n_kv_heads * per_row;
        const int col = blockIdx.x * kCpThreads + threadIdx.x;
        const int slab = col / (p.n_kv_heads * per_row), r = col - slab * p.n_kv_heads * per_row;
        const int head = r / per_row, part = r - head * per_row;
        uint16_t *base = static_cast<uint16_t *>(p.kv) + (size_t)slab * p.n_pages * p.n_kv_heads * ps * d +
                         (size_t)head * ps * d + part * 8;
        for (int j0 = s_moved; j0 < count; j0 += kCmBlock) {
            const int m = min(kCmBlock, count - j0);
            __syncthreads();
            for (int k = threadIdx.x; k < m; k += kCpThreads) {
                const int from = len + kept[j0 + k], to = len + j0 + k;
                s_from[k] = ((long long)row[from / ps] * p.n_kv_heads * ps + from % ps) * d;
                s_to[k] = ((long long)row[to / ps] * p.n_kv_heads * ps + to % ps) * d;
            }
            __syncthreads();
            if (col < cols)
                for (int k = 0; k < m; k += kCmLoads) {
                    uint4 v[kCmLoads];
#pragma unroll
                    for (int e = 0; e < kCmLoads; ++e)
                        if (k + e < m) v[e] = *reinterpret_cast<const uint4 *>(base + s_from[k + e]);
#pragma unroll
                    for (int e = 0; e < kCmLoads; ++e)
                        if (k + e < m) *reinterpret_cast<uint4 *>(base + s_to[k + e]) = v[e];
                }
        }
    }
    if (threadIdx.x == 0) {
        // every thread of this CTA read the length before the barriers above
        if (atomicAdd(&p.state[kStTickets + i], 1) == (int)gridDim.x - 1) {
            p.state[kStTickets + i] = 0;
            if (!bad) p.lengths[s] = len + count;
        }
    }
}

// ------------------------------------------------------------------ host side
int pages_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

mk_status pages_refuse(const char *who, const char *why, mk_status st) {
    char msg[240];
    snprintf(msg, sizeof msg, "%s: %s", who, why);
    set_op_error(msg);
    return st;
}

mk_status pages_check(const mk_pages *p, int layer, const char *who) {
    char msg[200];
    if (!p) return pages_refuse(who, "null pages");
    if (!p->kv || !p->table || !p->lengths || !p->refs || !p->state) return pages_refuse(who, "null pointer in pages");
    if (((uintptr_t)p->kv & 15) || (((uintptr_t)p->table | (uintptr_t)p->lengths | (uintptr_t)p->refs |
                                     (uintptr_t)p->state) & 3))
        return pages_refuse(who, "kv must be 16-byte aligned, the other arrays 4-byte");
    if (p->dtype != MK_BF16 && p->dtype != MK_FP16)
        return pages_refuse(who, "dtype must be MK_BF16 or MK_FP16", MK_ERR_UNSUPPORTED);
    if (p->head_dim != 64 && p->head_dim != 128 && p->head_dim != 256)
        return pages_refuse(who, "head_dim not in {64, 128, 256}", MK_ERR_UNSUPPORTED);
    if (p->n_layers < 1 || p->n_kv_heads < 1 || p->n_kv_heads > 1024 || p->n_layers > 4096 || p->page_size < 1 ||
        p->n_pages < 1 || p->n_pages > kPagesMaxPages || p->max_seqs < 1 || p->max_seqs > kPagesMaxSeqs ||
        p->max_pages < 1 || (long long)p->max_pages * p->page_size > (1 << 30)) {
        snprintf(msg, sizeof msg, "bad geometry (%d layers, %d KV heads, %d pages of %d, table %d x %d)", p->n_layers,
                 p->n_kv_heads, p->n_pages, p->page_size, p->max_seqs, p->max_pages);
        return pages_refuse(who, msg);
    }
    if (p->page_size % 16 && p->max_pages > 1)
        return pages_refuse(who, "page_size must be a multiple of 16 unless a sequence is one page",
                            MK_ERR_UNSUPPORTED);
    if (layer < -1 || layer >= p->n_layers) return pages_refuse(who, "layer out of range");
    return MK_OK;
}

mk_status pages_launched(cudaError_t e, const char *who) {
    if (e == cudaSuccess) return MK_OK;
    char msg[160];
    snprintf(msg, sizeof msg, "%s: launch failed: %s", who, cudaGetErrorString(e));
    set_op_error(msg);
    return MK_ERR_CUDA;
}

bool pages_rows_meet(const void *a, size_t width_a, size_t stride_a, const void *b, size_t width_b, size_t stride_b,
                     size_t rows) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    if (x + (rows - 1) * stride_a + width_a <= y || y + (rows - 1) * stride_b + width_b <= x) return false;
    if (stride_a != stride_b) return true;
    const size_t ahead = x <= y ? (y - x) % stride_a : (stride_a - (x - y) % stride_a) % stride_a;
    return ahead < width_a || ahead + width_b > stride_a;
}

static const char *pages_message(int code) {
    switch (code) {
        case kPgSeq: return "a sequence index is out of range or listed twice (entry, sequence)";
        case kPgCount: return "a count, length or kept index is out of range (entry, value)";
        case kPgPosition: return "a position has no page (entry, value)";
        case kPgFull: return "not enough free pages (needed, free)";
        case kPgShared: return "a write to a page that another sequence holds too: reserve first (entry, value)";
        case kPgPage: return "a page index is out of range, written twice or not held (entry, page)";
        case kPgBusy: return "the destination of a fork is not empty (entry, sequence)";
        case kPgTimeout: return "a device-side wait ran out";
        default: return "unknown error";
    }
}

static size_t pages_bytes(const mk_pages &p) {
    return (size_t)2 * p.n_layers * p.n_pages * p.n_kv_heads * p.page_size * p.head_dim * 2;
}

// A list of n sequences: 0 means nothing to do.
static mk_status pages_list(const mk_pages *p, int n, const void *a, const void *b, const char *who) {
    const mk_status st = pages_check(p, -1, who);
    if (st != MK_OK) return st;
    if (n < 0 || n > p->max_seqs) return pages_refuse(who, "the list must have between 0 and max_seqs entries");
    if (n && (!a || !b)) return pages_refuse(who, "null list");
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_pages_state_bytes(void) { return kPagesStateInts * sizeof(int32_t); }

extern "C" mk_status mk_pages_reserve(const mk_pages *p, const int32_t *seqs, const int32_t *counts, int n,
                                      void *stream) {
    const mk_status st = pages_list(p, n, seqs, counts, "pages_reserve");
    if (st != MK_OK || n == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    pages_reserve_kernel<<<1, kMgThreads, 0, s>>>(*p, seqs, counts, n);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        // at most one page a listed sequence
        const long long bytes = (long long)p->n_kv_heads * p->page_size * p->head_dim * 2;
        const long long units = 2LL * p->n_layers * n * ((bytes + kCpUnit - 1) / kCpUnit), most = 8LL * pages_sms();
        cfg.gridDim = dim3((unsigned)(units < most ? units : most));
        cfg.blockDim = dim3(kCpThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, pages_cow_kernel, *p);
    }
    return pages_launched(e, "pages_reserve");
}

extern "C" mk_status mk_pages_fork(const mk_pages *p, const int32_t *src, const int32_t *dst, int n, void *stream) {
    const mk_status st = pages_list(p, n, src, dst, "pages_fork");
    if (st != MK_OK || n == 0) return st;
    pages_fork_kernel<<<1, kMgThreads, 0, static_cast<cudaStream_t>(stream)>>>(*p, src, dst, n);
    return pages_launched(cudaGetLastError(), "pages_fork");
}

extern "C" mk_status mk_pages_free(const mk_pages *p, const int32_t *seqs, const int32_t *lengths, int n,
                                   void *stream) {
    const mk_status st = pages_list(p, n, seqs, seqs, "pages_free");
    if (st != MK_OK || n == 0) return st;
    pages_free_kernel<<<1, kMgThreads, 0, static_cast<cudaStream_t>(stream)>>>(*p, seqs, lengths, n);
    return pages_launched(cudaGetLastError(), "pages_free");
}

extern "C" mk_status mk_pages_compact(const mk_pages *p, const int32_t *seqs, const int32_t *n_keep,
                                      const int32_t *keep, int width, int n, void *stream) {
    const mk_status st = pages_list(p, n, seqs, n_keep, "pages_compact");
    if (st != MK_OK || n == 0) return st;
    if (keep && width < 1) return pages_refuse("pages_compact", "width must be positive");
    const long long cols = 2LL * p->n_layers * p->n_kv_heads * (p->head_dim / 8);
    const unsigned grid = keep ? (unsigned)((cols + kCpThreads - 1) / kCpThreads) : 1u;
    pages_compact_kernel<<<dim3(grid, n), kCpThreads, 0, static_cast<cudaStream_t>(stream)>>>(*p, seqs, n_keep, keep,
                                                                                              width, n);
    return pages_launched(cudaGetLastError(), "pages_compact");
}

extern "C" mk_status mk_pages_copy(const mk_pages *dst, const mk_pages *src, const int32_t *src_pages,
                                   const int32_t *dst_pages, int n, void *stream) {
    mk_status st = pages_check(dst, -1, "pages_copy");
    if (st == MK_OK) st = pages_check(src, -1, "pages_copy");
    if (st != MK_OK) return st;
    if (dst->n_layers != src->n_layers || dst->n_kv_heads != src->n_kv_heads || dst->head_dim != src->head_dim ||
        dst->page_size != src->page_size || dst->dtype != src->dtype)
        return pages_refuse("pages_copy", "the pools' pages must have the same shape and type");
    if (n < 0 || n > dst->n_pages || (n && (!src_pages || !dst_pages)))
        return pages_refuse("pages_copy", "needs 0 <= n <= n_pages and two lists");
    // The kernel takes two pools for one where their pages are the same bytes; other pools must have no byte in common.
    const bool same = dst->kv == src->kv && dst->n_pages == src->n_pages;
    const uintptr_t d0 = (uintptr_t)dst->kv, s0 = (uintptr_t)src->kv;
    if (!same && d0 < s0 + pages_bytes(*src) && s0 < d0 + pages_bytes(*dst))
        return pages_refuse("pages_copy", "the pools overlap and are not the same pool");
    if (n == 0) return MK_OK;
    const int smem = 2 * ((dst->n_pages + 31) / 32) * 4;
    if (smem > 48 * 1024) {
        // raised to the largest pool's at once: raised to this pool's, another thread's call could lower it again
        // before the launch
        static std::atomic<unsigned long long> configured{0};
        const cudaError_t e = tc_allow_smem(reinterpret_cast<const void *>(pages_copy_kernel),
                                            2 * (kPagesMaxPages / 32) * 4, configured);
        if (e != cudaSuccess) return pages_launched(e, "pages_copy");
    }
    const long long bytes = (long long)dst->n_kv_heads * dst->page_size * dst->head_dim * 2;
    const long long units = 2LL * dst->n_layers * n * ((bytes + kCpUnit - 1) / kCpUnit);
    const long long most = 8LL * pages_sms();
    pages_copy_kernel<<<(unsigned)(units < most ? units : most), kCpThreads, smem,
                        static_cast<cudaStream_t>(stream)>>>(*dst, *src, src_pages, dst_pages, n);
    return pages_launched(cudaGetLastError(), "pages_copy");
}

extern "C" mk_status mk_pages_status(const mk_pages *p, void *stream) {
    const mk_status st = pages_check(p, -1, "pages_status");
    if (st != MK_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int32_t w[4] = {0, 0, 0, 0};
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(s, &capture);
    if (e == cudaSuccess && capture != cudaStreamCaptureStatusNone)  // a wait would end the capture
        return pages_refuse("pages_status", "the stream is being captured", MK_ERR_STATE);
    if (e == cudaSuccess) e = cudaMemcpyAsync(w, p->state, sizeof w, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && w[kStErr]) e = cudaMemsetAsync(p->state, 0, sizeof w, s);
    if (e != cudaSuccess) return pages_launched(e, "pages_status");
    if (!w[kStErr]) return MK_OK;
    char msg[200];
    snprintf(msg, sizeof msg, "pages: %s: %d, %d", pages_message(w[kStErr]), w[kStEntry], w[kStValue]);
    set_op_error(msg);
    return w[kStErr] == kPgTimeout ? MK_ERR_TIMEOUT : w[kStErr] == kPgFull ? MK_ERR_STATE : MK_ERR_INVALID;
}
