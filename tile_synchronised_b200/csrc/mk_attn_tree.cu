// mk_attn_tree.cu -- attention of the new tokens of every sequence (a drafted
// tree, a chunk of a prompt, a single token) over a paged KV cache, on the
// 5th-generation tensor cores.
//
//   out[t][h] = sum_j p_j V_j,  p = softmax_j(q[t][h] . K_j / sqrt(d)),
//   j over the committed positions 0 .. len - 1 and those new tokens u (at
//   positions len + u) whose bit is set in row t of the mask (u <= t without
//   a mask).
//
// The T new tokens of the G = nq / nkv query heads that share a KV head are
// the rows of one matrix (row r = t G + g), up to 128 of them the M of an MMA,
// so the cache is read once for all of them and the arithmetic (4 d flops per
// row and position) stays behind the memory traffic (4 d bytes per position)
// for up to about 250 rows.  Per tile of NT positions:
//     S = Q K^T  (tensor memory, M = 128, N = NT), softmax in registers,
//     P (16 bit, tensor memory, over S) and O += P V (tensor memory, N = d).
// One thread owns one row of S, so the running maximum and sum need no
// exchange.  O is rescaled only when the maximum grew by more than 2^8 since
// the last rescale: P and the sum then stay within 32-bit range of the older
// maximum and the quotient is the same.
//
// Work: the units are (sequence, KV head, row tile, tile of positions), the
// tiles of one row tile consecutive; each CTA (one per SM) takes an equal
// contiguous range, whatever the lengths, which are only known on the device.
// A CTA that covers all tiles of an item writes its rows of `out`; else it
// writes (o, max, sum) to scratch, at most two such records per CTA, and
// tree_combine_kernel joins them.
//
// Roles: warps 0-3 softmax (thread = row), one warp loads K and V tiles by
// TMA into a ring (a page's share of a tile per copy; lanes look up the page
// table two tiles ahead), one lane issues the MMAs: QK of the next tile goes
// out before PV of this one, so the tensor core works while the softmax runs.
//
// P is rounded to the cache's 16-bit type (2^-9 relative in bf16, each
// element on its own, as V's own storage); S, the maximum, the sum, O and the
// records are 32 bits.
#include <cuda.h>
#include <math_constants.h>

#include <atomic>
#include <cmath>

#include "mk_kernel.h"
#include "mk_pages.h"
#include "mk_tc.cuh"

namespace mk {

constexpr int kTreeM = 128;          // rows of an MMA
constexpr int kTreeMaxStages = 12;

struct TreeArgs {
    mk_pages p;
    const uint16_t *q;
    uint16_t *out;
    long long q_stride, out_stride;  // 16-bit elements between tokens
    const int *seqs, *n_new;
    const uint32_t *mask;
    float *part_o;   // [2 x CTAs][rows_cap][d]
    float2 *part_ml; // [2 x CTAs][rows_cap]: maximum (base 2, scaled), sum
    const uint16_t *k, *v;  // this layer's pages
    int n, T, words, nq, G, seg, stages, rows_cap;
    float scale;     // log2(e) / sqrt(d)
};

// What one listed sequence needs: units, and the walk over a CTA's range.
struct TreeEntry {
    int seq, len, fresh;
};

__host__ __device__ constexpr int tree_nt(int d) { return d == 256 ? 64 : 128; }

// Shared memory behind the operand tiles.
struct TreeShared {
    uint64_t full[kTreeMaxStages], empty[kTreeMaxStages];
    uint64_t s_full[2], p_full[2], pv_done, q_full;
    uint32_t tmem;
    int abort, bad_v, pad;
};

// The units of entry e: KV heads x row tiles x tiles of positions.
__device__ __forceinline__ long long tree_units(const TreeArgs &a, const TreeEntry &e, int nt) {
    if (!e.fresh) return 0;
    const int rt = (e.fresh * a.G + kTreeM - 1) / kTreeM, tiles = (e.len + e.fresh + nt - 1) / nt;
    return (long long)a.p.n_kv_heads * rt * tiles;
}

// A run of tiles of one item that one CTA works through.
struct TreeSeg {
    int i, g, rt, t0, t1, tiles, slot;
    TreeEntry e;
};

struct TreeWalk {
    long long u, u1;
    int i, count;
    const long long *pref;  // [n + 1] units before each entry
    const TreeEntry *ent;
    // the next run, false at the end of the CTA's range
    __device__ __forceinline__ bool next(const TreeArgs &a, int nt, TreeSeg &s) {
        if (u >= u1) return false;
        while (pref[i + 1] <= u) ++i;
        s.i = i;
        s.e = ent[i];
        s.tiles = (s.e.len + s.e.fresh + nt - 1) / nt;
        const int rts = (s.e.fresh * a.G + kTreeM - 1) / kTreeM;
        const long long local = u - pref[i];
        const int item = (int)(local / s.tiles);
        s.t0 = (int)(local - (long long)item * s.tiles);
        s.g = item / rts;
        s.rt = item - s.g * rts;
        const long long left = u1 - u;
        s.t1 = left < s.tiles - s.t0 ? s.t0 + (int)left : s.tiles;
        s.slot = 2 * blockIdx.x + (count ? 1 : 0);
        ++count;
        u += s.t1 - s.t0;
        return true;
    }
};

// The CTAs that share U units out of `most`: at least kTreeMinUnits each.
constexpr int kTreeMinUnits = 2;
__device__ __forceinline__ int tree_ctas(long long U, int most) {
    const long long want = (U + kTreeMinUnits - 1) / kTreeMinUnits;
    return want < most ? (int)(want > 0 ? want : 1) : most;
}
__device__ __forceinline__ long long tree_first(long long U, int ctas, int c) { return U * c / ctas; }

// 32 visibility bits of row `row` (a new token) for new tokens 32 k .. 32 k + 31
// (k < 0: committed positions, all visible).
__device__ __forceinline__ uint32_t tree_word(const TreeArgs &a, int i, int t, int fresh, int k) {
    if (k < 0) return 0xFFFFFFFFu;
    const int u0 = k * 32;
    if (u0 >= fresh) return 0u;
    uint32_t w;
    if (a.mask)
        w = a.mask[((size_t)i * a.T + t) * a.words + k];
    else
        w = u0 > t ? 0u : (t - u0 >= 31 ? 0xFFFFFFFFu : (2u << (t - u0)) - 1u);
    return fresh - u0 >= 32 ? w : w & ((1u << (fresh - u0)) - 1u);
}
// ... for positions pos .. pos + 31.
__device__ __forceinline__ uint32_t tree_bits(const TreeArgs &a, int i, int t, const TreeEntry &e, int pos) {
    const int u = pos - e.len;
    const int k = u >> 5, sh = u & 31;
    const uint32_t lo = tree_word(a, i, t, e.fresh, k);
    return sh ? __funnelshift_r(lo, tree_word(a, i, t, e.fresh, k + 1), sh) : lo;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 consecutive fp32 columns of this thread's tensor-memory lane (no wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem]: operand A is P, 16-bit pairs in 32-bit columns.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(0u)
        : "memory");
}

// kind::f16, fp32 accumulate, A and B both bf16 or both fp16, A K-major, B
// K-major (K) or MN-major (V: positions are its K, d is contiguous).
template <bool BF16>
__host__ __device__ constexpr uint32_t tree_idesc(int n, bool b_mn) {
    return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTreeM >> 4) << 24);
}

template <bool BF16>
__device__ __forceinline__ bool any_nonfinite(const uint4 &v) {
    constexpr uint32_t lo = BF16 ? 0x00007F80u : 0x00007C00u, hi = lo << 16;
    bool bad = false;
    for (uint32_t w : {v.x, v.y, v.z, v.w}) bad = bad || (w & lo) == lo || (w & hi) == hi;
    return bad;
}

// The share of new tokens whose V holds an infinity or NaN.  In the MMA those
// rows of V are zeros, since 0 x inf in a row that does not see the token
// would be NaN; here every row that does see one adds p V itself, columns
// c0 .. c0 + 31.  Rarely runs.
template <int D, bool BF16>
__device__ __noinline__ void tree_add_nonfinite(const TreeArgs &a, const TreeSeg &s, int nt, int row, float m2,
                                                float bias, int c0, float *o) {
    const int t = row / a.G;
    const uint16_t *q = a.q + ((size_t)s.i * a.T + t) * a.q_stride + (size_t)(s.g * a.G + row % a.G) * D;
    const int from = max(s.e.len, s.t0 * nt), to = min(s.e.len + s.e.fresh, s.t1 * nt);
    for (int pos = from; pos < to; ++pos) {
        if (!(tree_bits(a, s.i, t, s.e, pos) & 1u)) continue;
        const int page = a.p.table[(size_t)s.e.seq * a.p.max_pages + pos / a.p.page_size];
        if (page < 0 || page >= a.p.n_pages) continue;
        const size_t at = (((size_t)page * a.p.n_kv_heads + s.g) * a.p.page_size + pos % a.p.page_size) * D;
        bool bad = false;
        for (int c = 0; c < D; c += 8) bad = bad || any_nonfinite<BF16>(*reinterpret_cast<const uint4 *>(a.v + at + c));
        if (!bad) continue;
        float dot = 0.f;
        for (int c = 0; c < D; ++c) dot = fmaf(from16<BF16>(q[c]), from16<BF16>(a.k[at + c]), dot);
        const float p = ex2(fmaf(dot, a.scale, bias - m2));
        for (int c = 0; c < 32; ++c) o[c] = fmaf(p, from16<BF16>(a.v[at + c0 + c]), o[c]);
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(192, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const TreeArgs a) {
    constexpr int NT = tree_nt(D), NH = D / 64;      // positions of a tile, 64-column blocks of a row
    constexpr uint32_t kQBytes = kTreeM * D * 2, kStage = NT * D * 2;
    constexpr uint32_t kO = 256;                      // tensor-memory column of O; S at 0 and 128
    constexpr float kBias = BF16 ? 0.f : 7.f;         // fp16 P: 2^7 above the maximum's 1, so that small
                                                      // values keep clear of its subnormals (at most 2^15)
    constexpr float kGrow = 8.f;                      // rescale O when the maximum grew by more (base 2)
    extern __shared__ __align__(1024) uint8_t tree_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tree_smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_q = smem, *ring = smem + kQBytes;
    const int S = a.stages;
    TreeShared &sh = *reinterpret_cast<TreeShared *>(ring + (size_t)S * kStage);
    long long *pref = reinterpret_cast<long long *>(&sh + 1);
    TreeEntry *ent = reinterpret_cast<TreeEntry *>(pref + a.n + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = &sh.abort;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], 4);
        }
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.q_full, 4);
        sh.abort = 0;
        sh.bad_v = 0;
        fence_barrier_init();
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the listed sequences and the units before each
    for (int i = tid; i < a.n; i += blockDim.x) {
        const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, i, a.T);
        if (e.err && blockIdx.x == 0) pages_fail(a.p.state, e.err, i, e.seq);
        ent[i] = TreeEntry{e.seq, e.len, e.fresh};
        pref[i + 1] = tree_units(a, ent[i], NT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) {
        long long carry = 0;
        for (int base = 0; base < a.n; base += 32) {
            long long x = base + lane < a.n ? pref[base + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
                if (lane >= o) x += y;
            }
            if (base + lane < a.n) pref[base + lane + 1] = carry + x;
            carry += __shfl_sync(0xFFFFFFFFu, x, 31);
        }
        if (lane == 0) pref[0] = 0;
    }
    __syncthreads();
    pdl_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sh.tmem);
    const long long U = pref[a.n];
    const int ctas = tree_ctas(U, gridDim.x);
    TreeWalk walk{0, 0, 0, 0, pref, ent};
    if ((int)blockIdx.x < ctas) {
        walk.u = tree_first(U, ctas, blockIdx.x);
        walk.u1 = tree_first(U, ctas, blockIdx.x + 1);
        int lo = 0, hi = a.n;  // the last entry that starts at or before u
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (pref[mid] <= walk.u)
                lo = mid;
            else
                hi = mid;
        }
        walk.i = lo;
    }
    TreeSeg sg;
    int issued = 0;  // ring loads the producer issued

    if (warp == 4) {
        // ---------------------------------------------------------- producer
        const int seg = a.seg, ns = NT / seg;
        const int nh = ns > 1 ? NH : 1;  // a whole tile's box covers every 64-column block
        const int my = lane / nh, blk = lane - my * nh;
        const int nkv = a.p.n_kv_heads, ps = a.p.page_size;
        const uint32_t seg_bytes = (uint32_t)seg * D * 2, off_smem = (uint32_t)(blk * NT + my * seg) * 128u;
        bool ok = true;
        while (ok && walk.next(a, NT, sg)) {
            const int *row = a.p.table + (size_t)sg.e.seq * a.p.max_pages;
            const int end = sg.e.len + sg.e.fresh;
            const bool mine = lane < ns * nh;
            auto look = [&](int t) {
                const int pos = t * NT + my * seg;
                return mine && t < sg.t1 && pos < end ? row[pos / ps] : -1;
            };
            int p0 = look(sg.t0), p1 = look(sg.t0 + 1);
            for (int t = sg.t0; ok && t < sg.t1; ++t) {
                const int p2 = look(t + 2);
                const int pos = t * NT + my * seg, off = pos - pos / ps * ps;
                const bool go = mine && pos < end;
                int page = p0;
                if (go && (page < 0 || page >= a.p.n_pages)) {
                    pages_fail(a.p.state, kPgPosition, sg.i, pos);
                    page = -1;  // out of the tensor: zeros
                }
                const int left = (end - t * NT + seg - 1) / seg;
                const uint32_t bytes = (uint32_t)(left < ns ? left : ns) * seg_bytes;
                for (int kv = 0; kv < 2; ++kv) {
                    const int s = issued % S;
                    if (issued >= S) ok = tc_wait(&sh.empty[s], ((issued / S) - 1) & 1u, abort);
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], bytes);
                    __syncwarp();
                    if (go)
                        tma_load_4d(ring + (size_t)s * kStage + off_smem, kv ? &map_v : &map_k, 0, off, blk,
                                    page < 0 ? -1 : page * nkv + sg.g, &sh.full[s]);
                    ++issued;
                }
                p0 = p1;
                p1 = p2;
            }
        }
    } else if (warp == 5) {
        // -------------------------------------------------------- MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_qk = tree_idesc<BF16>(NT, false), id_pv = tree_idesc<BF16>(D, true);
            int load = 0, tau = 0, seg_no = 0;  // ring loads used, tiles, runs
            bool ok = true;
            auto qk = [&](int x, int ld) {
                const int s = ld % S;
                if (!tc_wait(&sh.full[s], (ld / S) & 1u, abort)) return false;
                tc_fence_after();
                const uint8_t *st = ring + (size_t)s * kStage;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t blk = ks / 4, in = (ks % 4) * 32;
                    tc_mma(tmem + (uint32_t)(x & 1) * 128, smem_desc_sw128(s_q + blk * kTreeM * 128 + in, 16, 1024),
                           smem_desc_sw128(st + blk * NT * 128 + in, 16, 1024), id_qk, ks > 0);
                }
                tc_commit(&sh.s_full[x & 1]);
                tc_commit(&sh.empty[s]);
                return true;
            };
            while (ok && walk.next(a, NT, sg)) {
                const int nt = sg.t1 - sg.t0;
                ok = tc_wait(&sh.q_full, seg_no & 1u, abort);
                tc_fence_after();
                ok = ok && qk(tau, load);
                for (int i = 0; ok && i < nt; ++i) {
                    if (i + 1 < nt && !qk(tau + i + 1, load + 2 * i + 2)) {
                        ok = false;
                        break;
                    }
                    const int x = tau + i, ld = load + 2 * i + 1, s = ld % S;
                    if (!tc_wait(&sh.p_full[x & 1], (x >> 1) & 1u, abort) ||
                        !tc_wait(&sh.full[s], (ld / S) & 1u, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint8_t *st = ring + (size_t)s * kStage;
#pragma unroll
                    for (int ks = 0; ks < NT / 16; ++ks)
                        tc_mma_ta(tmem + kO, tmem + (uint32_t)(x & 1) * 128 + ks * 8,
                                  smem_desc_sw128(st + ks * 2048, NT * 128, 1024), id_pv, i > 0 || ks > 0);
                    tc_commit(&sh.pv_done);
                    tc_commit(&sh.empty[s]);
                }
                load += 2 * nt;
                tau += nt;
                ++seg_no;
            }
        }
    } else {
        // ----------------------------------------------------------- softmax
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        int load = 0, tau = 0;
        bool ok = true;
        while (walk.next(a, NT, sg)) {
            const int nt = sg.t1 - sg.t0, row0 = sg.rt * kTreeM, rows = min(kTreeM, sg.e.fresh * a.G - row0);
            const int row = row0 + tid, t = row / a.G;
            const bool live = tid < rows, warp_live = warp * 32 < rows;
            // Q rows of this item, swizzled as TMA would: 16-byte chunk c of
            // row r of a 64-column block goes to chunk c ^ (r mod 8)
            if (ok) {
                for (int x = lane; x < 32 * (D / 8); x += 32) {
                    const int r = warp * 32 + x / (D / 8), c = x % (D / 8);
                    if (r >= rows) continue;
                    const int rr = row0 + r, tt = rr / a.G;
                    const uint4 v = *reinterpret_cast<const uint4 *>(
                        a.q + ((size_t)sg.i * a.T + tt) * a.q_stride + (size_t)(sg.g * a.G + rr - tt * a.G) * D + c * 8);
                    *reinterpret_cast<uint4 *>(s_q + (c / 8) * kTreeM * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full);
            }
            float m = -CUDART_INF_F, l = 0.f;  // the maximum that P and the sum refer to (of S unscaled)
            for (int i = 0; ok && i < nt; ++i) {
                const int x = tau + i, p0 = (sg.t0 + i) * NT;
                const uint32_t sc = lanes + (uint32_t)(x & 1) * 128;
                ok = tc_wait(&sh.s_full[x & 1], (x >> 1) & 1u, abort);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                float s[NT];
                const bool tail = p0 + NT > sg.e.len;  // new tokens, or nothing, in this tile
                if (warp_live) {
#pragma unroll
                    for (int c = 0; c < NT; c += 32) tmem_ld32(sc + c, s + c);
                    tmem_wait_ld();
                    if (tail) {
#pragma unroll
                        for (int c = 0; c < NT; c += 32) {
                            const uint32_t w = live ? tree_bits(a, sg.i, t, sg.e, p0 + c) : 0u;
#pragma unroll
                            for (int k = 0; k < 32; ++k) s[c + k] = (w >> k) & 1u ? s[c + k] : -CUDART_INF_F;
                        }
                    }
                }
                if (i > 0) {
                    ok = tc_wait(&sh.pv_done, (x - 1) & 1u, abort);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tc_fence_after();
                }
                if (warp_live) {
                    float top = s[0];
#pragma unroll
                    for (int c = 1; c < NT; ++c) top = fmaxf(top, s[c]);
                    const bool grew = live && (top - m) * a.scale > kGrow;  // also from -inf
                    if (__any_sync(0xFFFFFFFFu, grew)) {
                        const float f = grew ? ex2((m - top) * a.scale) : 1.f;
                        if (grew) m = top;
                        l *= f;
                        if (i > 0) {
#pragma unroll
                            for (int c = 0; c < D; c += 32) {
                                float o[32];
                                tmem_ld32(lanes + kO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] *= f;
                                tmem_st32(lanes + kO + c, reinterpret_cast<const uint32_t *>(o));
                            }
                            tmem_wait_st();
                        }
                    }
                    const float ms = kBias - (m == -CUDART_INF_F ? 0.f : m) * a.scale;
                    uint32_t pk[NT / 2];
                    float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
                    for (int c = 0; c < NT; c += 2) {
                        const float e0 = ex2(fmaf(s[c], a.scale, ms)), e1 = ex2(fmaf(s[c + 1], a.scale, ms));
                        sum0 += e0;
                        sum1 += e1;
                        pk[c / 2] = pack16<BF16>(e0, e1);
                    }
                    l += sum0 + sum1;
#pragma unroll
                    for (int c = 0; c < NT / 2; c += 32) tmem_st32(sc + c, pk + c);
                    tmem_wait_st();
                }
                if (tail) {
                    // V rows of new tokens with an infinity or NaN, and rows
                    // behind the last token, become zeros
                    const int ld = load + 2 * i + 1, st = ld % S;
                    ok = tc_wait(&sh.full[st], (ld / S) & 1u, abort);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const int pos = p0 + tid;
                    if (tid < NT && pos >= sg.e.len) {
                        uint8_t *vr = ring + (size_t)st * kStage + tid * 128;
                        bool clear = pos >= sg.e.len + sg.e.fresh;
                        if (!clear) {
                            for (int c = 0; c < D / 8; ++c)
                                clear = clear || any_nonfinite<BF16>(*reinterpret_cast<const uint4 *>(
                                                     vr + (c / 8) * NT * 128 + (((c & 7) ^ (tid & 7)) << 4)));
                            if (clear) *reinterpret_cast<volatile int *>(&sh.bad_v) = 1;
                        }
                        if (clear)
                            for (int c = 0; c < D / 8; ++c)
                                *reinterpret_cast<uint4 *>(vr + (c / 8) * NT * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[x & 1]);
            }
            if (ok) ok = __all_sync(0xFFFFFFFFu, tc_wait(&sh.pv_done, (tau + nt - 1) & 1u, abort));
            tc_fence_after();
            load += 2 * nt;
            tau += nt;
            // ------------------------------------------------------ epilogue
            const bool whole = sg.t0 == 0 && sg.t1 == sg.tiles;
            const bool add = ok && *reinterpret_cast<volatile int *>(&sh.bad_v) && sg.t1 * NT > sg.e.len;
            const float nan = CUDART_NAN_F;
            if (warp_live) {
                const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                const int h = sg.g * a.G + row - t * a.G;
                uint16_t *to = a.out + ((size_t)sg.i * a.T + t) * a.out_stride + (size_t)h * D;
                float *rec = a.part_o + ((size_t)sg.slot * a.rows_cap + tid) * D;
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    if (ok) {
                        tmem_ld32(lanes + kO + c, o);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = nan;
                    }
                    if (live) {
                        if (add)
                            tree_add_nonfinite<D, BF16>(a, sg, NT, row, (m == -CUDART_INF_F ? 0.f : m) * a.scale,
                                                        kBias, c, o);
                        if (whole) {
#pragma unroll
                            for (int k = 0; k < 32; k += 8) {
                                uint4 w;
                                w.x = pack16<BF16>(o[k] * inv, o[k + 1] * inv);
                                w.y = pack16<BF16>(o[k + 2] * inv, o[k + 3] * inv);
                                w.z = pack16<BF16>(o[k + 4] * inv, o[k + 5] * inv);
                                w.w = pack16<BF16>(o[k + 6] * inv, o[k + 7] * inv);
                                *reinterpret_cast<uint4 *>(to + c + k) = w;
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                *reinterpret_cast<float4 *>(rec + c + k) =
                                    make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (live && !whole)
                    a.part_ml[(size_t)sg.slot * a.rows_cap + tid] = ok ? make_float2(m * a.scale, l) : make_float2(nan, nan);
            }
            tc_fence_before();
        }
    }
    // After a wait ran out some copies may be in flight: let the last one of
    // every stage land before the shared memory is freed.
    __syncwarp();
    if (warp == 4 && lane == 0 && *abort) {
        for (int x = issued > S ? issued - S : 0; x < issued; ++x)
            tc_drain(&sh.full[x % S], (uint32_t)(x / S) & 1u, kTcTimeoutNs);
        pages_fail(a.p.state, kPgTimeout, 0, blockIdx.x);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// Joins the records of every item that more than one CTA worked on: one warp
// per row, CTA (x, y, z) the rows 8 x .. 8 x + 7 of row tile z of KV head
// y of the entries in turn.
constexpr int kCombineRows = 8;

template <int D, bool BF16>
__global__ void __launch_bounds__(kCombineRows * 32) tree_combine_kernel(const TreeArgs a, int grid) {
    constexpr int NT = tree_nt(D), E = D / 32;
    __shared__ long long s_before, s_total;
    __shared__ long long s_red[2 * kCombineRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_rt = (kTreeM + kCombineRows - 1) / kCombineRows;
    const int i = blockIdx.y, rt = blockIdx.x / per_rt, r = (blockIdx.x - rt * per_rt) * kCombineRows + warp;
    const int g = blockIdx.z;
    // units before entry i, and of all entries
    long long before = 0, total = 0;
    for (int k = threadIdx.x; k < a.n; k += blockDim.x) {
        const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, k, a.T);
        const long long u = tree_units(a, TreeEntry{e.seq, e.len, e.fresh}, NT);
        total += u;
        if (k < i) before += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
    if (lane == 0) {
        s_red[2 * warp] = before;
        s_red[2 * warp + 1] = total;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        long long b = 0, t = 0;
        for (int k = 0; k < kCombineRows; ++k) {
            b += s_red[2 * k];
            t += s_red[2 * k + 1];
        }
        s_before = b;
        s_total = t;
    }
    __syncthreads();
    const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, i, a.T);
    const int row = rt * kTreeM + r;
    pdl_wait();  // the records are complete
    if (!e.fresh || row >= e.fresh * a.G) return;
    const int tiles = (e.len + e.fresh + NT - 1) / NT, rts = (e.fresh * a.G + kTreeM - 1) / kTreeM;
    const long long U = s_total, u0 = s_before + ((long long)g * rts + rt) * tiles, u1 = u0 + tiles;
    const int ctas = tree_ctas(U, grid);
    // the CTA of unit u is the last one whose first unit is at most u
    const int c0 = (int)(((u0 + 1) * ctas - 1) / U), c1 = (int)((u1 * ctas - 1) / U);
    if (c0 == c1) return;
    float M = -CUDART_INF_F;
    auto slot = [&](int c) { return (size_t)(2 * c + (tree_first(U, ctas, c) < u0 ? 1 : 0)) * a.rows_cap + r; };
    for (int c = c0; c <= c1; ++c) M = fmaxf(M, a.part_ml[slot(c)].x);
    float o[E], L = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) o[k] = 0.f;
    const float Ms = M == -CUDART_INF_F ? 0.f : M;
    for (int c = c0; c <= c1; ++c) {
        const size_t at = slot(c);
        const float2 ml = a.part_ml[at];
        const float f = ex2(ml.x - Ms);
        L = fmaf(f, ml.y, L);
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(a.part_o + at * D + k * 32 + lane * 2);
            o[k] = fmaf(f, v.x, o[k]);
            o[k + 1] = fmaf(f, v.y, o[k + 1]);
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int t = row / a.G;
    uint16_t *to = a.out + ((size_t)i * a.T + t) * a.out_stride + (size_t)(g * a.G + row - t * a.G) * D;
#pragma unroll
    for (int k = 0; k < E; k += 2)
        *reinterpret_cast<uint32_t *>(to + k * 32 + lane * 2) = pack16<BF16>(o[k] * inv, o[k + 1] * inv);
}

// ------------------------------------------------------------------ host side
static int tree_rows(int T, int G) { return (long long)T * G < kTreeM ? T * G : kTreeM; }

static size_t tree_scratch(int T, int nq, int nkv, int d, int grid) {
    return (size_t)2 * grid * tree_rows(T, nq / nkv) * (d + 2) * sizeof(float);
}

template <int D, bool BF16>
static cudaError_t launch_tree(const CUtensorMap &mk, const CUtensorMap &mv, TreeArgs &a, int grid, cudaStream_t s) {
    constexpr int stage = tree_nt(D) * D * 2;
    const int fixed = 1024 + kTreeM * D * 2 + (int)sizeof(TreeShared) + (a.n + 1) * 8 + a.n * (int)sizeof(TreeEntry);
    a.stages = (227 * 1024 - fixed) / stage;
    if (a.stages > kTreeMaxStages) a.stages = kTreeMaxStages;
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = tc_allow_smem(reinterpret_cast<const void *>(attn_tree_kernel<D, BF16>), 227 * 1024, configured);
    if (e != cudaSuccess) return e;
    attn_tree_kernel<D, BF16><<<grid, 192, fixed + a.stages * stage, s>>>(mk, mv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int rts = (int)(((long long)a.T * a.G + kTreeM - 1) / kTreeM);
    const int per_rt = rts > 1 ? kTreeM / kCombineRows : (a.T * a.G + kCombineRows - 1) / kCombineRows;
    cfg.gridDim = dim3((unsigned)(rts > 1 ? rts * per_rt : per_rt), (unsigned)a.n, (unsigned)a.p.n_kv_heads);
    cfg.blockDim = dim3(kCombineRows * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, BF16>, a, grid);
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_attention_tree_scratch_bytes(int T, int n_heads, int n_kv_heads, int head_dim) {
    if (T < 1 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || head_dim < 1) return 0;
    return tree_scratch(T, n_heads, n_kv_heads, head_dim, pages_sms());
}

extern "C" mk_status mk_attention_tree(const mk_pages *p, int layer, const void *q, long long q_stride, int n, int T,
                                       int n_heads, const int32_t *seqs, const int32_t *n_new, const uint32_t *mask,
                                       void *out, long long out_stride, void *scratch, size_t scratch_bytes,
                                       void *stream) {
    const char *who = "attention_tree";
    const mk_status st = pages_check(p, layer < 0 ? 1 << 30 : layer, who);
    if (st != MK_OK) return st;
    if (n < 0 || n > kPagesMaxSeqs || T < 1 || n_heads < 1 || n_heads % p->n_kv_heads ||
        (long long)T * (n_heads / p->n_kv_heads) > (1 << 24) || (long long)n * T > (1 << 30))
        return pages_refuse(who, "bad sizes: 0 <= n <= 1024, T >= 1, n_heads a multiple of n_kv_heads");
    if (n == 0) return MK_OK;
    if (!q || !out || !seqs || !scratch) return pages_refuse(who, "null pointer");
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)scratch) & 15)
        return pages_refuse(who, "q, out and scratch must be 16-byte aligned");
    const int d = p->head_dim;
    if (q_stride < (long long)n_heads * d || q_stride % 8 || out_stride < (long long)n_heads * d || out_stride % 8)
        return pages_refuse(who, "a stride is shorter than a row or not a multiple of 8");
    const int grid = pages_sms();
    if (scratch_bytes < tree_scratch(T, n_heads, p->n_kv_heads, d, grid))
        return pages_refuse(who, "scratch is smaller than mk_attention_tree_scratch_bytes");
    TreeArgs a{};
    a.p = *p;
    a.q = static_cast<const uint16_t *>(q);
    a.out = static_cast<uint16_t *>(out);
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.seqs = seqs;
    a.n_new = n_new;
    a.mask = mask;
    a.k = static_cast<const uint16_t *>(p->kv) + pages_offset(*p, 0, layer, 0);
    a.v = static_cast<const uint16_t *>(p->kv) + pages_offset(*p, 1, layer, 0);
    a.n = n;
    a.T = T;
    a.words = (T + 31) / 32;
    a.nq = n_heads;
    a.G = n_heads / p->n_kv_heads;
    a.rows_cap = tree_rows(T, a.G);
    a.part_o = static_cast<float *>(scratch);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)2 * grid * a.rows_cap * d);
    a.scale = (float)(1.4426950408889634 / std::sqrt((double)d));
    // a copy covers the part of a tile that lies in one page
    const int nt = tree_nt(d);
    int seg = nt;
    if (p->max_pages > 1)
        while (p->page_size % seg) seg /= 2;
    a.seg = seg;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)p->n_pages * p->n_kv_heads;
    const uint32_t blocks = seg == nt ? (uint32_t)(d / 64) : 1u;
    if (!tc_make_map_pages(&mk, a.k, rows, (uint32_t)p->page_size, (uint32_t)d, (uint32_t)seg, blocks) ||
        !tc_make_map_pages(&mv, a.v, rows, (uint32_t)p->page_size, (uint32_t)d, (uint32_t)seg, blocks)) {
        pages_refuse(who, "the driver refused the tensor map");
        return MK_ERR_CUDA;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = p->dtype == MK_BF16;
    cudaError_t e;
    switch (d) {
        case 64: e = bf16 ? launch_tree<64, true>(mk, mv, a, grid, s) : launch_tree<64, false>(mk, mv, a, grid, s); break;
        case 128: e = bf16 ? launch_tree<128, true>(mk, mv, a, grid, s) : launch_tree<128, false>(mk, mv, a, grid, s); break;
        default: e = bf16 ? launch_tree<256, true>(mk, mv, a, grid, s) : launch_tree<256, false>(mk, mv, a, grid, s);
    }
    return pages_launched(e, who);
}
