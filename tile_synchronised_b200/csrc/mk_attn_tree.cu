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
// the rows of one matrix (row r = t G + g), the tokens that fit 128 rows the M of
// an MMA, and the cache is read once for up to 256 rows (128 at d = 256).  Few
// rows are bound by that reading: 4 d bytes per position.  At 256 rows the 4 d
// flops per row and position take nearly as long on the tensor cores, the
// exponentials too, and the chain from one to the other twice that: 64 drafts at 3k to 4k
// positions keep HBM at 0.49 and the tensor pipe at 0.40 of their rates.  Per
// tile of NT positions:
//     S = Q K^T  (tensor memory, M = 128, N = NT), softmax in registers,
//     P (16 bit, tensor memory, over S) and O += P V (tensor memory, N = d).
// One thread owns one row of S, so the running maximum and sum need no
// exchange.  It holds 64 of the scores at a time: with more in registers
// the compiler spills, and with 227 KB of the SM given to the operands there is
// hardly an L1 to spill to (scores all in registers: 2.4 times slower).  O is
// rescaled only when the maximum grew by more than 2^8 since the last rescale:
// P and the sum then stay within 32-bit range of the older maximum and the
// quotient is the same.
//
// The softmax of a tile takes a group of four warps about as long as its K and
// V take to arrive, so (d <= 128) two groups work, each with an S and an O of
// its own.  Up to 128 rows they take alternate tiles of positions and their
// results are joined at the end of a run; above, they take 128 rows each of
// every tile.  At d = 256 tensor memory holds one O: one group, two S.
//
// Work: the units are (sequence, KV head, row tile, tile of positions), the
// tiles of one row tile consecutive (without a mask those up to its last
// token); each CTA (one per SM) takes an equal
// contiguous range, whatever the lengths, which are only known on the device.
// A CTA that covers all tiles of an item writes its rows of `out`; else it
// writes (o, max, sum) to scratch, at most two such records per CTA, and
// tree_combine_kernel joins them.
//
// Roles: the softmax warps; one warp loads Q and, into a ring, K and V tiles by
// TMA (a page's share of a tile per copy; the lanes look up 32 pages
// at a time, ahead); one lane issues the MMAs: with two jobs (tile, group) in
// flight, S of job j + 2 follows P V of job j.
//
// Measured (graph replays): single tokens of 16 sequences to 16k 102 us (5.9
// TB/s, 0.90 of the measured copy), 64 drafts of 16 sequences at 8k to 16k 216
// to 235 us (exponentials and MMAs 2048 cycles each per tile of 256 rows, the
// chain through both some 4000), 8 trees of 27 28 to 30 us, d = 256 trees 20 us,
// chunks of 500 tokens 31 to 35 us, one small tree 12 us: of the last four
// some 6 us pass before the first S and some 8 after the last P V.  A chunk of
// 4096 tokens behind 4096 at d = 128, 32 heads over 8: 520 us, 793 TFLOP/s, 0.57
// of the rate that a matrix product keeps up; at d = 64 434 us, 476 TFLOP/s.
//
// P is rounded to the cache's 16-bit type (2^-8 relative at most in bf16, each
// element on its own): both operands of an MMA have one type, and P in two parts
// would double the MMAs and the stores of P V.  Against 64 bits results are off by
// 2.3 parts in 1000 with it in bf16, 1.7 with P in 32 bits (the rounding of the
// result itself).  S, the maximum, the sum, O and the records are 32 bits.
#include <cuda.h>
#include <math_constants.h>

#include <atomic>
#include <cmath>
#include <utility>

#include "mk_kernel.h"
#include "mk_pages.h"
#include "mk_tc.cuh"

namespace mk {

constexpr int kTreeM = 128;          // rows of an MMA
constexpr int kTreeMaxStages = 12;
constexpr int kTreeMaxCtas = 192;    // of the grid, and so records of an item

// Softmax groups and positions of a tile at head size d.
__host__ __device__ constexpr int tree_groups(int d) { return d == 256 ? 1 : 2; }
__host__ __device__ constexpr int tree_nt(int d) { return d == 256 ? 64 : 128; }
__host__ __device__ constexpr int tree_threads(int d) { return (4 * tree_groups(d) + 2) * 32; }

struct TreeArgs {
    mk_pages p;
    const uint16_t *q;
    uint16_t *out;
    long long q_stride, out_stride;  // 16-bit elements between tokens
    const int *seqs, *n_new;
    const uint32_t *mask;
    float4 *part_o;  // [2 x CTAs][d / 4][rows_cap]: rows side by side, as the threads that write them
    float2 *part_ml; // [2 x CTAs][rows_cap]: maximum (base 2, scaled), sum
    const uint16_t *k, *v;  // this layer's pages
    int n, T, words, nq, G, seg, stages, q_tiles, rows_cap;
    int toks;        // new tokens of a row tile: 128 / G
    float scale;     // log2(e) / sqrt(d)
    int drop_q;      // tests of the time limit: the first run's Q is never loaded
    uint64_t wait_ns;  // time limit of a wait
};

// A listed sequence.
struct TreeEntry {
    int seq, len, fresh;
};

// A run of tiles of one item that one CTA works through, and where the walk
// over the CTA's range of units is (unit `at` of the item, `left` units to
// go); each warp has its own.
struct TreeRun {
    int i, g, rt, rts, t0, t1, tiles, slot, more, count, at;
    TreeEntry e;
    long long left;
};

// Shared memory behind the operand tiles.
struct TreeShared {
    uint64_t full[kTreeMaxStages], empty[kTreeMaxStages];
    uint64_t s_full[2], p_full[2], pv_done[2], q_full, q_empty, mma_end;
    TreeRun first, run[10];  // where the walk begins; of each warp
    float2 ml[2][kTreeM];    // the groups' maxima (scaled) and sums at the end of a run
    uint32_t tmem;
    int abort, bad_v;
    int bad_page[4];         // [r % 4] = r + 1: a page of the CTA's run r is missing
};

// Row tiles of entry e, and the tiles of positions that row tile rt needs:
// those up to its last token without a mask, else all.
template <int D>
__device__ __forceinline__ int tree_rts(const TreeArgs &a, const TreeEntry &e) {
    const int item = tree_groups(D) * a.toks;  // new tokens of an item
    return (e.fresh + item - 1) / item;
}
template <int D>
__device__ __forceinline__ int tree_tiles(const TreeArgs &a, const TreeEntry &e, int rt) {
    const int last = a.mask ? e.fresh : min(e.fresh, (rt + 1) * tree_groups(D) * a.toks);
    return (e.len + last + tree_nt(D) - 1) / tree_nt(D);
}
// Tiles of row tiles 0 .. rt - 1, rt <= rts.  Without a mask a sum of
// floor((x i + b) / m), taken with the steps of Euclid's algorithm on (x, m).
template <int D>
__device__ __forceinline__ long long tree_before(const TreeArgs &a, const TreeEntry &e, int rt, int rts) {
    if (a.mask || rts <= 1) return (long long)rt * tree_tiles<D>(a, e, 0);
    long long sum = rt == rts ? tree_tiles<D>(a, e, rts - 1) : 0;
    uint32_t n = rt == rts ? rts - 1 : rt, m = tree_nt(D), x = tree_groups(D) * a.toks, b = e.len + x + m - 1;
    while (n) {
        sum += (long long)n * (n - 1) / 2 * (x / m) + (long long)n * (b / m);
        x %= m;
        b %= m;
        const uint32_t y = x * n + b;
        n = y / m;
        b = y % m;
        const uint32_t was = m;
        m = x;
        x = was;
    }
    return sum;
}

// An item counts kTreeStart units more than it has tiles, in front of them: a
// run's Q, its first S and its epilogue take as long as some two tiles, so a
// CTA that goes through several short items gets fewer tiles.
constexpr int kTreeStart = 2;
template <int D>
__device__ __forceinline__ long long tree_start(const TreeArgs &a, const TreeEntry &e, int rt, int rts) {
    return tree_before<D>(a, e, rt, rts) + (long long)kTreeStart * rt;
}
// The units of entry e.
template <int D>
__device__ __forceinline__ long long tree_units(const TreeArgs &a, const TreeEntry &e) {
    const int rts = tree_rts<D>(a, e);
    return e.fresh ? a.p.n_kv_heads * tree_start<D>(a, e, rts, rts) : 0;
}

// n / d, mostly of small numbers (a 64-bit division takes hundreds of cycles).
__device__ __forceinline__ long long small_div(long long n, long long d) {
    return (n | d) >> 32 ? n / d : (long long)((uint32_t)n / (uint32_t)d);
}

// The warp's next run, false at the end of the CTA's range.
template <int D>
__device__ __forceinline__ bool tree_next(const TreeArgs &a, TreeRun &r, const TreeEntry *ent) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        r.more = 0;
        while (r.left > 0) {
            if (r.at == r.tiles + kTreeStart) {  // the next item
                r.at = 0;
                if (++r.rt == r.rts) {
                    r.rt = 0;
                    if (++r.g == a.p.n_kv_heads) {
                        r.g = 0;
                        do
                            r.e = ent[++r.i];
                        while (r.e.fresh == 0);
                        r.rts = tree_rts<D>(a, r.e);
                    }
                }
                r.tiles = tree_tiles<D>(a, r.e, r.rt);
            }
            const int to = (int)min((long long)(r.tiles + kTreeStart), r.at + r.left);
            r.t0 = max(r.at - kTreeStart, 0);
            r.t1 = max(to - kTreeStart, 0);
            r.left -= to - r.at;
            r.at = to;
            if (r.t0 < r.t1) {
                r.slot = 2 * blockIdx.x + (r.count ? 1 : 0);
                r.count = 1;
                r.more = 1;
                break;
            }
        }
    }
    __syncwarp();
    return r.more;
}

// The CTAs that share U units out of `most`: one unit each is enough (with at
// least 2, 4 or 8 a tree behind 1k positions took 1.2, 4 and 8 us more).
__device__ __forceinline__ int tree_ctas(long long U, int most) { return U < most ? (int)(U > 0 ? U : 1) : most; }
__device__ __forceinline__ long long tree_first(long long U, int ctas, int c) { return small_div(U * c, ctas); }

// The words of new token t's mask row: bit u of word k is new token 32 k + u
// (k < 0: committed positions, all visible).
__device__ __forceinline__ uint32_t tree_word(const TreeArgs &a, const uint32_t *mask_row, int t, int fresh, int k) {
    const int u0 = k * 32;
    uint32_t w;
    if (a.mask)  // loads without a branch, so that several can be in flight
        w = mask_row[min(max(k, 0), a.words - 1)];
    else
        w = t - u0 >= 31 ? 0xFFFFFFFFu : (2u << (max(t - u0, -1) & 31)) - 1u;
    if (!a.mask && t < u0) w = 0u;
    const uint32_t real = fresh - u0 >= 32 ? 0xFFFFFFFFu : fresh > u0 ? (1u << (fresh - u0)) - 1u : 0u;
    return k < 0 ? 0xFFFFFFFFu : w & real;
}
// Visibility of positions pos .. pos + 32 N - 1 to it.
template <int N>
__device__ __forceinline__ void tree_bits(const TreeArgs &a, int i, int t, const TreeEntry &e, int pos, uint32_t *bits) {
    const int u = pos - e.len, k = u >> 5, sh = u & 31;
    const uint32_t *row = a.mask + ((size_t)i * a.T + t) * a.words;
    uint32_t w[N + 1];
#pragma unroll
    for (int x = 0; x <= N; ++x) w[x] = tree_word(a, row, t, e.fresh, k + x);
#pragma unroll
    for (int x = 0; x < N; ++x) bits[x] = __funnelshift_r(w[x], w[x + 1], sh);
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
// Waits for this thread's tensor-memory loads.  The loaded registers are
// operands, so that no use of them can be moved above the wait.
__device__ __forceinline__ void tmem_wait_ld(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
// 16 columns (no wait), and the wait for them.
__device__ __forceinline__ void tmem_ld16n(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld16(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

// Packed pairs of 32-bit floats.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Is the phase `parity` of an mbarrier complete?  (Does not wait.)
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// The barrier of the softmax threads.
template <int NG>
__device__ __forceinline__ void softmax_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(NG * 128) : "memory");
}

// What a thread writes at the end of a run: columns c0 .. c1 - 1 of its row.
struct TreeOut {
    uint32_t o_mine, o_other;  // tensor memory of the group's O and of the other's
    float f0, f1;              // their weights
    float inv;                 // 1 / sum for the result, 1 for a record
    float m2, bias;
    int c0, c1, g, t;
    bool join, mine, other, live, whole, ok;  // join: both groups' O go into a row
    float4 *rec;
    uint16_t *to;
};

// With ADD also the share of new tokens whose V holds an infinity or NaN.  In
// the MMA those rows of V are zeros, since 0 x inf in a row that does not see
// the token would be NaN; here every row that does see one adds p V itself.
template <int D, bool BF16, bool ADD>
__device__ __forceinline__ void tree_write(const TreeArgs &a, const TreeRun &r, const TreeOut w) {
#pragma unroll 1
    for (int c = w.c0; c < w.c1; c += 32) {
        float o[32];
        tmem_ld32(w.o_mine + c, o);
        if (w.join) {
            float x[32];
            tmem_ld32(w.o_other + c, x);
            tmem_wait_ld(o);
            tmem_wait_ld(x);
#pragma unroll
            for (int k = 0; k < 32; ++k) {  // an O that no tile went into is not used
                o[k] = w.mine ? o[k] * w.f0 : 0.f;
                o[k] = w.other ? fmaf(x[k], w.f1, o[k]) : o[k];
            }
        } else {
            tmem_wait_ld(o);
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = w.ok ? o[k] : CUDART_NAN_F;
        if (w.live) {
            if constexpr (ADD) {
                const uint16_t *q = a.q + ((size_t)r.i * a.T + w.t) * a.q_stride + (size_t)(r.g * a.G + w.g) * D;
                const int to = min(r.e.len + r.e.fresh, r.t1 * tree_nt(D));
                for (int pos = max(r.e.len, r.t0 * tree_nt(D)); pos < to; ++pos) {
                    uint32_t see;
                    tree_bits<1>(a, r.i, w.t, r.e, pos, &see);
                    if (!(see & 1u)) continue;
                    const int page = a.p.table[(size_t)r.e.seq * a.p.max_pages + pos / a.p.page_size];
                    if (page < 0 || page >= a.p.n_pages) continue;
                    const size_t at = (((size_t)page * a.p.n_kv_heads + r.g) * a.p.page_size + pos % a.p.page_size) * D;
                    bool bad = false;
                    for (int k = 0; k < D; k += 8)
                        bad = bad || any_nonfinite<BF16>(*reinterpret_cast<const uint4 *>(a.v + at + k));
                    if (!bad) continue;
                    float dot = 0.f;
                    for (int k = 0; k < D; ++k) dot = fmaf(from16<BF16>(q[k]), from16<BF16>(a.k[at + k]), dot);
                    const float p = ex2(fmaf(dot, a.scale, w.bias - (w.m2 == -CUDART_INF_F ? 0.f : w.m2)));
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = fmaf(p, from16<BF16>(a.v[at + c + k]), o[k]);
                }
            }
            if (w.whole) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint4 v;
                    v.x = pack16<BF16>(o[k] * w.inv, o[k + 1] * w.inv);
                    v.y = pack16<BF16>(o[k + 2] * w.inv, o[k + 3] * w.inv);
                    v.z = pack16<BF16>(o[k + 4] * w.inv, o[k + 5] * w.inv);
                    v.w = pack16<BF16>(o[k + 6] * w.inv, o[k + 7] * w.inv);
                    *reinterpret_cast<uint4 *>(w.to + c + k) = v;
                }
            } else {
                float4 *rec = w.rec + (size_t)(c / 4) * a.rows_cap;
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                    rec[(size_t)(k / 4) * a.rows_cap] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            }
        }
        __syncwarp();
    }
}
template <int D, bool BF16>
__device__ __noinline__ void tree_write_add(const TreeArgs &a, const TreeRun &r, const TreeOut w) {
    tree_write<D, BF16, true>(a, r, w);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(tree_threads(D), 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TreeArgs a) {
    constexpr int NT = tree_nt(D), NH = D / 64;  // positions of a tile, 64-column blocks of a row
    constexpr int NG = tree_groups(D), kLoader = 4 * NG, kIssuer = kLoader + 1;
    constexpr uint32_t kQBytes = kTreeM * D * 2, kStage = NT * D * 2;
    constexpr uint32_t kO = 256;                  // tensor-memory column of the first O; S at 0 and 128
    constexpr float kBias = BF16 ? 0.f : 7.f;     // fp16 P: 2^7 above the maximum's 1, so that small
                                                  // values keep clear of its subnormals (at most 2^15)
    constexpr float kGrow = 8.f;                  // rescale O when the maximum grew by more (base 2)
    extern __shared__ __align__(1024) uint8_t tree_smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tree_smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_q = smem, *ring = smem + a.q_tiles * kQBytes;
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
            mbar_init(&sh.pv_done[s], 1);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.mma_end, 1);
        sh.abort = 0;
        sh.bad_v = 0;
        for (int s = 0; s < 4; ++s) sh.bad_page[s] = 0;
        fence_barrier_init();
    }
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kLoader && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v) : "memory");
    // the listed sequences and the units before each
    for (int i = tid; i < a.n; i += blockDim.x) {
        const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, i, a.T);
        if (e.err && blockIdx.x == 0) pages_fail(a.p.state, e.err, i, e.seq);
        ent[i] = TreeEntry{e.seq, e.len, e.fresh};
        pref[i + 1] = tree_units<D>(a, ent[i]);
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
        __syncwarp();
        if (lane == 0) {  // where this CTA begins
            TreeRun &r = sh.first;
            const long long U = carry;
            const int ctas = tree_ctas(U, gridDim.x);
            const bool mine = (int)blockIdx.x < ctas;
            const long long u = mine ? tree_first(U, ctas, blockIdx.x) : 0;
            r.left = mine ? tree_first(U, ctas, blockIdx.x + 1) - u : 0;
            r.count = 0;
            pref[0] = 0;
            if (r.left) {
                int lo = 0, hi = a.n;  // the last entry that starts at or before u
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (pref[mid] <= u)
                        lo = mid;
                    else
                        hi = mid;
                }
                r.i = lo;
                r.e = ent[lo];
                r.rts = tree_rts<D>(a, r.e);
                const long long head = tree_start<D>(a, r.e, r.rts, r.rts), local = u - pref[lo];
                r.g = (int)small_div(local, head);
                const long long rest = local - r.g * head;
                lo = 0, hi = r.rts;  // the last row tile that starts at or before it
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (tree_start<D>(a, r.e, mid, r.rts) <= rest)
                        lo = mid;
                    else
                        hi = mid;
                }
                r.rt = lo;
                r.at = (int)(rest - tree_start<D>(a, r.e, lo, r.rts));
                r.tiles = tree_tiles<D>(a, r.e, lo);
            }
        }
    }
    __syncthreads();
    pdl_launch_dependents();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&sh.tmem);
    TreeRun &run = sh.run[warp];
    if (lane == 0) run = sh.first;
    int issued = 0, q_issued = 0;  // the loader's ring loads and runs whose Q it loaded
    // Jobs of a run, in order: with two row tiles (both groups on every tile)
    // job j is group j & 1 of tile j / 2, else S buffer j & 1 of tile j.
    auto two_rows = [&]() { return NG == 2 && run.e.fresh - run.rt * 2 * a.toks > a.toks; };

    if (warp == kLoader) {
        // ------------------------------------------------------------ loader
        const int seg = a.seg, ns = NT / seg, per = 32 / ns;
        const int nh = ns > 1 ? NH : 1;  // a whole tile's box covers every 64-column block
        const int my = lane / nh, blk = lane - my * nh;
        const int nkv = a.p.n_kv_heads, ps = a.p.page_size, off_step = NT % ps, seg_log = 31 - __clz(seg);
        const uint32_t seg_bytes = (uint32_t)seg * D * 2, off_smem = (uint32_t)(blk * NT + my * seg) * 128u;
        const uint32_t q_bytes = (uint32_t)(a.toks * a.G) * D * 2;
        int slot = 0, seg_no = 0;
        uint32_t phase = 1;  // of empty[slot]: the first round waits for nothing
        bool ok = true;
        while (ok && tree_next<D>(a, run, ent)) {
            const int *row = a.p.table + (size_t)run.e.seq * a.p.max_pages;
            const int end = run.e.len + run.e.fresh, t0 = run.t0, t1 = run.t1, g = run.g;
            const bool mine = lane < ns * nh;
            // lane x holds the page of part x % ns of tile tb + x / ns
            auto look = [&](int tb) {
                const int t = tb + lane / ns, pos = t * NT + lane % ns * seg;
                return t < t1 && pos < end ? row[pos / ps] : -1;
            };
            // Q: 64 columns x G heads x tokens are the swizzled rows of an MMA operand
            auto load_q = [&]() {
                if (seg_no && !tc_wait(&sh.q_empty, (seg_no - 1) & 1u, abort, a.wait_ns)) return false;
                if (lane == 0) {
                    const int tiles = two_rows() ? 2 : 1, tok = run.i * a.T + run.rt * NG * a.toks;
                    mbar_arrive_expect_tx(&sh.q_full, tiles * q_bytes);
                    for (int x = 0; x < tiles; ++x)
                        for (int c = 0; c < NH; ++c)
                            tma_load_4d(s_q + x * kQBytes + c * kTreeM * 128, &map_q, 0, c, g * a.G, tok + x * a.toks,
                                        &sh.q_full);
                }
                ++q_issued;
                return true;
            };
            int tb = t0, pages = look(tb), next = look(tb + per);
            int off = (t0 * NT + my * seg) % ps;  // of this lane's part in its page
            if (seg_no == 0 && !a.drop_q) ok = load_q();
            for (int t = t0; ok && t < t1; ++t) {
                if (t - tb == per) {
                    tb = t;
                    pages = next;
                    next = look(tb + per);
                }
                int page = __shfl_sync(0xFFFFFFFFu, pages, ((t - tb) * ns + my) & 31);
                const int pos = t * NT + my * seg;
                const bool go = mine && pos < end;
                if (go && (page < 0 || page >= a.p.n_pages)) {
                    pages_fail(a.p.state, kPgPosition, run.i, pos);
                    // the run's rows become NaN.  By the softmax's epilogue of a run the loader is three runs
                    // ahead at most: the third one's Q waits for S of the second, and that for P of the first
                    *reinterpret_cast<volatile int *>(&sh.bad_page[seg_no & 3]) = seg_no + 1;
                    page = -1;  // out of the tensor: zeros
                }
                __syncwarp();
                const int head = page < 0 ? -1 : page * nkv + g, left = (end - t * NT + seg - 1) >> seg_log;
                const uint32_t bytes = (uint32_t)(left < ns ? left : ns) * seg_bytes;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(0xFFFFFFFFu, tc_wait(&sh.empty[slot], phase, abort, a.wait_ns));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], bytes);
                    __syncwarp();
                    if (go)
                        tma_load_4d(ring + (size_t)slot * kStage + off_smem, kv ? &map_v : &map_k, 0, off, blk, head,
                                    &sh.full[slot]);
                    ++issued;
                    if (++slot == S) slot = 0, phase ^= 1u;
                }
                off += off_step;
                if (off >= ps) off -= ps;
                // the last Q is free once its last S is done; this run's first tile does not wait for that
                if (t == t0 && seg_no) ok = ok && __all_sync(0xFFFFFFFFu, load_q());
            }
            ++seg_no;
        }
    } else if (warp == kIssuer) {
        // -------------------------------------------------------- MMA issuer
        constexpr uint32_t id_qk = tree_idesc<BF16>(NT, false), id_pv = tree_idesc<BF16>(D, true);
        // descriptors of the first 16 columns (positions); a step of 16 adds
        // 32 bytes along a row (16 rows), in units of 16 bytes
        const uint64_t d_q = smem_desc_sw128(s_q, 16, 1024), d_k = smem_desc_sw128(ring, 16, 1024),
                       d_v = smem_desc_sw128(ring, NT * 128, 1024);
        // ring slots of the next K (even loads) and the next V (odd ones)
        int k_slot = 0, v_slot = 1, seg_no = 0;
        uint32_t k_phase = 0, v_phase = 0;
        uint32_t used[2] = {0, 0};  // jobs of each S buffer whose P has been taken
        bool ok = true;
        auto step = [&](int &slot, uint32_t &phase) {
            slot += 2;
            if (slot >= S) slot -= S, phase ^= 1u;
        };
        // The whole warp runs the loop (its values stay uniform, as the MMA's
        // operands have to be); one elected lane issues.
        while (ok && tree_next<D>(a, run, ent)) {
            const int nt = __shfl_sync(0xFFFFFFFFu, run.t1 - run.t0, 0);
            const bool two = __shfl_sync(0xFFFFFFFFu, (int)two_rows(), 0);
            const int jobs = two ? 2 * nt : nt;
            auto qk_issue = [&](int j) {  // by the elected lane, once K is there
                const int b = j & 1;
                const uint64_t dk = d_k + (uint32_t)k_slot * (kStage >> 4), dq = d_q + (two && b ? kQBytes >> 4 : 0);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma(tmem + (uint32_t)b * 128, dq + (ks / 4) * (kTreeM * 8) + (ks % 4) * 2,
                           dk + (ks / 4) * (NT * 8) + (ks % 4) * 2, id_qk, ks > 0);
                tc_commit(&sh.s_full[b]);
                if (!two || b) tc_commit(&sh.empty[k_slot]);
                if (j == jobs - 1) tc_commit(&sh.q_empty);
            };
            auto qk = [&](int j) {
                if (!__all_sync(0xFFFFFFFFu, tc_wait(&sh.full[k_slot], k_phase, abort, a.wait_ns))) return false;
                tc_fence_after();
                if (elect_one()) qk_issue(j);
                __syncwarp();
                if (!two || (j & 1)) step(k_slot, k_phase);
                return true;
            };
            ok = __all_sync(0xFFFFFFFFu, tc_wait(&sh.q_full, seg_no & 1u, abort, a.wait_ns));
            tc_fence_after();
            ok = ok && qk(0) && (jobs < 2 || qk(1));
#pragma unroll 1
            for (int j = 0; ok && j < jobs; ++j) {
                const int b = j & 1;
                // With K of job j + 2 there already, its S goes out right behind P V
                const bool k_there = __all_sync(0xFFFFFFFFu, j + 2 < jobs && mbar_test_wait(&sh.full[k_slot], k_phase));
                ok = tc_wait(&sh.full[v_slot], v_phase, abort, a.wait_ns) &&
                     tc_wait(&sh.p_full[b], used[b] & 1u, abort, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                ++used[b];
                tc_fence_after();
                const uint64_t dv = d_v + (uint32_t)v_slot * (kStage >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < NT / 16; ++ks)
                        tc_mma_ta(tmem + kO + (NG == 2 ? (uint32_t)b * D : 0u), tmem + (uint32_t)b * 128 + ks * 8,
                                  dv + ks * 128, id_pv, j >= NG || ks > 0);
                    // the softmax waits for P V where it changes O (one group), and at the end of the run
                    if (NG == 1 || j + 2 >= jobs) tc_commit(&sh.pv_done[NG == 2 ? b : 0]);
                    if (!two || b) tc_commit(&sh.empty[v_slot]);
                    if (k_there) qk_issue(j + 2);
                }
                __syncwarp();
                if (!two || b) step(v_slot, v_phase);
                if (k_there) {
                    if (!two || b) step(k_slot, k_phase);
                } else if (j + 2 < jobs) {
                    ok = qk(j + 2);
                }
            }
            ++seg_no;
        }
    } else {
        // ----------------------------------------------------------- softmax
        const int grp = warp >> 2, gw = warp & 3;  // gw: its tensor-memory lanes
        const int gt = gw * 32 + lane;             // row within the group's 128
        const uint32_t lanes = tmem + ((uint32_t)(gw * 32) << 16);
        int load = 0, no = 0;  // ring loads of earlier runs, and their number
        uint32_t seen[2] = {0, 0}, done = 0;  // S of each buffer taken, P V waited for
        bool ok = true;
        const int my_tok = gt / a.G, my_g = gt - my_tok * a.G;
        while (tree_next<D>(a, run, ent)) {
            const int nt = run.t1 - run.t0, t0 = run.t0, entry = run.i;
            const TreeEntry e = run.e;
            const bool two = two_rows(), join = NG == 2 && !two;
            const int tok0 = run.rt * NG * a.toks + (two ? grp * a.toks : 0);  // first token of this row tile
            const int rows = min(a.toks, e.fresh - tok0) * a.G, t = tok0 + my_tok;
            const bool live = gt < rows, warp_live = gw * 32 < rows;
            float m = -CUDART_INF_F, l = 0.f;  // the maximum that P and the sum refer to (of S unscaled)
            const int step = join ? 2 : 1, first = join ? grp : 0;
            for (int i = first; i < nt; i += step) {
                const int b = NG == 2 ? grp : i & 1, p0 = (t0 + i) * NT;
                const uint32_t sc = lanes + (uint32_t)b * 128;
                const bool tail = p0 + NT > e.len;  // new tokens, or nothing, in this tile
                uint32_t bits[NT / 32];
                if (tail) {
                    tree_bits<NT / 32>(a, entry, live ? t : 0, e, p0, bits);
#pragma unroll
                    for (int c = 0; c < NT / 32; ++c) bits[c] = live ? bits[c] : 0u;
                }
                ok = ok && tc_wait(&sh.s_full[b], seen[b] & 1u, abort, a.wait_ns);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                ++seen[b];
                tc_fence_after();
                // Two passes over S, for its maximum and for P, 64 scores at a
                // time.  Rolled loops: unrolled, the compiler's schedule
                // overflows the registers, and there is hardly an L1 to spill to.
                float lo[32], hi[32], top = -CUDART_INF_F;
                auto hide = [&](float *v, uint32_t w) {
                    if (tail && __any_sync(0xFFFFFFFFu, w != 0xFFFFFFFFu)) {
                        asm volatile("" : "+r"(w));  // else the bit tests are kept from pass to pass
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = (w >> k) & 1u ? v[k] : -CUDART_INF_F;
                    }
                };
                auto read = [&](int c) {
                    tmem_ld32(sc + c, lo);
                    tmem_ld32(sc + c + 32, hi);
                    tmem_wait_ld(lo);
                    tmem_wait_ld(hi);
                    hide(lo, c ? bits[NT / 32 - 2] : bits[0]);
                    hide(hi, c ? bits[NT / 32 - 1] : bits[1]);
                };
                auto max32 = [&](const float *v) {
                    float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                    for (int k = 4; k < 32; k += 2) x[(k / 2) & 3] = max3(x[(k / 2) & 3], v[k], v[k + 1]);
                    return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                };
                if (warp_live) {
#pragma unroll 1
                    for (int c = NT - 64; c >= 0; c -= 64) {
                        read(c);
                        top = max3(top, max32(lo), max32(hi));
                    }
                }
                if (NG == 1 && i > 0) {  // P V of the last tile (two groups: S came after it)
                    ok = tc_wait(&sh.pv_done[0], done & 1u, abort, a.wait_ns);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    ++done;
                    tc_fence_after();
                }
                if (warp_live) {
                    const bool grew = live && (top - m) * a.scale > kGrow;  // also from -inf
                    if (__any_sync(0xFFFFFFFFu, grew)) {
                        const float f = grew ? ex2((m - top) * a.scale) : 1.f;
                        if (grew) m = top;
                        l *= f;
                        if (i > first) {
                            const uint32_t oc = lanes + kO + (uint32_t)(grp * D);
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float o[16];
                                tmem_ld16n(oc + c, o);
                                tmem_wait_ld16(o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] *= f;
                                tmem_st16(oc + c, reinterpret_cast<const uint32_t *>(o));
                            }
                        }
                    }
                    const float ms = kBias - (m == -CUDART_INF_F ? 0.f : m) * a.scale;
                    const uint64_t scale2 = pair(a.scale, a.scale), ms2 = pair(ms, ms);
                    uint64_t sum0 = 0, sum1 = 0;
                    auto exps = [&](const float *v, uint32_t to) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float e0, e1;
                            unpair(fma2(pair(v[k], v[k + 1]), scale2, ms2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            if (k & 2)
                                sum1 = add2(sum1, pair(e0, e1));
                            else
                                sum0 = add2(sum0, pair(e0, e1));
                            pk[k / 2] = pack16<BF16>(e0, e1);
                        }
                        tmem_st16(to, pk);
                    };
                    // P goes over S from the front: over scores in registers, or used
                    // up; the first pass left the first 64 in registers
#pragma unroll 1
                    for (int c = 0; c < NT; c += 64) {
                        if (c) read(c);
                        exps(lo, sc + c / 2);
                        exps(hi, sc + c / 2 + 16);
                    }
                    float x, y;
                    unpair(add2(sum0, sum1), x, y);
                    l += x + y;
                    tmem_wait_st();
                }
                if (tail && (!two || grp == 0)) {
                    // V rows of new tokens with an infinity or NaN, and rows
                    // behind the last token, become zeros; with two row tiles
                    // by the first group, whose P V comes first
                    const int ld = load + 2 * i + 1, st = ld % S;
                    ok = tc_wait(&sh.full[st], (ld / S) & 1u, abort, a.wait_ns);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const int pos = p0 + gt;
                    if (gt < NT && pos >= e.len) {
                        uint8_t *vr = ring + (size_t)st * kStage + gt * 128;
                        auto chunk = [&](int c) {  // 16-byte chunk c of the row
                            return reinterpret_cast<uint4 *>(vr + (c / 8) * NT * 128 + (((c & 7) ^ (gt & 7)) << 4));
                        };
                        bool clear = pos >= e.len + e.fresh;
                        if (!clear) {
#pragma unroll 8
                            for (int c = 0; c < D / 8; ++c) clear |= any_nonfinite<BF16>(*chunk(c));
                            if (clear) *reinterpret_cast<volatile int *>(&sh.bad_v) = 1;
                        }
                        if (clear)
                            for (int c = 0; c < D / 8; ++c) *chunk(c) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[b]);
            }
            // ------------------------------------------------------ epilogue
            TreeOut w;
            w.mine = first < nt;  // this group had a tile (group 0 always has)
            if (ok && w.mine) {
                ok = __all_sync(0xFFFFFFFFu, tc_wait(&sh.pv_done[grp], done & 1u, abort, a.wait_ns));
                ++done;
            }
            load += 2 * nt;
            const bool fine = ok && *reinterpret_cast<volatile int *>(&sh.bad_page[no & 3]) != no + 1;
            ++no;
            const float nan = CUDART_NAN_F;
            if (join) {
                sh.ml[grp][gt] = fine ? make_float2(m * a.scale, l) : make_float2(nan, nan);
                tc_fence_before();
                softmax_sync<NG>();
            }
            tc_fence_after();
            w.ok = fine;
            w.join = join;
            w.live = live;
            w.whole = run.t0 == 0 && run.t1 == run.tiles;
            w.m2 = m * a.scale;
            w.bias = kBias;
            w.f0 = 1.f;
            w.f1 = 0.f;
            bool other = false;
            if (join) {  // weights of the groups' results; each thread writes half of the row
                const float mx = sh.ml[grp ^ 1][gt].x, lx = sh.ml[grp ^ 1][gt].y;
                other = grp == 1 || nt > 1;
                const float top = fmaxf(w.m2, mx), tm = top == -CUDART_INF_F ? 0.f : top;
                w.f0 = ex2(w.m2 - tm);
                w.f1 = ex2(mx - tm);
                l = (w.mine ? l * w.f0 : 0.f) + (other ? lx * w.f1 : 0.f);
                w.m2 = top;
            }
            if (warp_live) {
                w.inv = w.whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
                w.g = my_g;
                w.t = t;
                w.o_mine = lanes + kO + (uint32_t)(grp * D);
                w.other = other;
                w.o_other = join ? lanes + kO + (uint32_t)((grp ^ 1) * D) : w.o_mine;
                w.c0 = join ? grp * (D / 2) : 0;
                w.c1 = join ? w.c0 + D / 2 : D;
                w.rec = a.part_o + (size_t)run.slot * (D / 4) * a.rows_cap + (two ? grp * kTreeM : 0) + gt;
                w.to = a.out + ((size_t)run.i * a.T + t) * a.out_stride + (size_t)(run.g * a.G + my_g) * D;
                if (__any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile int *>(&sh.bad_v) && run.t1 * NT > run.e.len))
                    tree_write_add<D, BF16>(a, run, w);
                else
                    tree_write<D, BF16, false>(a, run, w);
                if (live && !w.whole && (!join || grp == 0))
                    a.part_ml[(size_t)run.slot * a.rows_cap + (two ? grp * kTreeM : 0) + gt] =
                        fine ? make_float2(w.m2, l) : make_float2(nan, nan);
            }
            tc_fence_before();
            if (join) softmax_sync<NG>();  // O and the maxima have been read
        }
    }
    // After a wait ran out some copies and MMAs may be in flight.  Which role's
    // it was, and whether any, is known once all of them have ended: then the
    // last copy of every stage and the last MMA are waited for, before the
    // shared and the tensor memory are freed.
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        if (warp == kLoader && lane == 0) {
            for (int x = issued > S ? issued - S : 0; x < issued; ++x)
                tc_drain(&sh.full[x % S], (uint32_t)(x / S) & 1u, kTcTimeoutNs);
            if (q_issued) tc_drain(&sh.q_full, (uint32_t)(q_issued - 1) & 1u, kTcTimeoutNs);
            pages_fail(a.p.state, kPgTimeout, 0, blockIdx.x);
        }
        __syncwarp();
        if (warp == kIssuer) {
            if (elect_one()) tc_commit(&sh.mma_end);
            __syncwarp();
            tc_drain(&sh.mma_end, 0u, kTcTimeoutNs);
        }
        __syncthreads();
    }
    if (warp == kIssuer) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// Joins the records of every item that more than one CTA worked on: CTA
// (x, i, g) 8 R rows and up to 128 columns of an item of KV head g of entry i,
// a thread 4 columns of R rows (8 rows of a column block are side by side in a
// record).  The time is that of one round of loads after another, so the first
// 16 of a thread go out before the weights are known.  R = 4 where that leaves
// CTAs enough: a CTA takes some 3 us whatever it finds to join.
template <int D>
struct Combine {
    static constexpr int kCols = D < 128 ? D : 128, kThreads = 2 * kCols, kWarps = kThreads / 32;
};

template <int D, bool BF16, int R>
__global__ void __launch_bounds__(Combine<D>::kThreads) tree_combine_kernel(const __grid_constant__ TreeArgs a, int grid) {
    constexpr int NG = tree_groups(D), kCombineRows = 8 * R, kCols = Combine<D>::kCols;
    constexpr int kCombineThreads = Combine<D>::kThreads, kWarps = Combine<D>::kWarps;
    constexpr int kBatch = 16 / R;  // records whose loads a thread has in flight
    __shared__ long long s_red[2][kWarps];
    __shared__ float s_w[kTreeMaxCtas][kCombineRows];  // weight of each record's row
    __shared__ float s_inv[kCombineRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.y, g = blockIdx.z / (D / kCols), c4 = blockIdx.z % (D / kCols) * (kCols / 4) + warp * 4 + (lane >> 3);
    const int blocks = (a.rows_cap + kCombineRows - 1) / kCombineRows;
    const int rt = blockIdx.x / blocks, r0 = (blockIdx.x - rt * blocks) * kCombineRows;
    // units before entry i, and of all entries
    long long before = 0, total = 0;
    for (int k = threadIdx.x; k < a.n; k += kCombineThreads) {
        const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, k, a.T);
        const long long u = tree_units<D>(a, TreeEntry{e.seq, e.len, e.fresh});
        total += u;
        if (k < i) before += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
        total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    }
    if (lane == 0) {
        s_red[0][warp] = before;
        s_red[1][warp] = total;
    }
    const PagesEntry e = pages_entry(a.p, a.seqs, a.n_new, i, a.T);
    __syncthreads();
    before = total = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        before += s_red[0][k];
        total += s_red[1][k];
    }
    const TreeEntry te{e.seq, e.len, e.fresh};
    const int rts = tree_rts<D>(a, te);
    int c0 = 0, c1 = 0, slot0 = 0;
    if (rt < rts) {
        const long long start = before + g * tree_start<D>(a, te, rts, rts) + tree_start<D>(a, te, rt, rts);
        const long long u0 = start + kTreeStart, u1 = u0 + tree_tiles<D>(a, te, rt);
        const int ctas = tree_ctas(total, grid);
        // the CTA of unit u is the last one whose first unit is at most u
        c0 = (int)(((u0 + 1) * ctas - 1) / total);
        c1 = (int)((u1 * ctas - 1) / total);
        // of these CTAs only the first one's record can be its second
        slot0 = 2 * c0 + (tree_first(total, ctas, c0) < start ? 1 : 0);
    }
    const int count = c1 - c0 + 1;
    pdl_wait();              // the records are complete
    // none, or the item's only CTA wrote the result; or rows of no token
    const auto token = [&](int r) { return (rt * NG + r / kTreeM) * a.toks + (r & (kTreeM - 1)) / a.G; };
    const auto real = [&](int r) { return r < a.rows_cap && (r & (kTreeM - 1)) < a.toks * a.G && token(r) < e.fresh; };
    if (c0 == c1 || !real(r0)) return;
    auto slot = [&](int c) { return (size_t)(c == 0 ? slot0 : 2 * (c0 + c)); };
    const size_t pitch = (size_t)(D / 4) * a.rows_cap;
    const float4 *rec = a.part_o + (size_t)c4 * a.rows_cap + r0 + (lane & 7);
    float4 v[kBatch][R];
    bool live[R];
#pragma unroll
    for (int x = 0; x < R; ++x) live[x] = real(r0 + 8 * x + (lane & 7));
    auto load = [&](int first) {
#pragma unroll
        for (int c = 0; c < kBatch; ++c)
#pragma unroll
            for (int x = 0; x < R; ++x)
                if (first + c < count && live[x])
                    v[c][x] = rec[slot(first + c) * pitch + 8 * x];
    };
    load(0);
    {  // kL lanes a row: maximum, weights and sum
        constexpr int kL = kCombineThreads / kCombineRows;
        const int x = threadIdx.x / kL, c_first = threadIdx.x % kL;
        const bool mine = real(r0 + x);
        float M = -CUDART_INF_F, L = 0.f;
        for (int c = c_first; mine && c < count; c += kL) M = fmaxf(M, a.part_ml[slot(c) * a.rows_cap + r0 + x].x);
#pragma unroll
        for (int o = kL / 2; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
        if (M == -CUDART_INF_F) M = 0.f;
        for (int c = c_first; mine && c < count; c += kL) {
            const float2 ml = a.part_ml[slot(c) * a.rows_cap + r0 + x];
            const float f = ex2(ml.x - M);
            s_w[c][x] = f;
            L = fmaf(f, ml.y, L);
        }
#pragma unroll
        for (int o = kL / 2; o; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
        if (c_first == 0) s_inv[x] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();
    {
        float4 o[R];
#pragma unroll
        for (int x = 0; x < R; ++x) o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int first = 0; first < count; first += kBatch) {
            if (first) load(first);
#pragma unroll
            for (int c = 0; c < kBatch; ++c)
#pragma unroll
                for (int x = 0; x < R; ++x) {
                    if (first + c >= count || !live[x]) continue;
                    const float f = s_w[first + c][8 * x + (lane & 7)];
                    o[x].x = fmaf(f, v[c][x].x, o[x].x);
                    o[x].y = fmaf(f, v[c][x].y, o[x].y);
                    o[x].z = fmaf(f, v[c][x].z, o[x].z);
                    o[x].w = fmaf(f, v[c][x].w, o[x].w);
                }
        }
#pragma unroll
        for (int x = 0; x < R; ++x) {
            if (!live[x]) continue;
            const int r = r0 + 8 * x + (lane & 7), gt = r & (kTreeM - 1), t = token(r);
            const float inv = s_inv[8 * x + (lane & 7)];
            uint16_t *to = a.out + ((size_t)i * a.T + t) * a.out_stride + (size_t)(g * a.G + gt % a.G) * D;
            *reinterpret_cast<uint2 *>(to + c4 * 4) =
                make_uint2(pack16<BF16>(o[x].x * inv, o[x].y * inv), pack16<BF16>(o[x].z * inv, o[x].w * inv));
        }
    }
}

// ------------------------------------------------------------------ host side
// Rows of a record: those of all new tokens, or of two whole row tiles.
static int tree_rows_cap(int T, int G, int d) {
    const int toks = kTreeM / G;
    return T <= toks ? T * G : tree_groups(d) * kTreeM;
}

static int tree_grid() {
    const int sms = pages_sms();
    return sms < kTreeMaxCtas ? sms : kTreeMaxCtas;
}

// What mk_debug_attention_tree_wait set.
static std::atomic<unsigned long long> tree_wait_ns{kTcTimeoutNs};
static std::atomic<int> tree_drop_q{0};

static size_t tree_scratch(int T, int nq, int nkv, int d, int grid) {
    return (size_t)2 * grid * tree_rows_cap(T, nq / nkv, d) * (d + 2) * sizeof(float);
}

template <int D, bool BF16>
static cudaError_t launch_tree(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, TreeArgs &a,
                               int grid, cudaStream_t s) {
    constexpr int stage = tree_nt(D) * D * 2;
    a.q_tiles = tree_groups(D) == 2 && a.T > a.toks ? 2 : 1;
    const int fixed = 1024 + a.q_tiles * kTreeM * D * 2 + (int)sizeof(TreeShared) + (a.n + 1) * 8 +
                      a.n * (int)sizeof(TreeEntry);
    a.stages = (227 * 1024 - fixed) / stage;
    if (a.stages > kTreeMaxStages) a.stages = kTreeMaxStages;
    static std::atomic<unsigned long long> configured{0};
    cudaError_t e = tc_allow_smem(reinterpret_cast<const void *>(attn_tree_kernel<D, BF16>), 227 * 1024, configured);
    if (e != cudaSuccess) return e;
    attn_tree_kernel<D, BF16><<<grid, tree_threads(D), fixed + a.stages * stage, s>>>(mq, mk, mv, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // 8 rows a CTA, or 32 where 8 make more than 6 CTAs an SM.  The whole call with 8 and with 32, us, at 512 CTAs
    // of 8 rows: d = 64 16.6 to 19.4 and 19.2 to 20.0, d = 128 22.2 to 24.8 and 20.9 to 25.1, d = 256 22.5 to 24.5
    // and 22.9 to 24.5; at 128: 14.2 and 16.9, 14.8 and 18.7, 17.6 and 23.3; at 1024: 20.3 to 28.9 and 18.0 to 26.0,
    // 29.9 to 41.4 and 20.5 to 32.1, 29.7 to 43.6 and 21.2 to 33.8.
    const int item = tree_groups(D) * a.toks, rts = (a.T + item - 1) / item;
    const auto blocks = [&](int rows) { return (a.rows_cap + rows - 1) / rows; };
    constexpr int col_blocks = D / Combine<D>::kCols;
    const bool few = (long long)rts * blocks(8) * a.n * a.p.n_kv_heads * col_blocks <= 6LL * grid;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rts * blocks(few ? 8 : 32)), (unsigned)a.n,
                       (unsigned)(a.p.n_kv_heads * col_blocks));
    cfg.blockDim = dim3(Combine<D>::kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, BF16, 1>, a, grid)
               : cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, BF16, 4>, a, grid);
}

}  // namespace mk

using namespace mk;

extern "C" size_t mk_attention_tree_scratch_bytes(int T, int n_heads, int n_kv_heads, int head_dim) {
    if (T < 1 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > kTreeM ||
        head_dim < 1)
        return 0;
    return tree_scratch(T, n_heads, n_kv_heads, head_dim, tree_grid());
}

extern "C" mk_status mk_debug_attention_tree_wait(unsigned long long wait_ns, int drop_q) {
    if (drop_q != 0 && drop_q != 1) return pages_refuse("debug_attention_tree_wait", "drop_q must be 0 or 1");
    tree_wait_ns.store(wait_ns ? wait_ns : kTcTimeoutNs, std::memory_order_relaxed);
    tree_drop_q.store(drop_q, std::memory_order_relaxed);
    return MK_OK;
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
    if (n_heads / p->n_kv_heads > kTreeM)
        return pages_refuse(who, "at most 128 query heads per KV head", MK_ERR_UNSUPPORTED);
    if (n == 0) return MK_OK;
    if (!q || !out || !seqs || !scratch) return pages_refuse(who, "null pointer");
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)scratch) & 15)
        return pages_refuse(who, "q, out and scratch must be 16-byte aligned");
    const int d = p->head_dim;
    if (q_stride < (long long)n_heads * d || q_stride % 8 || out_stride < (long long)n_heads * d || out_stride % 8)
        return pages_refuse(who, "a stride is shorter than a row or not a multiple of 8");
    const int grid = tree_grid();
    if (scratch_bytes < tree_scratch(T, n_heads, p->n_kv_heads, d, grid))
        return pages_refuse(who, "scratch is smaller than mk_attention_tree_scratch_bytes");
    const size_t rows = (size_t)n * T, width = (size_t)n_heads * d * 2;
    if (pages_rows_meet(q, width, (size_t)q_stride * 2, out, width, (size_t)out_stride * 2, rows))
        return pages_refuse(who, "out must not overlap q");
    const size_t used = tree_scratch(T, n_heads, p->n_kv_heads, d, grid);
    for (const auto &x : {std::make_pair(q, q_stride), std::make_pair((const void *)out, out_stride)})
        if (pages_rows_meet(x.first, (rows - 1) * x.second * 2 + width, used, scratch, used, used, 1))
            return pages_refuse(who, "scratch must not overlap q or out");
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
    a.toks = kTreeM / a.G;
    a.rows_cap = tree_rows_cap(T, a.G, d);
    a.part_o = static_cast<float4 *>(scratch);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + (size_t)2 * grid * a.rows_cap * (d / 4));
    a.scale = (float)(1.4426950408889634 / std::sqrt((double)d));
    a.wait_ns = tree_wait_ns.load(std::memory_order_relaxed);
    a.drop_q = tree_drop_q.load(std::memory_order_relaxed);
    // a copy covers the part of a tile that lies in one page
    const int nt = tree_nt(d);
    int seg = nt;
    if (p->max_pages > 1)
        while (p->page_size % seg) seg /= 2;
    a.seg = seg;
    CUtensorMap mq, mk, mv;
    const uint64_t heads = (uint64_t)p->n_pages * p->n_kv_heads;
    const uint32_t blocks = seg == nt ? (uint32_t)(d / 64) : 1u;
    if (!tc_make_map_heads(&mq, q, (uint64_t)n * T, (uint64_t)q_stride, (uint32_t)n_heads, (uint32_t)d, (uint32_t)a.G,
                           (uint32_t)a.toks) ||
        !tc_make_map_pages(&mk, a.k, heads, (uint32_t)p->page_size, (uint32_t)d, (uint32_t)seg, blocks) ||
        !tc_make_map_pages(&mv, a.v, heads, (uint32_t)p->page_size, (uint32_t)d, (uint32_t)seg, blocks)) {
        pages_refuse(who, "the driver refused the tensor map");
        return MK_ERR_CUDA;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf16 = p->dtype == MK_BF16;
    cudaError_t e;
    if (d == 64)
        e = bf16 ? launch_tree<64, true>(mq, mk, mv, a, grid, s) : launch_tree<64, false>(mq, mk, mv, a, grid, s);
    else if (d == 128)
        e = bf16 ? launch_tree<128, true>(mq, mk, mv, a, grid, s) : launch_tree<128, false>(mq, mk, mv, a, grid, s);
    else
        e = bf16 ? launch_tree<256, true>(mq, mk, mv, a, grid, s) : launch_tree<256, false>(mq, mk, mv, a, grid, s);
    return pages_launched(e, who);
}
