"""Page management and the norm + rotation + append pass against plain
implementations: integers and moved values bit for bit, computed values within
the bounds derived in paged_common.rope_reference."""
import pytest
import torch

from paged_common import Pool, filled, generator, pack_bits, random_tree, rope_reference, tree_reference, visible

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]


def ints(*v):
    return torch.tensor(v[0] if len(v) == 1 and isinstance(v[0], (list, tuple)) else v, dtype=torch.int32).cuda()


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("layers,nkv,d,ps,dtype", [(1, 1, 64, 16, torch.bfloat16), (3, 2, 128, 48, torch.float16),
                                                   (2, 4, 256, 32, torch.bfloat16), (5, 8, 64, 128, torch.float16)])
def test_a_run_of_operations(layers, nkv, d, ps, dtype):
    """Random reserves, forks, commits, cuts and frees, compared after each."""
    g = generator(layers * 100 + ps)
    r = lambda a, b: int(torch.randint(a, b + 1, (1,), generator=g))  # noqa: E731
    pool = Pool(layers, nkv, d, ps, 40, 9, 8, dtype, seed=3)
    cache = pool.to_cache()
    for step in range(60):
        what = r(0, 5)
        order = torch.randperm(9, generator=g).tolist()
        if what <= 2:  # new tokens for some sequences, an accepted path of each
            seqs = order[:r(1, 9)]
            T = r(1, 40)
            seqs = [s for s in seqs if int(pool.lengths[s]) + T <= 8 * ps]
            if not seqs:
                continue
            before = pool.clone()
            fits = pool.reserve(seqs, [T] * len(seqs))
            cache.reserve(ints(seqs), ints([T] * len(seqs)))
            if not fits:
                pool = before
                import tile_synchronised_b200 as mk
                with pytest.raises(mk.MkError, match="not enough free pages"):
                    cache.check()
                pool.same_as(cache)
                continue
            pool.same_as(cache)
            for s in seqs:  # the new tokens' values
                for t in range(T):
                    page, off = pool.at(s, int(pool.lengths[s]) + t)
                    v = torch.randn((2, layers, nkv, d), generator=g).to(dtype)
                    pool.kv[:, :, page, :, off] = v
            cache.kv.copy_(pool.kv)
            keep = [sorted(torch.randperm(T, generator=g)[:r(0, T)].tolist()) for _ in seqs]
            pool.compact(seqs, keep)
            padded = torch.full((len(seqs), T), -9, dtype=torch.int32)
            for i, k in enumerate(keep):
                padded[i, :len(k)] = torch.tensor(k, dtype=torch.int32)
            cache.compact(ints(seqs), ints([len(k) for k in keep]), padded.cuda())
        elif what == 3:
            empty = [s for s in order if int(pool.lengths[s]) == 0 and int(pool.table[s, 0]) < 0]
            full = [s for s in order if int(pool.lengths[s]) > 0]
            if not empty or not full:
                continue
            src = [full[r(0, len(full) - 1)] for _ in empty]
            pool.fork(src, empty)
            cache.fork(ints(src), ints(empty))
        else:
            seqs = order[:r(1, 4)]
            cut = [r(0, int(pool.lengths[s])) for s in seqs] if what == 4 else None
            pool.free(seqs, cut)
            cache.free(ints(seqs), None if cut is None else ints(cut))
        cache.check()
        pool.same_as(cache)
    cache.free(ints(list(range(9))))
    cache.check()
    assert int(cache.refs.abs().sum()) == 0 and int(cache.lengths.sum()) == 0 and (cache.table == -1).all()


def test_sharers_of_a_page_copy_in_list_order():
    """Three holders of a partly filled page, all reserved in one call: two
    copy, the last one keeps it."""
    pool = filled([21], [0], layers=2, extra=3, spare=6, poison=False)
    cache = pool.to_cache()
    pool.fork([0, 0], [1, 2])
    cache.fork(ints(0, 0), ints(1, 2))
    pool.reserve([2, 0, 1], [3, 3, 11])
    cache.reserve(ints(2, 0, 1), ints(3, 3, 11))
    cache.check()
    pool.same_as(cache)
    assert int(cache.refs.max()) == 3  # the full first page is still shared


def test_reserve_without_counts_or_at_a_page_end():
    pool = filled([32, 16, 0], [0, 0, 0], spare=4, poison=False)
    cache = pool.to_cache()
    for counts in ([0, 0, 0], [0, 1, 1]):
        pool.reserve([0, 1, 2], counts)
        cache.reserve(ints(0, 1, 2), ints(counts))
        cache.check()
        pool.same_as(cache)
    cache.reserve(ints([]), ints([]))


def test_a_pool_larger_than_one_scan():
    """Free pages far behind the first 1024, more than one for each sequence."""
    n = 5000
    pool = Pool(1, 1, 64, 16, n, 40, 60)
    pool.refs[:] = 1
    free = torch.randperm(n, generator=generator(5))[:2000]
    pool.refs[free] = 0
    cache = pool.to_cache()
    counts = [16 * (i % 50) + i for i in range(40)]
    assert pool.reserve(list(range(40)), counts)
    cache.reserve(ints(list(range(40))), ints(counts))
    cache.check()
    pool.same_as(cache)


def test_long_commits_move_in_order():
    """More kept positions than one block of offsets, each one place down, and
    a commit without moves."""
    T = 700
    pool = filled([5, 9], [T, T], layers=1, nkv=1, ps=16, poison=False)
    cache = pool.to_cache()
    keep = [list(range(1, T)), [t for t in range(T) if t % 3]]
    padded = torch.zeros((2, T), dtype=torch.int32)
    for i, k in enumerate(keep):
        padded[i, :len(k)] = torch.tensor(k)
    pool.compact([0, 1], keep)
    cache.compact(ints(0, 1), ints([len(k) for k in keep]), padded.cuda())
    cache.check()
    pool.same_as(cache)
    cache.free(ints(0, 1), ints(5, 9))
    pool.free([0, 1], [5, 9])
    cache.reserve(ints(0, 1), ints(30, 2))
    pool.reserve([0, 1], [30, 2])
    pool.compact([0, 1], [list(range(30)), [0, 1]])
    cache.compact(ints(0, 1), ints(30, 2))
    cache.check()
    pool.same_as(cache)


@pytest.mark.parametrize("layers,nkv,d,ps", [(1, 1, 64, 16), (3, 2, 128, 48), (2, 8, 256, 128)])
def test_copy_between_pools_and_within_one(layers, nkv, d, ps):
    a, b = Pool(layers, nkv, d, ps, 13, 1, 1, seed=1), Pool(layers, nkv, d, ps, 9, 1, 1, seed=2)
    ca, cb = a.to_cache(), b.to_cache()
    b.kv[:, :, [4, 0, 8]] = a.kv[:, :, [12, 12, 3]]
    cb.copy(ints(12, 12, 3), ints(4, 0, 8), source=ca)
    cb.check()
    b.same_as(cb)
    a.kv[:, :, [1, 2]] = a.kv[:, :, [0, 0]]
    ca.copy(ints(0, 0), ints(1, 2))
    ca.check()
    a.same_as(ca)


def test_wrong_entries_are_left_out_and_reported():
    import tile_synchronised_b200 as mk
    pool = filled([20, 33, 8], [12, 12, 12], layers=2, spare=8, extra=2, poison=False, seed=6)
    cache = pool.to_cache()

    def expect(text):
        with pytest.raises(mk.MkError, match=text):
            cache.check()
        cache.check()
        pool.same_as(cache)

    for seqs in ([0, 7, 1], [0, -3, 1]):  # out of range: the others are done
        cache.reserve(ints(seqs), ints(28, 30, 15))
        pool.reserve([0, 1], [28, 15])
        expect("sequence index")
    cache.reserve(ints(2, 2), ints(40, 40))  # listed twice
    expect("sequence index")
    cache.reserve(ints(2, 0), ints(-1, 1))
    expect("count")
    cache.reserve(ints(2), ints(10 ** 6))
    expect("no page")
    cache.fork(ints(0, 0), ints(3, 3))
    expect("sequence index")
    cache.fork(ints(0, 3), ints(3, 4))  # a dst that is a src
    pool.fork([], [])
    # entry 0's dst is entry 1's src: left out; entry 1 forks an empty sequence
    expect("sequence index")
    cache.fork(ints(0), ints(1))
    expect("not empty")
    cache.free(ints(0, 0))
    expect("sequence index")
    cache.free(ints(0, 1), ints(21, 30))
    pool.free([1], [30])
    expect("count")
    keep = torch.tensor([[0, 2, 2], [0, 1, 2]], dtype=torch.int32).cuda()
    cache.compact(ints(0, 1), ints(3, 2), keep)  # not ascending
    pool.compact([1], [[0, 1]])
    expect("kept index")
    cache.compact(ints(0, 0), ints(1, 1), keep)
    expect("sequence index")
    cache.compact(ints(0, 2), ints(4, 1), keep)  # more than the list is wide
    pool.compact([2], [[0]])
    expect("kept index")
    cache.compact(ints(2), ints(2), torch.tensor([[0, 4000]], dtype=torch.int32).cuda())
    expect("no page")
    # a move into a page that another sequence holds too
    cache.fork(ints(0), ints(3))
    pool.fork([0], [3])
    cache.compact(ints(0), ints(2), torch.tensor([[1, 2]], dtype=torch.int32).cuda())
    expect("reserve first")
    # copies: out of range, written twice, a source that is written
    n = cache.n_pages
    for src, dst, good in (([0, n], [1, 2], [(0, 1)]), ([0, 1], [-1, 2], [(1, 2)]), ([0, 1, 4], [2, 2, 3], [(4, 3)]),
                           ([0, 1], [1, 2], [(0, 1)])):
        cache.copy(ints(src), ints(dst))
        for s, d in good:
            pool.kv[:, :, d] = pool.kv[:, :, s]
        expect("page index")


def test_a_fork_of_a_row_with_a_hole_is_left_undone():
    import tile_synchronised_b200 as mk
    for page in (-1, 99):
        pool = filled([40, 33], [0, 0], layers=1, spare=2, extra=2, poison=False, seed=8)
        pool.table[0, 1] = page
        cache = pool.to_cache()
        cache.fork(ints(0, 1), ints(2, 3))
        pool.fork([1], [3])
        with pytest.raises(mk.MkError, match="no page"):
            cache.check()
        pool.same_as(cache)


def test_operations_in_a_captured_graph():
    """A step's operations captured once, replayed on other lists."""
    pool = filled([20, 33], [0, 0], layers=2, spare=8, extra=1, poison=False, seed=7)
    cache = pool.to_cache()
    seqs, counts, n_keep = ints(0, 1), ints(5, 5), ints(2, 2)
    keep = torch.tensor([[1, 3, 0], [0, 4, 0]], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.reserve(seqs, counts)
        cache.compact(seqs, n_keep, keep)
    pool.same_as(cache)  # nothing ran yet
    for s, c, k in (([0, 1], [5, 5], [[1, 3], [0, 4]]), ([1, 0], [10, 7], [[2, 5, 9], []])):
        seqs.copy_(ints(s))
        counts.copy_(ints(c))
        n_keep.copy_(ints([len(x) for x in k]))
        for i, x in enumerate(k):
            keep[i, :len(x)] = ints(x)
        g.replay()
        pool.reserve(s, c)
        pool.compact(s, k)
        cache.check()
        pool.same_as(cache)


# ------------------------------------------------------------------ norm + rotation + append
ROPE = [  # lengths, T, nq, nkv, d, page size, type, input type, gains, depth
    ([0], 1, 2, 2, 64, 16, torch.bfloat16, torch.float32, True, False),
    ([5, 0, 31], 1, 32, 8, 128, 16, torch.bfloat16, torch.float32, True, False),
    ([40, 3], 9, 12, 4, 256, 16, torch.float16, torch.float16, False, True),
    ([100000, 999], 4, 4, 2, 64, 4096, torch.bfloat16, torch.bfloat16, True, True),  # far positions
    ([10, 60, 7], 35, 14, 2, 64, 32, torch.float16, torch.float32, True, True),
    ([77], 5, 8, 8, 128, 48, torch.bfloat16, torch.bfloat16, False, False),
    ([1, 2, 3], 17, 1, 1, 256, 16, torch.bfloat16, torch.float32, True, False),
]


@pytest.mark.parametrize("lengths,T,nq,nkv,d,ps,dtype,src,norm,tree", ROPE)
def test_norm_rope_append_matches_64_bits(lengths, T, nq, nkv, d, ps, dtype, src, norm, tree):
    import tile_synchronised_b200 as mk
    n = len(lengths)
    g = generator(31)
    new = [max(0, T - 3 * i) for i in range(n)]
    pool = filled(lengths, [T] * n, layers=2, nkv=nkv, d=d, ps=ps, dtype=dtype, seed=32, poison=False)
    qkv = (torch.randn((n, T, (nq + 2 * nkv) * d), generator=g) * 2).to(src)
    gains = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2)] if norm else [None, None]
    depth = None
    if tree:
        depth = torch.stack([visible(random_tree(T, 40 + i)).sum(1).int() - 1 for i in range(n)])
    cache = pool.to_cache()
    seqs = torch.randperm(n, generator=g).tolist()
    q0 = torch.full((n, T, nq, d), 7.0, dtype=dtype)
    q = mk.qk_norm_rope(qkv.cuda(), cache, 1, ints(seqs), nq, 500000.0, *(None if x is None else x.cuda() for x in gains),
                        eps=1e-6, n_new=ints(new), depth=None if depth is None else depth.cuda(), out=q0.cuda())
    cache.check()
    ref, bound, kv = rope_reference(pool, 1, qkv, nq, 500000.0, *gains, 1e-6, seqs, new, depth, q0)
    assert ((q.cpu().double() - ref).abs() <= bound).all()
    got = cache.kv.cpu()
    for (i, t), (k, v, kb) in kv.items():
        page, off = pool.at(seqs[i], lengths[seqs[i]] + t)
        assert ((got[0, 1, page, :, off].double() - k).abs() <= kb).all()
        assert torch.equal(got[1, 1, page, :, off], v.to(dtype))
        got[:, 1, page, :, off] = pool.kv[:, 1, page, :, off]
    assert torch.equal(got, pool.kv)  # nothing else was written


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("only", ["q", "k"])
def test_a_gain_for_one_of_q_and_k(d, only):
    """3 q heads and 1 KV head: q and k heads side by side in a warp, one normed."""
    import tile_synchronised_b200 as mk
    g = generator(35)
    T, nq = 6, 3
    pool = filled([9], [T], nkv=1, d=d, seed=36, poison=False)
    cache = pool.to_cache()
    qkv = torch.randn((1, T, (nq + 2) * d), generator=g)
    gain = (1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16)
    gains = (gain, None) if only == "q" else (None, gain)
    q = mk.qk_norm_rope(qkv.cuda(), cache, 0, ints(0), nq, 10000.0, *(None if x is None else x.cuda() for x in gains))
    cache.check()
    ref, bound, kv = rope_reference(pool, 0, qkv, nq, 10000.0, *gains, 1e-6, [0], [T], None, torch.zeros_like(q.cpu()))
    assert ((q.cpu().double() - ref).abs() <= bound).all()
    got = cache.kv.cpu()
    for (i, t), (k, v, kb) in kv.items():
        page, off = pool.at(0, 9 + t)
        assert ((got[0, 0, page, :, off].double() - k).abs() <= kb).all()
        assert torch.equal(got[1, 0, page, :, off], v.to(torch.bfloat16))


def test_zero_and_tiny_heads():
    """A head of zeros stays zero under the norm, without a NaN."""
    import tile_synchronised_b200 as mk
    pool = filled([3], [2], nkv=1, d=64, poison=False)
    cache = pool.to_cache()
    qkv = torch.zeros((1, 2, 3 * 64))
    qkv[0, 1] = 1e-25
    gain = torch.ones(64, dtype=torch.bfloat16).cuda()
    q = mk.qk_norm_rope(qkv.cuda(), cache, 0, ints(0), 1, 10000.0, gain, gain, eps=1e-6)
    cache.check()
    assert (q == 0).all() or q.abs().max() < 1e-20
    assert torch.isfinite(cache.kv.float()).all()


def test_slots_that_may_not_be_written():
    """No page, a shared page, a sequence listed twice: reported, K/V untouched."""
    import tile_synchronised_b200 as mk
    pool = filled([10, 14], [0, 0], nkv=2, extra=2, spare=3, poison=False)
    cache = pool.to_cache()
    qkv = torch.randn((1, 3, 8 * 64), generator=generator(1)).cuda()
    mk.qk_norm_rope(qkv, cache, 0, ints(1), 4, 10000.0)  # token 2 would need another page
    with pytest.raises(mk.MkError, match="no page"):
        cache.check()
    cache.kv.copy_(pool.kv)
    cache.fork(ints(0), ints(2))
    pool.fork([0], [2])
    q = mk.qk_norm_rope(qkv, cache, 0, ints(2), 4, 10000.0)
    with pytest.raises(mk.MkError, match="reserve first"):
        cache.check()
    pool.same_as(cache)
    two = mk.qk_norm_rope(torch.cat([qkv, qkv]), cache, 0, ints(0, 0), 4, 10000.0)
    with pytest.raises(mk.MkError, match="sequence index"):
        cache.check()
    pool.same_as(cache)
    assert torch.equal(two[0], q[0]) and torch.equal(two[1], q[0])  # q does not depend on the slot


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_drafting_loop(dtype):
    """Prompt, fork, drafted trees, accepted paths, single tokens, frees, on one
    pool with two layers: every attention against 64 bits over the pages'
    own bytes, and the pages against the plain pool."""
    import tile_synchronised_b200 as mk
    layers, nq, nkv, d, ps, theta = 2, 8, 2, 64, 16, 10000.0
    pool = Pool(layers, nkv, d, ps, 64, 6, 12, dtype, seed=50)
    cache = pool.to_cache()
    g = generator(51)
    gain = torch.ones(d, dtype=torch.bfloat16)

    def step(seqs, T, parents, keep):
        n = len(seqs)
        seen = None if parents is None else torch.stack([visible(p) for p in parents])
        depth = None if parents is None else (seen.sum(-1) - 1).int()
        assert pool.reserve(seqs, [T] * n)
        cache.reserve(ints(seqs), ints([T] * n))
        for layer in range(layers):
            qkv = torch.randn((n, T, (nq + 2 * nkv) * d), generator=g)
            q = mk.qk_norm_rope(qkv.cuda(), cache, layer, ints(seqs), nq, theta, gain.cuda(), gain.cuda(),
                                depth=None if depth is None else depth.cuda())
            out = mk.attention_tree(q, cache, layer, ints(seqs),
                                    mask=None if parents is None else mk.tree_mask(torch.tensor(parents)).cuda())
            cache.check()
            ref, bound, kv = rope_reference(pool, layer, qkv, nq, theta, gain, gain, 1e-6, seqs, [T] * n, depth,
                                            torch.zeros((n, T, nq, d), dtype=dtype))
            assert ((q.cpu().double() - ref).abs() <= bound).all()
            new = cache.kv.cpu()
            for (i, t), (k, v, kb) in kv.items():
                page, off = pool.at(seqs[i], int(pool.lengths[seqs[i]]) + t)
                assert ((new[0, layer, page, :, off].double() - k).abs() <= kb).all()
                pool.kv[:, layer, page, :, off] = new[:, layer, page, :, off]
            pool.same_as(cache)
            ref, bound = tree_reference(pool, layer, q.cpu(), seqs, [T] * n, seen, torch.zeros(q.shape, dtype=dtype))
            assert ((out.cpu().double() - ref).abs() <= bound).all()
        pool.compact(seqs, keep)
        width = max(1, max(len(k) for k in keep))
        padded = torch.zeros((n, width), dtype=torch.int32)
        for i, k in enumerate(keep):
            padded[i, :len(k)] = torch.tensor(k, dtype=torch.int32)
        cache.compact(ints(seqs), ints([len(k) for k in keep]), padded.cuda())
        cache.check()
        pool.same_as(cache)

    def path(parents, leaf):
        out = []
        while leaf >= 0:
            out.insert(0, leaf)
            leaf = parents[leaf]
        return out

    step([0, 1], 37, None, [list(range(37)), list(range(20))])      # prompts, causal
    pool.fork([0, 1, 0], [2, 3, 4])
    cache.fork(ints(0, 1, 0), ints(2, 3, 4))
    for it in range(3):
        seqs = [4, 0, 3, 2, 1]
        parents = [random_tree(11, 60 + 5 * it + i) for i in range(5)]
        step(seqs, 11, parents, [path(parents[i], (3 * i + 5 * it) % 11) for i in range(5)])
        step(seqs, 1, None, [[0]] * 5)                               # a single token
    pool.free([0, 3], [30, 0])
    cache.free(ints(0, 3), ints(30, 0))
    step([0], 6, None, [[0, 1, 2]])
    pool.same_as(cache)


def test_projection_to_attention_to_projection():
    """linear_tc's fp32 rows feed qk_norm_rope, attention_tree's 16-bit rows
    feed linear_tc: one attention block over new tokens of two sequences."""
    import tile_synchronised_b200 as mk
    n, T, nq, nkv, d, hidden = 2, 6, 4, 2, 64, 256
    g = generator(70)
    pool = filled([25, 9], [T, T], nkv=nkv, d=d, seed=71)
    cache = pool.to_cache()
    x = torch.randn((n * T, hidden), generator=g).to(torch.bfloat16)
    w = (torch.randn(((nq + 2 * nkv) * d, hidden), generator=g) * 0.05).to(torch.bfloat16)
    wo = (torch.randn((hidden, nq * d), generator=g) * 0.05).to(torch.bfloat16)
    qkv = mk.linear_tc(x.cuda(), w.cuda()).view(n, T, -1)
    q = mk.qk_norm_rope(qkv, cache, 0, ints(0, 1), nq, 10000.0)
    o = mk.attention_tree(q, cache, 0, ints(0, 1))
    y = mk.linear_tc(o.view(n * T, nq * d), wo.cuda())
    cache.check()
    pool.kv = cache.kv.cpu()
    ref, bound = tree_reference(pool, 0, q.cpu(), [0, 1], [T, T], None, torch.zeros_like(q.cpu()))
    assert ((o.cpu().double() - ref).abs() <= bound).all()
    exact = o.cpu().double().view(n * T, -1) @ wo.double().T
    slack = 2 * nq * d * 2.0 ** -24 * (o.cpu().double().view(n * T, -1).abs() @ wo.double().abs().T)
    assert ((y.cpu().double() - exact).abs() <= slack + 2.0 ** -23 * exact.abs()).all()


def test_offsets_behind_32_bits():
    """The same sequences in a small pool and at the end of one of more than
    2^32 values: the same bits."""
    import tile_synchronised_b200 as mk
    nkv, ps, d, nq, T = 8, 64, 128, 16, 5
    small = filled([130, 64, 7], [64, 64, 64], layers=1, nkv=nkv, d=d, ps=ps, seed=21, poison=False)
    a = small.to_cache()
    n = a.n_pages
    pages = 33100
    kv = torch.empty((2, 1, pages, nkv, ps, d), dtype=torch.bfloat16, device="cuda")
    assert kv.numel() // 2 > 2 ** 31 and kv.numel() > 2 ** 32
    kv[:, :, pages - n:] = a.kv
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - n:] = a.refs
    b = mk.PagedCache.over(kv, torch.where(a.table >= 0, a.table + (pages - n), -1), a.lengths.clone(), refs)
    seqs = ints(2, 0, 1)
    qkv = torch.randn((3, T, (nq + 2 * nkv) * d), generator=generator(4)).cuda()
    mask = pack_bits(torch.stack([visible(random_tree(T, k)) for k in range(3)])).cuda()
    got = []
    for c in (a, b):
        q = mk.qk_norm_rope(qkv, c, 0, seqs, nq, 10000.0)
        o = mk.attention_tree(q, c, 0, seqs, mask=mask)
        c.compact(seqs, ints(3, 2, 1), torch.tensor([[0, 2, 4], [1, 3, 0], [4, 0, 0]], dtype=torch.int32).cuda())
        c.check()
        got.append((q, o, c.lengths, c.kv[:, :, c.n_pages - n:]))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    src, dst = ints(pages - n, pages - 1), ints(0, 1)
    b.copy(src, dst)
    b.check()
    assert torch.equal(kv[:, :, 0], kv[:, :, pages - n]) and torch.equal(kv[:, :, 1], kv[:, :, pages - 1])


def test_a_check_during_a_capture_is_refused():
    import tile_synchronised_b200 as mk
    pool = filled([20, 5], [0, 0], layers=1, spare=4, seed=9)
    cache = pool.to_cache()
    seqs, counts = ints(0, 1), ints(12, 27)  # up to the table's 32 positions
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.reserve(seqs, counts)
        with pytest.raises(mk.MkError, match="captured"):
            cache.check()
    pool.same_as(cache)
    graph.replay()
    cache.check()
    pool.reserve([0, 1], [12, 27])
    pool.same_as(cache)


def test_a_reserve_behind_a_page_outside_the_pool_is_left_undone():
    import tile_synchronised_b200 as mk
    pool = filled([20, 33], [28, 3], layers=1, spare=8, extra=1, poison=False, seed=10)
    pool.refs[pool.table[0, 2]] = 0  # the row ends behind the partly filled page
    pool.table[0, 1:] = torch.tensor([99, -1], dtype=torch.int32)
    cache = pool.to_cache()
    cache.reserve(ints(0, 1, 2), ints(28, 15, 17))
    with pytest.raises(mk.MkError, match="page index"):
        cache.check()
    pool.reserve([1, 2], [15, 17])
    pool.same_as(cache)


@pytest.mark.parametrize("n,T", [(2, 5), (8, 151)])
def test_q_in_place_and_between_the_rows_of_qkv(n, T):
    """q over qkv's own q heads, and q rows between the rows of qkv: the bits of
    a q of its own.  The attention's result between the rows of its q."""
    import tile_synchronised_b200 as mk
    nq, nkv, d = 20, 4, 64
    pool = filled([40 + i for i in range(n)], [T] * n, nkv=nkv, d=d, seed=37, poison=False)
    a, b, c = (pool.to_cache() for _ in range(3))
    width = (nq + 2 * nkv) * d
    hold = torch.randn((n, T, width + nq * d), generator=generator(38)).to(torch.bfloat16).cuda()
    qkv = hold[..., :width]
    gain = (1 + 0.2 * torch.randn(d, generator=generator(39))).to(torch.bfloat16).cuda()
    seqs = ints(list(range(n)))
    ref = mk.qk_norm_rope(qkv.clone(), a, 0, seqs, nq, 10000.0, gain, gain)
    between = hold[..., width:].view(n, T, nq, d)
    assert torch.equal(mk.qk_norm_rope(qkv, b, 0, seqs, nq, 10000.0, gain, gain, out=between), ref)
    over = hold[..., :nq * d].view(n, T, nq, d)
    mk.qk_norm_rope(qkv, c, 0, seqs, nq, 10000.0, gain, gain, out=over)
    assert torch.equal(over, ref)
    for x in (a, b, c):
        x.check()
        assert torch.equal(x.kv, a.kv)
    o = mk.attention_tree(ref, a, 0, seqs)
    mk.attention_tree(between, a, 0, seqs, out=over)
    assert torch.equal(over, o)
    with pytest.raises(mk.MkError, match="overlap"):
        mk.attention_tree(between, a, 0, seqs, out=hold[..., width - 8:-8].view(n, T, nq, d))


def test_tensors_dropped_behind_a_call_on_another_stream():
    """While the other stream has not run the call yet, memory of its tensors
    is not given to others."""
    import tile_synchronised_b200 as mk
    n, T, nq, nkv, d = 2, 600, 32, 2, 64
    pool = filled([20, 33], [T, T], nkv=nkv, d=d, spare=2, seed=40, poison=False)
    cache = pool.to_cache()
    side = torch.cuda.Stream()
    seqs, zero = ints(0, 1), ints(0, 0)
    qkv = torch.randn((n, T, (nq + 2 * nkv) * d), generator=generator(41)).to(torch.bfloat16)
    ref = mk.qk_norm_rope(qkv.cuda(), cache, 0, seqs, nq, 10000.0)
    att = mk.attention_tree(ref, cache, 0, seqs)
    warm = pool.to_cache()  # a kernel's first launch may wait for the device
    warm.reserve(seqs, zero)
    warm.compact(seqs, zero)
    warm.free(seqs)
    torch.cuda.synchronize()

    def dropped(make, call):
        x = make()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)  # some 50 ms
        got, at = call(x), x.data_ptr()
        del x
        others = [make() for _ in range(3)]
        assert not side.query()
        assert all(o.data_ptr() != at for o in others)
        side.synchronize()
        return got

    qkv = qkv.cuda()
    assert torch.equal(dropped(lambda: qkv.clone(), lambda x: mk.qk_norm_rope(x, cache, 0, seqs, nq, 10000.0, stream=side)), ref)
    assert torch.equal(dropped(lambda: ref.clone(), lambda x: mk.attention_tree(x, cache, 0, seqs, stream=side)), att)
    dropped(lambda: zero.clone(), lambda x: cache.reserve(seqs, x, stream=side))
    dropped(lambda: zero.clone(), lambda x: cache.compact(seqs, x, stream=side))
    cut = ints(20, 20)
    dropped(lambda: cut.clone(), lambda x: cache.free(seqs, x, stream=side))
    cache.check()
    assert cache.lengths.tolist() == [20, 20]


def test_a_capture_on_a_stream_that_the_calls_are_given():
    """Tensors made and dropped inside the capture."""
    import tile_synchronised_b200 as mk
    T, nq, nkv, d = 5, 4, 2, 64
    pool = filled([20, 33], [T, T], nkv=nkv, d=d, spare=2, seed=42, poison=False)
    a, b = pool.to_cache(), pool.to_cache()
    qkv = torch.randn((2, T, (nq + 2 * nkv) * d), generator=generator(43)).cuda()
    seqs = ints(0, 1)
    ref = mk.attention_tree(mk.qk_norm_rope(qkv, a, 0, seqs, nq, 10000.0), a, 0, seqs)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        q = mk.qk_norm_rope(qkv * 1.0, b, 0, seqs, nq, 10000.0, stream=side)
        out = mk.attention_tree(q, b, 0, seqs, stream=side)
        del q
        b.compact(seqs, seqs + 1, stream=side)
    for _ in range(2):
        b.lengths.copy_(a.lengths)
        out.zero_()
        graph.replay()
        b.check()
        assert torch.equal(out, ref) and b.lengths.tolist() == [21, 35]
