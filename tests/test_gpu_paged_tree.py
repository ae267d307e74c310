"""Tree attention over a paged cache against a 64-bit implementation.

Every slot that holds no position is NaN, so reading one shows.  Tolerances
are the bounds derived in paged_common.tree_reference.
"""
import pytest
import torch

from paged_common import filled, generator, pack_bits, random_tree, tree_reference, visible

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]


def make(lengths, T, nq, nkv, d, ps, dtype, seed, n_new=None, q_std=1.5, **kw):
    n = len(lengths)
    new = [T] * n if n_new is None else n_new
    pool = filled(lengths, new, nkv=nkv, d=d, ps=ps, dtype=dtype, seed=seed, **kw)
    q = (torch.randn((n, T, nq, d), generator=generator(seed + 7)) * q_std).to(dtype)
    return pool, q, new


def run_and_compare(pool, q, seqs, new, seen, layer=0, cache=None, **kw):
    import tile_synchronised_b200 as mk
    cache = pool.to_cache() if cache is None else cache
    out = torch.full_like(q, 7.0).cuda()
    got = mk.attention_tree(q.cuda(), cache, layer, torch.tensor(seqs, dtype=torch.int32).cuda(),
                            n_new=torch.tensor(new, dtype=torch.int32).cuda(),
                            mask=None if seen is None else pack_bits(seen).cuda(), out=out, **kw)
    cache.check()
    ref, bound = tree_reference(pool, layer, q, seqs, new, seen, torch.full_like(q, 7.0))
    got = got.cpu().double()
    for i in range(len(seqs)):  # rows behind the last new token stay
        assert (got[i, new[i]:] == 7.0).all()
    off = (got - ref).abs()
    nan = torch.isnan(ref)
    assert (torch.isnan(got) | torch.isinf(got))[nan].all()
    assert torch.isfinite(got[~nan]).all()
    assert (off[~nan] <= bound[~nan]).all(), float((off[~nan] / bound[~nan].clamp_min(1e-30)).max())
    return got


def trees(n, T, seed):
    return torch.stack([visible(random_tree(T, seed + i)) for i in range(n)])


# lengths, T, nq, nkv, d, page size, type
SHAPES = [
    ([0], 1, 2, 2, 64, 16, torch.bfloat16),                      # one token, nothing before it
    ([1, 0, 17], 1, 8, 2, 128, 16, torch.bfloat16),              # single tokens, ragged
    ([127, 128, 129, 64, 255, 256], 1, 4, 1, 64, 64, torch.bfloat16),  # around a tile
    ([40], 5, 4, 2, 64, 16, torch.float16),
    ([100, 3, 250], 7, 6, 2, 128, 32, torch.bfloat16),           # group 3
    ([63, 64, 65], 9, 12, 4, 256, 16, torch.bfloat16),           # d = 256: tiles of 64
    ([30, 200], 33, 8, 1, 128, 48, torch.float16),               # group 8, pages of 48: 264 rows
    ([300], 128, 4, 4, 64, 128, torch.bfloat16),                 # 128 rows a head
    ([500, 10], 40, 14, 2, 64, 256, torch.bfloat16),             # group 7, pages over two tiles
    ([900], 65, 16, 2, 256, 64, torch.float16),                  # 520 rows at d = 256
    ([2500, 1, 700], 21, 8, 2, 128, 16, torch.bfloat16),
]


@pytest.mark.parametrize("lengths,T,nq,nkv,d,ps,dtype", SHAPES)
def test_tree_matches_64_bits(lengths, T, nq, nkv, d, ps, dtype):
    pool, q, new = make(lengths, T, nq, nkv, d, ps, dtype, 11)
    run_and_compare(pool, q, list(range(len(lengths))), new, trees(len(lengths), T, 5))


@pytest.mark.parametrize("lengths,T,nq,nkv,d,ps,dtype", SHAPES)
def test_causal_matches_64_bits(lengths, T, nq, nkv, d, ps, dtype):
    n = len(lengths)
    new = [max(0, T - 2 * i) for i in range(n)]  # ragged, possibly none
    pool, q, new = make(lengths, T, nq, nkv, d, ps, dtype, 12, n_new=new)
    run_and_compare(pool, q, list(range(n)), new, None)


# Many row tiles of one sequence, each with fewer positions than the next: tokens of a row tile that divide a tile of
# positions, are more than one, or neither; lengths of zero, one and around a tile.
CHUNKS = [
    ([0, 130], 300, 8, 2, 64, 16, torch.bfloat16),    # 64 tokens a row tile, tiles of 128
    ([1, 77], 260, 6, 2, 128, 48, torch.float16),     # 84 tokens
    ([127], 520, 1, 1, 64, 128, torch.bfloat16),      # 256 tokens
    ([5, 64, 0], 150, 7, 1, 256, 32, torch.bfloat16), # 18 tokens, tiles of 64
    ([63], 37, 128, 1, 64, 64, torch.bfloat16),       # 2 tokens
]


@pytest.mark.parametrize("lengths,T,nq,nkv,d,ps,dtype", CHUNKS)
def test_long_chunks_match_64_bits(lengths, T, nq, nkv, d, ps, dtype):
    n = len(lengths)
    pool, q, new = make(lengths, T, nq, nkv, d, ps, dtype, 31, n_new=[T - 33 * i for i in range(n)])
    run_and_compare(pool, q, list(range(n)), new, None)


def test_many_sequences_in_any_order():
    lengths = [(37 * i) % 211 for i in range(50)]
    pool, q, new = make(lengths, 3, 4, 2, 64, 16, torch.bfloat16, 13)
    seqs = torch.randperm(50, generator=generator(3)).tolist()
    run_and_compare(pool, q, seqs, new, trees(50, 3, 9))


def test_one_sequence_listed_twice():
    pool, q, new = make([90], 4, 4, 2, 64, 16, torch.bfloat16, 14)
    q2 = torch.cat([q, -q])
    seen = torch.cat([trees(1, 4, 1), trees(1, 4, 2)])
    run_and_compare(pool, q2, [0, 0], new * 2, seen)


def test_rows_that_see_nothing_are_zero():
    pool, q, new = make([0, 0], 6, 4, 2, 64, 16, torch.bfloat16, 15)
    seen = trees(2, 6, 4)
    seen[0, 2] = False
    seen[1] = False
    got = run_and_compare(pool, q, [0, 1], new, seen)
    assert (got[0, 2] == 0).all() and (got[1] == 0).all()


def test_masks_that_leave_out_the_token_itself():
    pool, q, new = make([20], 40, 4, 2, 64, 16, torch.bfloat16, 16)
    seen = torch.rand((1, 40, 40), generator=generator(8)) < 0.3
    run_and_compare(pool, q, [0], new, seen)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [64, 256])
def test_nonfinite_in_hidden_tokens_stays_hidden(value, d):
    """A drafted token whose V (or K) is not finite reaches only the rows that
    see it."""
    T, L = 37, 150
    pool, q, new = make([L], T, 4, 2, d, 16, torch.bfloat16, 17)
    seen = trees(1, T, 21)
    hidden = torch.zeros(T, dtype=torch.bool)
    hidden[[5, 33]] = True
    page, off = pool.at(0, L + 5)
    pool.kv[1, 0, page, 0, off, 3] = value  # V, one value of one head
    page, off = pool.at(0, L + 33)
    pool.kv[0, 0, page, 1, off] = float("nan")  # K of the other head
    seen[0, :, 33] = False
    got = run_and_compare(pool, q, [0], new, seen)
    sees = seen[0, :, 5]
    assert not torch.isfinite(got[0, sees][:, :2, 3]).any()
    assert torch.isfinite(got[0, ~sees]).all()


def test_lowest_and_infinite_scores():
    """Committed K rows so large that scores reach 1e5 either way, and a row of
    K that is -inf in one place: weights of 0 and 1, no NaN where q is finite."""
    pool, q, new = make([200], 4, 4, 2, 64, 16, torch.bfloat16, 18)
    page, off = pool.at(0, 77)
    pool.kv[0, 0, page, :, off] *= 10000.0
    q = q.abs() + torch.tensor(0.1, dtype=q.dtype)
    page, off = pool.at(0, 90)
    pool.kv[0, 0, page, :, off] = -1.0
    pool.kv[0, 0, page, :, off, 5] = float("-inf")
    import tile_synchronised_b200 as mk
    cache = pool.to_cache()
    got = mk.attention_tree(q.cuda(), cache, 0, torch.zeros(1, dtype=torch.int32).cuda()).cpu().double()
    assert torch.isfinite(got).all()
    K, V = (pool.rows(x, 0, 0, 204).double() for x in (0, 1))
    for t in range(4):
        for h in range(4):
            s = (K[h // 2, :201 + t] @ q[0, t, h].double()) / 8
            w = torch.softmax(s, 0)
            ref = w @ V[h // 2, :201 + t]
            # a score of size S is off by 66 2^-23 S in 32 bits
            slack = 2 * 66 * 2.0 ** -23 * float((K[h // 2, :201 + t].nan_to_num(0, 0, 0).abs() @ q[0, t, h].double().abs()).max()) / 8
            tol = (2 * 2.0 ** -8 + slack) * (w @ V[h // 2, :201 + t].abs()) + 1e-6
            assert ((got[0, t, h] - ref).abs() <= tol + slack * V[h // 2].abs().amax()).all()


def test_growing_scores_rescale():
    """Scores that rise along the cache, by more and by less than a rescale's
    threshold per tile."""
    for step in (0.002, 0.02, 0.2):
        pool, q, new = make([1500], 5, 4, 2, 64, 64, torch.bfloat16, 19, poison=False)
        for pos in range(1505):
            page, off = pool.at(0, pos)
            pool.kv[0, 0, page, :, off] = (pool.kv[0, 0, page, :, off].float() * 0.1 + step * pos / 8).to(pool.kv.dtype)
        q = (q.float().abs() * 0.3).to(q.dtype)
        run_and_compare(pool, q, [0], new, None)


def test_strided_tokens_and_layers():
    """q and out as parts of wider rows, the second of three layers."""
    import tile_synchronised_b200 as mk
    n, T, nq, nkv, d = 2, 5, 4, 2, 64
    pool = filled([33, 70], [T, T], layers=3, nkv=nkv, d=d, seed=20)
    wide = torch.randn((n, T, (nq + 3) * d), generator=generator(1)).to(torch.bfloat16).cuda()
    q = wide[..., d:(nq + 1) * d].view(n, T, nq, d)
    hold = torch.full((n, T, (nq + 1) * d), 5.0, dtype=torch.bfloat16, device="cuda")
    out = hold[..., :nq * d].view(n, T, nq, d)
    seen = trees(n, T, 6)
    cache = pool.to_cache()
    mk.attention_tree(q, cache, 1, torch.arange(n, dtype=torch.int32).cuda(), mask=pack_bits(seen).cuda(), out=out)
    cache.check()
    ref, bound = tree_reference(pool, 1, q.cpu(), [0, 1], [T, T], seen, out.cpu())
    assert ((out.cpu().double() - ref).abs() <= bound).all()
    assert (hold[..., nq * d:] == 5.0).all()


def test_results_repeat_bit_for_bit_and_scratch_does_not_matter():
    import tile_synchronised_b200 as mk
    pool, q, new = make([3000, 5, 900], 20, 8, 2, 128, 32, torch.bfloat16, 22)
    cache = pool.to_cache()
    seqs = torch.arange(3, dtype=torch.int32).cuda()
    a = mk.attention_tree(q.cuda(), cache, 0, seqs)
    need = mk.load().mk_attention_tree_scratch_bytes(20, 8, 2, 128)
    scratch = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(mk.attention_tree(q.cuda(), cache, 0, seqs, scratch=scratch), a)


def test_another_stream_and_a_captured_graph():
    """The call on a side stream, and captured once and replayed with other
    lengths, tokens and masks."""
    import tile_synchronised_b200 as mk
    pool, q, new = make([200, 60], 6, 4, 2, 64, 16, torch.bfloat16, 23)
    seen = trees(2, 6, 3)
    cache = pool.to_cache()
    side = torch.cuda.Stream()
    seqs, qd, bits = torch.arange(2, dtype=torch.int32).cuda(), q.cuda(), pack_bits(seen).cuda()
    n_new = torch.tensor(new, dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    got = mk.attention_tree(qd, cache, 0, seqs, n_new=n_new, mask=bits, stream=side)
    side.synchronize()
    ref, bound = tree_reference(pool, 0, q, [0, 1], new, seen, torch.zeros_like(q))
    assert ((got.cpu().double() - ref).abs() <= bound).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mk.attention_tree(qd, cache, 0, seqs, n_new=n_new, mask=bits)
    for lengths, new in (([200, 60], [6, 6]), ([11, 58], [6, 3]), ([0, 64], [1, 0])):
        cache.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        seen = trees(2, 6, 30 + lengths[0])
        bits.copy_(pack_bits(seen))
        out.fill_(7.0)
        g.replay()
        cache.check()
        pool.lengths[:] = torch.tensor(lengths)
        ref, bound = tree_reference(pool, 0, q, [0, 1], new, seen, torch.full_like(q, 7.0))
        assert ((out.cpu().double() - ref).abs() <= bound).all()


def test_model_cache_as_pages():
    """A context's contiguous cache (one page per sequence): a single token
    agrees with attention_decode over the same bytes."""
    import synth
    import tile_synchronised_b200 as mk
    shape = synth.TINY
    model = mk.Model(shape, synth.make_weights(shape, device="cuda"), batch=2)
    model.prefill(torch.randint(0, shape.vocab, (2, 50), generator=generator(2)))
    cache = mk.PagedCache.of_model(model)
    assert cache.page_size == shape.max_seq and cache.lengths.tolist() == [50, 50]
    cache.lengths.fill_(49)  # the last position as the new token
    q = torch.randn((2, 1, shape.n_heads, shape.head_dim), generator=generator(4)).to(torch.bfloat16).cuda()
    k, v = model.kv_views()
    for layer in range(shape.n_layers):
        got = mk.attention_tree(q, cache, layer, torch.arange(2, dtype=torch.int32).cuda())
        ref = mk.attention_decode(q[:, 0].float(), k[layer], v[layer], 50)
        cache.check()
        # attention_decode is exact to 1e-4 max |V|; the rest as in tree_reference (half a step of
        # the result and of the weights, both below half a step of max |V|)
        vmax = float(v[layer, :, :, :50].float().abs().max())
        assert float((got[:, 0].float() - ref).abs().max()) <= (2 * 2.0 ** -8 + 2e-4) * vmax


def test_bad_entries_are_reported_and_leave_their_rows():
    import tile_synchronised_b200 as mk
    pool, q, new = make([40, 30], 4, 4, 2, 64, 16, torch.bfloat16, 24, extra=1)
    cache = pool.to_cache()
    q3 = torch.cat([q, q[:1]]).cuda()
    out = torch.full_like(q3, 7.0)
    ref, bound = tree_reference(pool, 0, q, [0, 1], [4, 4], None, torch.zeros_like(q))
    for seqs, n_new, text in (([0, 5, 1], [4, 4, 4], "sequence index"), ([0, -1, 1], [4, 4, 4], "sequence index"),
                              ([0, 1, 1], [4, 9, 4], "count"), ([0, 1, 1], [4, -1, 4], "count")):
        out.fill_(7.0)
        mk.attention_tree(torch.cat([q[:1], q[:1], q[1:]]).cuda(), cache, 0, torch.tensor(seqs, dtype=torch.int32).cuda(),
                          n_new=torch.tensor(n_new, dtype=torch.int32).cuda(), out=out)
        with pytest.raises(mk.MkError, match=text):
            cache.check()
        cache.check()
        assert (out[1] == 7.0).all()
        assert ((out[[0, 2]].cpu().double() - ref).abs() <= bound).all()
    # a position without a page, or with one outside the pool, reads as zeros and is reported
    for page in (-1, 10 ** 6):
        cache.table[0, 1] = page
        got = mk.attention_tree(q.cuda(), cache, 0, torch.arange(2, dtype=torch.int32).cuda())
        with pytest.raises(mk.MkError, match="no page"):
            cache.check()
        assert ((got[1].cpu().double() - ref[1]).abs() <= bound[1]).all()
    # past the table's width
    cache.lengths[0] = cache.max_pages * 16 - 2
    mk.attention_tree(q.cuda(), cache, 0, torch.arange(2, dtype=torch.int32).cuda())
    with pytest.raises(mk.MkError, match="no page"):
        cache.check()


@pytest.mark.parametrize("T,d", [(1, 64), (70, 128), (9, 256)])  # two groups on one tile, two row tiles, one group
def test_a_wait_that_runs_out_is_reported(T, d):
    """Every CTA's first Q is left out: its K and V are all on their way by the
    time the wait for it runs out.  The rows are NaN, the status says so, and the
    next call is as before."""
    import tile_synchronised_b200 as mk
    from tile_synchronised_b200 import _lib
    lib = mk.load()
    pool, q, new = make([300, 5], T, 8, 2, d, 16, torch.bfloat16, 61)
    cache = pool.to_cache()
    seqs = torch.arange(2, dtype=torch.int32).cuda()
    good = mk.attention_tree(q.cuda(), cache, 0, seqs)
    cache.check()
    assert lib.mk_debug_attention_tree_wait(20_000_000, 1) == _lib.MK_OK  # 20 ms
    try:
        bad = mk.attention_tree(q.cuda(), cache, 0, seqs)
        with pytest.raises(mk.MkError, match="ran out") as e:
            cache.check()
    finally:
        assert lib.mk_debug_attention_tree_wait(0, 0) == _lib.MK_OK
    assert e.value.status == _lib.MK_ERR_TIMEOUT
    assert torch.isnan(bad).all()
    again = mk.attention_tree(q.cuda(), cache, 0, seqs)
    cache.check()
    assert torch.equal(again, good)


def test_tree_mask_on_the_gpu_reads_no_index_outside_a_row():
    """Parents that are no smaller index count as -1 there."""
    import tile_synchronised_b200 as mk
    parents = [random_tree(40, 3), random_tree(40, 4)]
    odd = torch.tensor(parents)
    odd[0, 7], odd[0, 8], odd[1, 0], odd[1, 39] = 40, 8, 5, -3
    parents[0][7] = parents[0][8] = parents[1][0] = parents[1][39] = -1
    assert torch.equal(mk.tree_mask(odd.cuda()).cpu(), pack_bits(torch.stack([visible(p) for p in parents])))


@pytest.mark.parametrize("page", [-1, 10 ** 6])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_see_a_missing_page_are_nan(d, page):
    """Many sequences, several to a CTA, some with a hole: all their rows are
    NaN, no other row is touched by it, and the next call is as before."""
    import tile_synchronised_b200 as mk
    n, T = 60, 3
    lengths = [20 + (41 * i) % 300 for i in range(n)]
    pool, q, new = make(lengths, T, 8, 4, d, 16, torch.bfloat16, 62)
    cache = pool.to_cache()
    seqs = torch.arange(n, dtype=torch.int32).cuda()
    good = mk.attention_tree(q.cuda(), cache, 0, seqs)
    cache.check()
    was = cache.table.clone()
    holes = [0, 7, 8, 31, 59]
    for k, s in enumerate(holes):
        cache.table[s, (k * 3) % ((lengths[s] + 15) // 16)] = page
    got = mk.attention_tree(q.cuda(), cache, 0, seqs)
    with pytest.raises(mk.MkError, match="no page"):
        cache.check()
    rest = [i for i in range(n) if i not in holes]
    assert torch.isnan(got[holes]).all()
    assert torch.equal(got[rest], good[rest])
    cache.table.copy_(was)
    assert torch.equal(mk.attention_tree(q.cuda(), cache, 0, seqs), good)
    cache.check()


def test_a_long_sequence_with_a_missing_page():
    """One sequence over many CTAs, hole in the middle: every row NaN.  A hole
    among the new tokens of a chunk: the row tiles before it are right."""
    import tile_synchronised_b200 as mk
    pool, q, new = make([9000], 4, 4, 2, 128, 16, torch.bfloat16, 63)
    cache = pool.to_cache()
    cache.table[0, 250] = -1
    got = mk.attention_tree(q.cuda(), cache, 0, torch.zeros(1, dtype=torch.int32).cuda())
    with pytest.raises(mk.MkError, match="no page"):
        cache.check()
    assert torch.isnan(got).all()
    pool, q, new = make([100], 500, 4, 2, 64, 16, torch.bfloat16, 64)  # row tiles of 64 new tokens, two at a time
    cache = pool.to_cache()
    good = mk.attention_tree(q.cuda(), cache, 0, torch.zeros(1, dtype=torch.int32).cuda())
    cache.check()
    cache.table[0, 25] = -1  # new tokens 300 .. 315
    got = mk.attention_tree(q.cuda(), cache, 0, torch.zeros(1, dtype=torch.int32).cuda())
    with pytest.raises(mk.MkError, match="no page"):
        cache.check()
    assert torch.isnan(got[0, 300:]).all() and torch.equal(got[0, :256], good[0, :256])


def test_no_new_token_in_any_entry():
    pool, q, _ = make([40, 0, 300], 5, 4, 2, 128, 16, torch.bfloat16, 65)
    run_and_compare(pool, q, [2, 0, 1], [0, 0, 0], None)


def test_two_calls_at_once_on_one_cache():
    """Two streams, scratch of their own, other sequences: the bits of one
    call after the other."""
    import tile_synchronised_b200 as mk
    pool, q, new = make([2000 - 60 * i for i in range(16)], 9, 16, 4, 128, 32, torch.bfloat16, 66)
    cache = pool.to_cache()
    qd, halves = q.cuda(), [torch.arange(a, a + 8, dtype=torch.int32).cuda() for a in (0, 8)]
    one = [mk.attention_tree(qd[8 * h:8 * h + 8], cache, 0, halves[h]) for h in (0, 1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [mk.attention_tree(qd[8 * h:8 * h + 8], cache, 0, halves[h], stream=streams[h]) for h in (0, 1)]
        torch.cuda.synchronize()
        cache.check()
        assert torch.equal(got[0], one[0]) and torch.equal(got[1], one[1])
