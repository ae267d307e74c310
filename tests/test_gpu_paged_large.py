"""The paged operators at sizes where the kernels are in their steady state:
many tiles of an item per CTA, several items per CTA, joins of many records,
four tokens a CTA in the rotation pass, long chunks, and the largest lists and
pools.  Against the same 64-bit implementations and bounds as the small cases."""
import pytest
import torch

from paged_common import Pool, filled, generator, random_tree, rope_reference, visible
from test_gpu_paged_cache import ints
from test_gpu_paged_tree import make, run_and_compare, trees

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def tiles(lengths, T, nq, nkv, d):
    """(items, units) of a call whose rows all see every position: a unit is a
    tile of 128 positions (64 at d = 256), and an item starts with two."""
    nt, rows = (64, 128) if d == 256 else (128, 256)
    item = rows // 128 * (128 // (nq // nkv))
    rts = -(-T // item)
    return len(lengths) * nkv * rts, sum(nkv * rts * (-(-(L + T) // nt) + 2) for L in lengths)


def grow(pool, step):
    """K rises along the positions, so that scores of positive queries do."""
    for s in range(pool.table.shape[0]):
        n = int(pool.lengths[s])
        pos = torch.arange(n)
        page, off = pool.table[s].long()[pos // pool.ps], pos % pool.ps
        k = pool.kv[0, 0][page, :, off].float() * 0.1 + step * pos[:, None, None] / 8
        pool.kv[0, 0].index_put_((page[:, None], torch.arange(k.shape[1])[None], off[:, None]), k.to(pool.kv.dtype))


# lengths, T, nq, nkv, d, page size, type: at most 128 rows (groups on alternate tiles), more (two row tiles), d = 256
STEADY = [([4100 - 130 * i for i in range(16)], 5, 16, 8, 64, 64, torch.bfloat16),
          ([4100 - 130 * i for i in range(16)], 7, 8, 8, 128, 16, torch.float16),
          ([6200 - 90 * i for i in range(16)], 48, 16, 4, 64, 128, torch.float16),
          ([6200 - 90 * i for i in range(16)], 50, 12, 4, 128, 32, torch.bfloat16),
          ([3300 - 110 * i for i in range(12)], 9, 8, 4, 256, 64, torch.bfloat16)]


@pytest.mark.parametrize("step", [None, 0.002, 0.02, 0.2])
@pytest.mark.parametrize("lengths,T,nq,nkv,d,ps,dtype", STEADY)
def test_many_tiles_of_an_item_per_cta(lengths, T, nq, nkv, d, ps, dtype, step):
    """Scores at random, and rising along the cache by more and by less than a
    rescale's threshold per tile.  Each CTA goes round its ring of copies."""
    items, units = tiles(lengths, T, nq, nkv, d)
    depth = {64: 12, 128: 6, 256: 5}[d]  # of the ring, in copies; a tile takes two
    assert units // sms() > depth and units // sms() * items < units * 2
    pool, q, new = make(lengths, T, nq, nkv, d, ps, dtype, 81, poison=step is None)
    seen = trees(len(lengths), T, 7)
    if step is not None:
        grow(pool, step)
        q = (q.float().abs() * 0.3).to(dtype)
    run_and_compare(pool, q, list(range(len(lengths))), new, seen)


@pytest.mark.parametrize("d,nq,nkv,dtype", [(64, 32, 8, torch.bfloat16), (128, 16, 4, torch.float16),
                                            (256, 8, 4, torch.bfloat16)])
@pytest.mark.parametrize("causal", [True, False])
def test_several_items_of_two_row_tiles_per_cta(d, nq, nkv, dtype, causal):
    """Short sequences, each with more than 128 rows: Q is reloaded under the
    last S of the item before; items end and begin inside a CTA's range, and the
    last row tiles are ragged."""
    lengths, T = [(53 * i) % 300 for i in range(40)], 70
    items, units = tiles(lengths, T, nq, nkv, d)
    assert items > 2 * sms()
    new = [T - (i * 7) % T for i in range(40)]
    pool, q, _ = make(lengths, T, nq, nkv, d, 16, dtype, 82, n_new=new)
    run_and_compare(pool, q, list(range(40)), new, None if causal else trees(40, T, 8))


@pytest.mark.parametrize("d,T,dtype", [(64, 100, torch.bfloat16), (128, 111, torch.bfloat16), (128, 100, torch.float16),
                                       (256, 61, torch.float16)])
def test_joins_of_more_records_than_are_loaded_at_a_time(d, T, dtype):
    """Items of many rows that five or six CTAs share: the join with 32 rows a
    CTA, several rounds of records, a ragged last row tile."""
    lengths, nq, nkv = [6000, 4700], 32, 8
    items, units = tiles(lengths, T, nq, nkv, d)
    rows = 128 if d == 256 else 256
    assert items * (rows // 8) * (2 if d == 256 else 1) > 6 * sms()  # more CTAs than the join with 8 rows each is for
    assert sms() > 4 * items  # some items have more than four records
    pool, q, new = make(lengths, T, nq, nkv, d, 64, dtype, 83)
    run_and_compare(pool, q, [0, 1], new, trees(2, T, 9))


@pytest.mark.parametrize("L,T,nq,nkv,d,ps,dtype", [(700, 2100, 4, 1, 64, 64, torch.bfloat16),
                                                   (0, 4097, 1, 1, 128, 128, torch.bfloat16),
                                                   (33, 2047, 2, 1, 256, 48, torch.float16)])
def test_chunks_of_thousands_of_tokens(L, T, nq, nkv, d, ps, dtype):
    pool, q, new = make([L], T, nq, nkv, d, ps, dtype, 84)
    run_and_compare(pool, q, [0], new, None)


def test_the_longest_list_of_sequences():
    n = 1024
    lengths = [(7 * i) % 45 for i in range(n)]
    new = [(i * 5) % 3 for i in range(n)]
    pool, q, _ = make(lengths, 2, 2, 1, 64, 16, torch.bfloat16, 85, n_new=new)
    order = torch.randperm(n, generator=generator(5)).tolist()
    inverse = [new[s] for s in order]
    run_and_compare(pool, q, order, inverse, None)


def test_pages_of_the_longest_list_of_sequences():
    """512 sequences forked into 512 more, all 1024 reserved, committed, cut and freed."""
    pool = filled([(11 * i) % 60 + 1 for i in range(512)], [0] * 512, layers=2, nkv=1, extra=512, spare=2600,
                  poison=False, seed=86)
    pool.table = torch.cat([pool.table, torch.full((1024, 3), -1, dtype=torch.int32)], 1)
    cache = pool.to_cache()
    src, dst = list(range(512)), list(range(512, 1024))
    pool.fork(src, dst)
    cache.fork(ints(src), ints(dst))
    order = torch.randperm(1024, generator=generator(6)).tolist()
    counts = [(3 * i) % 20 for i in range(1024)]
    assert pool.reserve(order, counts)
    cache.reserve(ints(order), ints(counts))
    cache.check()
    pool.same_as(cache)
    keep = [list(range(0, c, 2)) for c in counts]
    padded = torch.zeros((1024, 10), dtype=torch.int32)
    for i, k in enumerate(keep):
        padded[i, :len(k)] = torch.tensor(k, dtype=torch.int32)
    pool.compact(order, keep)
    cache.compact(ints(order), ints([len(k) for k in keep]), padded.cuda())
    cache.check()
    pool.same_as(cache)
    cut = [int(pool.lengths[s]) * (i % 4) // 4 for i, s in enumerate(order)]
    pool.free(order, cut)
    cache.free(ints(order), ints(cut))
    cache.check()
    pool.same_as(cache)


def test_a_pool_of_hundreds_of_thousands_of_pages():
    """Copies whose bitmaps are larger than a CTA's default shared memory, and
    reserves whose free pages are far apart."""
    import tile_synchronised_b200 as mk
    n = 200_001
    kv = torch.randint(-2 ** 15, 2 ** 15, (2, 1, n, 1, 16, 64), dtype=torch.int16, device="cuda",
                       generator=torch.Generator("cuda").manual_seed(1))
    refs = torch.ones(n, dtype=torch.int32, device="cuda")
    holes = torch.randperm(n, generator=generator(7))[:300].sort().values
    refs[holes.cuda()] = 0
    cache = mk.PagedCache.over(kv.view(torch.bfloat16), torch.full((20, 15), -1, dtype=torch.int32, device="cuda"),
                               torch.zeros(20, dtype=torch.int32, device="cuda"), refs)
    want = kv.clone()
    pages = torch.randperm(n, generator=generator(8))[:10000].cuda()
    src, dst = pages[:5000], pages[5000:]
    want[:, :, dst] = want[:, :, src]
    cache.copy(src.int(), dst.int())
    cache.check()
    assert torch.equal(kv, want)
    cache.reserve(ints(list(range(20))), ints([16 * 15] * 20))
    cache.check()
    assert torch.equal(cache.table.cpu().flatten(), holes.int())
    assert int(refs.min()) == 1
    with pytest.raises(mk.MkError, match="not enough"):
        cache.free(ints(0))
        cache.reserve(ints(0, 1), ints(16 * 15, 0))
        cache.check()
        cache.lengths[1] = 16 * 14 + 1
        cache.table[1, 14] = -1
        cache.reserve(ints(1), ints(1))
        cache.check()


def test_copies_in_large_pools_at_once():
    """Four threads, each with a pool of its own size and a stream: no call
    changes what another's launch needs."""
    import threading

    import tile_synchronised_b200 as mk
    lib, failed = mk.load(), []

    def work(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                kv = torch.zeros((2, 1, n, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
                kv[:, :, :8] = torch.arange(1, 9, device="cuda")[None, None, :, None, None, None].to(kv.dtype)
                cache = mk.PagedCache.over(kv, ints([[-1]]), ints([0]), torch.zeros(n, dtype=torch.int32, device="cuda"))
                src, dst = ints(list(range(8))), ints(list(range(n - 8, n)))
                args = (cache._ref, cache._ref, src.data_ptr(), dst.data_ptr(), 8, stream.cuda_stream)
                bad = sum(lib.mk_pages_copy(*args) != 0 for _ in range(10000))
                cache.check()
                assert bad == 0, f"{bad} calls failed"
                assert torch.equal(kv[:, :, n - 8:], kv[:, :, :8])
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in (1 << 19, 200_000, 400_000, 250_000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


# ------------------------------------------------------------------ norm + rotation + append
ROPE = [(8, 149 + (i % 3), *heads, d, dtype, src, bool(i & 1), bool(i & 2))
        for i, (d, dtype, src, heads) in enumerate(
            (d, dtype, src, heads) for d, heads in ((64, (5, 3)), (128, (32, 8)), (256, (20, 8)))
            for dtype in (torch.bfloat16, torch.float16) for src in (torch.float32, dtype))]
ROPE.append((600, 2, 2, 1, 64, torch.bfloat16, torch.float32, True, False))  # fewer tokens than a CTA takes


@pytest.mark.parametrize("n,T,nq,nkv,d,dtype,src,norm,tree", ROPE)
def test_four_tokens_a_cta(n, T, nq, nkv, d, dtype, src, norm, tree):
    import tile_synchronised_b200 as mk
    assert n * T >= 8 * sms()
    g = generator(91)
    lengths = [(17 * i) % 90 for i in range(n)]
    new = [max(0, T - i % 7) for i in range(n)]  # ends inside a CTA's tokens
    pool = filled(lengths, [T] * n, nkv=nkv, d=d, dtype=dtype, seed=92, poison=False)
    qkv = (torch.randn((n, T, (nq + 2 * nkv) * d), generator=g) * 2).to(src)
    gains = [(1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2)] if norm else [None, None]
    depth = None
    if tree:
        depth = torch.stack([visible(random_tree(T, 40 + i)).sum(1).int() - 1 for i in range(n)])
    cache = pool.to_cache()
    seqs = torch.randperm(n, generator=g).tolist()
    room = [min(new[i], T) for i in range(n)]
    q0 = torch.full((n, T, nq, d), 7.0, dtype=dtype)
    q = mk.qk_norm_rope(qkv.cuda(), cache, 0, ints(seqs), nq, 500000.0, *(None if x is None else x.cuda() for x in gains),
                        eps=1e-6, n_new=ints(room), depth=None if depth is None else depth.cuda(), out=q0.cuda())
    cache.check()
    ref, bound, kv = rope_reference(pool, 0, qkv, nq, 500000.0, *gains, 1e-6, seqs, room, depth, q0)
    assert ((q.cpu().double() - ref).abs() <= bound).all()
    got = cache.kv.cpu()
    for (i, t), (k, v, kb) in kv.items():
        page, off = pool.at(seqs[i], lengths[seqs[i]] + t)
        assert ((got[0, 0, page, :, off].double() - k).abs() <= kb).all()
        assert torch.equal(got[1, 0, page, :, off], v.to(dtype))
        got[:, 0, page, :, off] = pool.kv[:, 0, page, :, off]
    assert torch.equal(got, pool.kv)  # nothing else was written
