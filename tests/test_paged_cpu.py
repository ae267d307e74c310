"""Host-side checks of the paged-cache entry points: refusals before any
launch, the tree mask, and the plain implementations the GPU tests use."""
import ctypes as C
import os
import subprocess
import sys

import pytest
import torch

import tile_synchronised_b200 as mk
from paged_common import Pool, filled, pack_bits, random_tree, tree_reference, visible
from tile_synchronised_b200 import _lib

OK, INVALID, UNSUPPORTED = _lib.MK_OK, _lib.MK_ERR_INVALID, _lib.MK_ERR_UNSUPPORTED
PTR = C.c_void_p(4096)


def pages(**kw):
    v = dict(n_layers=2, n_kv_heads=2, head_dim=64, page_size=16, n_pages=8, max_seqs=4, max_pages=3, dtype=0,
             kv=4096, table=4096, lengths=4096, refs=4096, state=4096)
    v.update(kw)
    return C.byref(_lib.MkPages(*[v[f] for f, _ in _lib.MkPages._fields_]))


def reason():
    return _lib.load().mk_last_error(None).decode()


BAD_POOLS = [(dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(state=None), INVALID),
             (dict(kv=4104), INVALID), (dict(lengths=4097), INVALID), (dict(dtype=2), UNSUPPORTED),
             (dict(dtype=-1), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
             (dict(page_size=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_pages=(1 << 19) + 1), INVALID),
             (dict(max_seqs=0), INVALID), (dict(max_seqs=1025), INVALID), (dict(max_pages=0), INVALID),
             (dict(n_layers=0), INVALID), (dict(n_kv_heads=0), INVALID),
             (dict(page_size=1 << 16, max_pages=1 << 15), INVALID)]


@pytest.mark.parametrize("kw,status", BAD_POOLS, ids=[str(k) for k, _ in BAD_POOLS])
def test_every_call_refuses_a_bad_pool(kw, status):
    lib = _lib.load()
    p = pages(**kw)
    assert lib.mk_pages_reserve(p, PTR, PTR, 1, None) == status and reason().startswith("pages_reserve")
    assert lib.mk_pages_fork(p, PTR, PTR, 1, None) == status
    assert lib.mk_pages_compact(p, PTR, PTR, None, 0, 1, None) == status
    assert lib.mk_pages_free(p, PTR, None, 1, None) == status
    assert lib.mk_pages_copy(p, pages(), PTR, PTR, 1, None) == status
    assert lib.mk_pages_copy(pages(), p, PTR, PTR, 1, None) == status
    assert lib.mk_pages_status(p, None) == status
    assert lib.mk_qk_norm_rope(p, 0, PTR, 2, 1024, 1, 1, 4, PTR, None, None, None, None, 0.0, 1e4, PTR, 256,
                               None) == status
    assert lib.mk_attention_tree(p, 0, PTR, 256, 1, 1, 4, PTR, None, None, PTR, 256, PTR, 1 << 30, None) == status


def test_null_pool():
    lib = _lib.load()
    assert lib.mk_pages_reserve(None, PTR, PTR, 1, None) == INVALID and "null" in reason()


def test_lists_are_checked_and_empty_ones_do_nothing():
    lib, p = _lib.load(), pages()
    for f in (lib.mk_pages_reserve, lib.mk_pages_fork):
        assert f(p, PTR, PTR, 5, None) == INVALID  # more entries than sequences
        assert f(p, PTR, PTR, -1, None) == INVALID
        assert f(p, None, PTR, 1, None) == INVALID
        assert f(p, PTR, None, 1, None) == INVALID
        assert f(p, None, None, 0, None) == OK
    assert lib.mk_pages_free(p, None, None, 1, None) == INVALID
    assert lib.mk_pages_free(p, None, None, 0, None) == OK
    assert lib.mk_pages_compact(p, PTR, None, PTR, 4, 1, None) == INVALID
    assert lib.mk_pages_compact(p, PTR, PTR, PTR, 0, 1, None) == INVALID
    assert lib.mk_pages_copy(p, p, PTR, PTR, 9, None) == INVALID
    assert lib.mk_pages_copy(p, p, PTR, None, 1, None) == INVALID
    assert lib.mk_pages_copy(p, p, None, None, 0, None) == OK
    for other in (dict(n_layers=1), dict(page_size=32), dict(head_dim=128), dict(dtype=1), dict(n_kv_heads=1)):
        assert lib.mk_pages_copy(p, pages(**other), PTR, PTR, 1, None) == INVALID and "same shape" in reason()


def test_qk_norm_rope_refusals():
    lib, p = _lib.load(), pages()

    def call(layer=0, qkv=PTR, dt=2, qs=512, n=1, T=1, nq=4, seqs=PTR, g=None, eps=1e-6, theta=1e4, q=PTR, os=256):
        return lib.mk_qk_norm_rope(p, layer, qkv, dt, qs, n, T, nq, seqs, None, None, g, None, eps, theta, q, os, None)

    for kw in (dict(layer=-1), dict(layer=2), dict(qkv=None), dict(q=None), dict(seqs=None), dict(qs=511), dict(qs=504),
               dict(qs=516), dict(os=255), dict(os=252), dict(n=5), dict(n=-1), dict(T=0), dict(nq=0),
               dict(theta=0.0), dict(theta=float("nan")), dict(eps=-1.0), dict(eps=float("nan")),
               dict(qkv=C.c_void_p(4100)), dict(q=C.c_void_p(4104)), dict(g=C.c_void_p(4098))):
        assert call(**kw) == INVALID, kw
    assert call(dt=1) == UNSUPPORTED and call(dt=7) == UNSUPPORTED
    assert call(n=0) == OK


def test_attention_tree_refusals():
    lib, p = _lib.load(), pages()

    def call(layer=0, q=PTR, qs=256, n=1, T=1, nq=4, seqs=PTR, out=PTR, os=256, scratch=PTR, sb=1 << 30):
        return lib.mk_attention_tree(p, layer, q, qs, n, T, nq, seqs, None, None, out, os, scratch, sb, None)

    for kw in (dict(layer=-1), dict(layer=2), dict(q=None), dict(out=None), dict(seqs=None), dict(scratch=None),
               dict(qs=255), dict(qs=260), dict(os=248), dict(n=1025), dict(n=-1), dict(T=0), dict(nq=3), dict(nq=0),
               dict(T=1 << 24), dict(sb=16), dict(q=C.c_void_p(4104)), dict(out=C.c_void_p(4104)),
               dict(scratch=C.c_void_p(4104))):
        assert call(**kw) == INVALID, kw
    assert call(n=0) == OK
    assert lib.mk_attention_tree_scratch_bytes(0, 4, 2, 64) == 0
    assert lib.mk_attention_tree_scratch_bytes(1, 5, 2, 64) == 0
    small, large = (lib.mk_attention_tree_scratch_bytes(T, 4, 2, 64) for T in (1, 1000))
    assert 0 < small < large == lib.mk_attention_tree_scratch_bytes(64, 4, 2, 64) * (large // lib.mk_attention_tree_scratch_bytes(64, 4, 2, 64))


def test_python_cache_refuses_wrong_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        mk.PagedCache.over(torch.zeros((2, 1, 4, 1, 16, 64), dtype=torch.bfloat16), torch.zeros((1, 4)),
                           torch.zeros(1), torch.zeros(4))


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 70])
def test_tree_mask_is_the_ancestor_relation(T):
    parents = [random_tree(T, s) for s in range(3)]
    got = mk.tree_mask(torch.tensor(parents))
    assert got.dtype == torch.int32 and got.shape == (3, T, (T + 31) // 32)
    assert torch.equal(got, pack_bits(torch.stack([visible(p) for p in parents])))


def test_plain_pool_rules():
    pool = filled([21, 5], [0, 0], extra=2, spare=5, poison=False)
    a = pool.clone()
    pool.fork([0], [2])
    assert pool.refs.sum() == a.refs.sum() + 2
    assert pool.reserve([2, 0], [2, 2])  # the fork copies its last page, the parent keeps it
    assert int(pool.table[2, 0]) == int(pool.table[0, 0]) and int(pool.table[2, 1]) != int(pool.table[0, 1])
    assert int(pool.table[0, 1]) == int(a.table[0, 1])
    assert torch.equal(pool.rows(0, 0, 2, 21), a.rows(0, 0, 0, 21))
    pool.compact([2], [[1]])
    assert torch.equal(pool.rows(1, 0, 2, 22)[:, :21], a.rows(1, 0, 0, 21))
    full = pool.clone()
    full.refs += 1
    assert not full.reserve([1], [12]) and torch.equal(full.table, pool.table)
    pool.free([0, 1, 2])
    assert int(pool.refs.sum()) == 0


def test_plain_attention_rules():
    """One visible token returns its V; a row that sees nothing is zero."""
    pool = filled([0], [3])
    q = torch.randn((1, 3, 4, 64)).to(torch.bfloat16)
    seen = torch.eye(3, dtype=torch.bool)[None].clone()
    seen[0, 2, 2] = False
    ref, _ = tree_reference(pool, 0, q, [0], [3], seen, torch.zeros_like(q))
    for t in range(2):
        assert torch.equal(ref[0, t, 2], pool.rows(1, 0, 0, 3)[1, t].double())
    assert (ref[0, 2] == 0).all()


def test_pool_class_clone_is_independent():
    p = Pool(1, 1, 64, 16, 2, 1, 2)
    q = p.clone()
    q.kv.zero_()
    assert p.kv.abs().sum() > 0


def test_the_wait_hook_checks_its_argument():
    lib = _lib.load()
    assert lib.mk_debug_attention_tree_wait(0, 2) == INVALID
    assert lib.mk_debug_attention_tree_wait(0, 0) == OK


@pytest.mark.parametrize("parents", [[[-1, 1]], [[-1, 2]], [[0, 0]], [[-1, 0, 1], [-1, 0, -2]], [[-1, 0, 10 ** 6]]])
def test_tree_mask_refuses_parents_that_do_not_come_first(parents):
    with pytest.raises(ValueError, match="smaller index"):
        mk.tree_mask(torch.tensor(parents))
    for wrong in (torch.tensor([-1, 0]), torch.tensor([[-1.0, 0.0]])):
        with pytest.raises(ValueError, match="integers"):
            mk.tree_mask(wrong)


def test_the_package_imports_without_cuda_in_torch():
    """A torch built without CUDA lacks the private names that shorten a call."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import tile_synchronised_b200 as mk\n"
            "print(mk.tree_mask(torch.tensor([[-1, 0, 0]])).tolist())\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.strip() == "[[[1], [3], [5]]]"


def test_copies_between_overlapping_pools_are_refused():
    """2 layers x 8 pages x 2 heads x 16 x 64 values: 128 KiB of K and V."""
    lib = _lib.load()
    size = 2 * 2 * 8 * 2 * 16 * 64 * 2
    at = 1 << 20
    a = pages(kv=at)
    for kv, n in ((at + 16, 8), (at + size - 16, 8), (at - 16, 8), (at - size // 2 + 16, 4), (at, 7), (at, 9)):
        for dst, src in ((a, pages(kv=kv, n_pages=n)), (pages(kv=kv, n_pages=n), a)):
            assert lib.mk_pages_copy(dst, src, None, None, 0, None) == INVALID and "overlap" in reason()
    for kv, n in ((at, 8), (at + size, 8), (at - size // 2, 4)):  # the same pool, and neighbours
        assert lib.mk_pages_copy(a, pages(kv=kv, n_pages=n), None, None, 0, None) == OK


def test_outputs_that_overlap_inputs_are_refused():
    """No such call gets as far as a launch."""
    lib, p = _lib.load(), pages()
    at = 1 << 24

    def rope(qkv, dt, qs, q, os, n=2, T=3):
        return lib.mk_qk_norm_rope(p, 0, C.c_void_p(qkv), dt, qs, n, T, 4, PTR, None, None, None, None, 1e-6, 1e4,
                                   C.c_void_p(q), os, None)

    # rows of 8 heads of 64: 2048 bytes in fp32, 1024 in 16 bits; q rows of 4: 512
    for args in ((at, 2, 512, at, 256), (at, 2, 512, at + 2032, 256), (at, 2, 512, at + 6 * 2048 - 16, 256),
                 (at, 2, 512, at - 6 * 512 + 16, 256), (at, 2, 512, at, 1024), (at, 0, 512, at, 256),
                 (at, 0, 512, at + 16, 512), (at, 0, 512, at + 512, 512), (at, 0, 1024, at + 1536 + 16, 1024),
                 (at, 0, 1024, at - 496, 1024)):
        assert rope(*args) == INVALID and "overlap" in reason(), args

    def attend(q, qs, out, os, scratch=1 << 28, n=2, T=3):
        return lib.mk_attention_tree(p, 0, C.c_void_p(q), qs, n, T, 4, PTR, None, None, C.c_void_p(out), os,
                                     C.c_void_p(scratch), 1 << 26, None)

    for args in ((at, 256, at, 256), (at, 256, at + 16, 256), (at, 256, at + 6 * 512 - 16, 256),
                 (at, 256, at - 6 * 512 + 16, 256), (at, 512, at + 496, 512), (at, 512, at + 528, 512),
                 (at, 512, at + 512, 256), (at + 2048 - 496, 512, at, 512)):
        assert attend(*args) == INVALID and "out must not overlap q" in reason(), args
    for scratch in (at, at + 5 * 512, at - 16, (1 << 25), (1 << 25) + 5 * 512):
        assert attend(at, 256, 1 << 25, 256, scratch) == INVALID and "scratch must not" in reason(), scratch
