"""A KV cache in pages and the operators over it: PagedCache (reserve, fork,
compact, free, copy), qk_norm_rope and attention_tree.

One step with drafted tokens:

    cache.reserve(seqs, counts)                                  # room for T new tokens
    for layer in ...:
        q = qk_norm_rope(qkv, cache, layer, seqs, n_heads, theta, ..., depth=depth)
        o = attention_tree(q, cache, layer, seqs, mask=mask)
    cache.compact(seqs, n_keep, keep)                            # the accepted path
    cache.check()                                                # errors seen on the device

Lists (seqs, counts, ...) are int32 CUDA tensors; they are read when the
kernels run, so a captured step follows their contents.

Calls run on the current stream, or on `stream`.  There they are not ordered
with what the current stream does, and a result that they allocate is that
stream's; the tensors that they are given may be dropped at once.
"""
from __future__ import annotations

import ctypes as C

import torch

from ._lib import MK_BF16, MK_FP16, MK_FP32, MkPages, check, load

_TYPES = {torch.bfloat16: MK_BF16, torch.float16: MK_FP16, torch.float32: MK_FP32}


def _public_raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# The same without 2 us of checks and objects a call, where this torch has them (one built without CUDA does not).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_INT32 = torch.int32


def _elsewhere(device: torch.device, stream) -> bool:
    """Does a call have to switch to another device or stream first?"""
    if stream is None:
        return _get_device() != device.index
    if stream.device != device:
        raise ValueError(f"the stream must be one of {device}")
    return True


def _on(device: torch.device, stream):
    """The context of such a call: allocations made inside belong to its stream."""
    return torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream)


def _lend(stream, cache: "PagedCache", *tensors) -> None:
    """For a call on a stream that it was given: the memory it uses stays what
    it is until that stream is done with it, also if the caller drops it."""
    if stream is not None:
        for t in (cache.kv, cache.table, cache.lengths, cache.refs, cache._state, *tensors):
            if t is not None:
                t.record_stream(stream)


def _ints(t, name: str, shape: tuple, index: int):
    """The address of an int32 list of that shape on CUDA device `index` (None stays None)."""
    if t is None:
        return None
    if t.dtype is not _INT32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on cuda:{index}")
    return t.data_ptr()


class PagedCache:
    """A pool of pages and the sequences in it (mk_pages).

    kv [2, n_layers, n_pages, n_kv_heads, page_size, head_dim] (K, then V;
    bf16 or fp16), table int32 [max_seqs, max_pages] (-1: no page), lengths
    int32 [max_seqs] (committed positions), refs int32 [n_pages] (sequences
    that hold the page).  Sequences are rows of the table.  Operations on one
    cache must be ordered (one stream, or events between)."""

    def __init__(self, n_layers: int, n_kv_heads: int, head_dim: int, page_size: int, n_pages: int, max_seqs: int,
                 max_pages: int, dtype: torch.dtype = torch.bfloat16, device=None):
        dev = torch.device("cuda" if device is None else device)
        self._bind(torch.empty((2, n_layers, n_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=dev),
                   torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=dev),
                   torch.zeros(max_seqs, dtype=torch.int32, device=dev),
                   torch.zeros(n_pages, dtype=torch.int32, device=dev))

    @classmethod
    def over(cls, kv: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor) -> "PagedCache":
        """A cache over tensors of the caller (used in place)."""
        self = cls.__new__(cls)
        self._bind(kv, table, lengths, refs)
        return self

    @classmethod
    def of_model(cls, model) -> "PagedCache":
        """A Model's (or TcDecoder's) contiguous cache as one page per sequence,
        at the model's position."""
        s = model.shape
        kv = model.kv.view(torch.bfloat16).view(2, s.n_layers, model.batch, s.n_kv_heads, model.max_seq, s.head_dim)
        dev = kv.device
        return cls.over(kv, torch.arange(model.batch, dtype=torch.int32, device=dev).view(-1, 1),
                        torch.full((model.batch,), model.position, dtype=torch.int32, device=dev),
                        torch.ones(model.batch, dtype=torch.int32, device=dev))

    def _bind(self, kv, table, lengths, refs):
        if kv.dim() != 6 or kv.shape[0] != 2 or kv.dtype not in (torch.bfloat16, torch.float16) or not kv.is_cuda \
                or not kv.is_contiguous():
            raise ValueError("kv must be a contiguous bf16 or fp16 CUDA tensor [2, n_layers, n_pages, n_kv_heads, "
                             "page_size, head_dim]")
        _, self.n_layers, self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = kv.shape
        if table.dim() != 2:
            raise ValueError("table must be [max_seqs, max_pages]")
        self.max_seqs, self.max_pages = table.shape
        self.device, self.dtype = kv.device, kv.dtype
        self._index = kv.device.index
        _ints(table, "table", (self.max_seqs, self.max_pages), self._index)
        _ints(lengths, "lengths", (self.max_seqs,), self._index)
        _ints(refs, "refs", (self.n_pages,), self._index)
        self.kv, self.table, self.lengths, self.refs = kv, table, lengths, refs
        self.lib = load()
        self._state = torch.zeros(self.lib.mk_pages_state_bytes() // 4, dtype=torch.int32, device=kv.device)
        self._struct = MkPages(self.n_layers, self.n_kv_heads, self.head_dim, self.page_size, self.n_pages,
                               self.max_seqs, self.max_pages, _TYPES[kv.dtype], kv.data_ptr(), table.data_ptr(),
                               lengths.data_ptr(), refs.data_ptr(), self._state.data_ptr())
        self._ref = C.byref(self._struct)
        self._scratch = {}

    # ---------------------------------------------------------------- calls
    def _call(self, name: str, stream, *args) -> None:
        if _elsewhere(self.device, stream):
            with _on(self.device, stream):
                return self._call(name, None, *args)
        st = getattr(self.lib, name)(self._ref, *args, _raw_stream(self._index))
        if st:
            check(st, None, name, op=True)

    def _scratch_bytes(self, T: int, n_heads: int) -> int:
        """Scratch of attention_tree, a function of these sizes alone."""
        need = self._scratch.get((T, n_heads))
        if need is None:
            need = self.lib.mk_attention_tree_scratch_bytes(T, n_heads, self.n_kv_heads, self.head_dim)
            self._scratch[T, n_heads] = need
        return need

    def _list(self, name: str, t: torch.Tensor, n: int) -> int:
        return _ints(t, name, (n,), self._index)

    def reserve(self, seqs: torch.Tensor, counts: torch.Tensor, stream=None) -> None:
        """Room for counts[i] new tokens of sequence seqs[i], in pages it holds alone."""
        n = seqs.numel()
        self._call("mk_pages_reserve", stream, self._list("seqs", seqs, n), self._list("counts", counts, n), n)
        _lend(stream, self, seqs, counts)

    def fork(self, src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
        """Empty sequence dst[i] shares the pages of src[i]'s committed positions."""
        n = src.numel()
        self._call("mk_pages_fork", stream, self._list("src", src, n), self._list("dst", dst, n), n)
        _lend(stream, self, src, dst)

    def compact(self, seqs: torch.Tensor, n_keep: torch.Tensor, keep: torch.Tensor | None = None, stream=None) -> None:
        """Commit n_keep[i] new tokens of sequence seqs[i]: those at the
        ascending indexes keep[i], or the first ones."""
        n = seqs.numel()
        width = 0 if keep is None else keep.shape[-1]
        self._call("mk_pages_compact", stream, self._list("seqs", seqs, n), self._list("n_keep", n_keep, n),
                   _ints(keep, "keep", (n, width), self._index), width, n)
        _lend(stream, self, seqs, n_keep, keep)

    def free(self, seqs: torch.Tensor, lengths: torch.Tensor | None = None, stream=None) -> None:
        """Cut sequence seqs[i] to lengths[i] positions (0 by default) and give up the pages behind."""
        n = seqs.numel()
        self._call("mk_pages_free", stream, self._list("seqs", seqs, n),
                   None if lengths is None else self._list("lengths", lengths, n), n)
        _lend(stream, self, seqs, lengths)

    def copy(self, src_pages: torch.Tensor, dst_pages: torch.Tensor, source: "PagedCache | None" = None,
             stream=None) -> None:
        """Page dst_pages[k] = page src_pages[k] of `source` (this cache by
        default; one whose kv has no byte in common with this one's), in every layer."""
        n = src_pages.numel()
        src = self if source is None else source
        if src.device != self.device:
            raise ValueError("the two caches must be on the same device")
        self._call("mk_pages_copy", stream, src._ref, self._list("src_pages", src_pages, n),
                   self._list("dst_pages", dst_pages, n), n)
        _lend(stream, self, src_pages, dst_pages, src.kv, src._state)

    def check(self, stream=None) -> None:
        """Raise MkError for the first error the cache's kernels met since the
        last check (waits for the stream)."""
        self._call("mk_pages_status", stream)


def tree_mask(parents: torch.Tensor) -> torch.Tensor:
    """The mask of attention_tree (int32 bits [n, T, (T + 31) // 32]) of trees
    given by parents [n, T]: the index of each token's parent, smaller than its
    own, or -1 for a child of the last committed token.  Other parents are
    refused on the CPU; on a GPU, where looking would wait for it, they count
    as -1."""
    if parents.dim() != 2 or parents.is_floating_point():
        raise ValueError("parents must be integers [n, T]")
    n, T = parents.shape
    p = parents.long()
    good = (p >= -1) & (p < torch.arange(T, device=p.device))
    if not p.is_cuda and not good.all():
        raise ValueError("a parent must be -1 or a smaller index than its child's")
    p = torch.where(good, p, -1)  # no index leaves its row
    seen = torch.eye(T, dtype=torch.bool, device=p.device).repeat(n, 1, 1)
    rows = torch.arange(n, device=p.device)
    for t in range(1, T):  # a row's parent comes before it and is complete
        up = p[:, t].clamp_min(0)
        seen[:, t] |= seen[rows, up] & (p[:, t] >= 0)[:, None]
    words = (T + 31) // 32
    bits = torch.zeros((n, T, words * 32), dtype=torch.int64, device=p.device)
    bits[:, :, :T] = seen
    packed = (bits.view(n, T, words, 32) << torch.arange(32, device=p.device)).sum(-1)
    return torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)


def _tokens(x: torch.Tensor, name: str, shape: tuple, dtypes, index: int, width: int) -> int:
    """Checks a [n, T, ...] tensor whose tokens are dense rows of `width` values
    at one stride; returns that stride in elements."""
    if x.shape != shape or x.dtype not in dtypes or x.get_device() != index:
        raise ValueError(f"{name} must be {list(shape)} of {' or '.join(str(t) for t in dtypes)} on cuda:{index}")
    if x.is_contiguous():
        return width
    n, T = shape[:2]
    width = 1
    for k in range(x.dim() - 1, 1, -1):
        if x.shape[k] != 1 and x.stride(k) != width:
            raise ValueError(f"{name}: the values of a token must be contiguous")
        width *= x.shape[k]
    step = x.stride(1) if T > 1 else x.stride(0) if n > 1 else width
    if n > 1 and T > 1 and x.stride(0) != T * step:
        raise ValueError(f"{name}: tokens must be at one stride")
    return step


def qk_norm_rope(qkv: torch.Tensor, cache: PagedCache, layer: int, seqs: torch.Tensor, n_heads: int, theta: float,
                 q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None, eps: float = 1e-6,
                 n_new: torch.Tensor | None = None, depth: torch.Tensor | None = None,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Per-head RMSNorm of q and k (with gains), rotation by each token's
    position, K and V into the cache: qkv [n, T, (n_heads + 2 n_kv_heads) *
    head_dim] (fp32 or the cache's type; token t of entry i is new token t of
    sequence seqs[i], rotated by length + depth[i, t], depth = t by default)
    -> q [n, T, n_heads, head_dim] in the cache's type.  Tokens t >= n_new[i]
    are left out."""
    if qkv.dim() != 3:
        raise ValueError("qkv must be [n, T, (n_heads + 2 n_kv_heads) * head_dim]")
    n, T, _ = qkv.shape
    d, dev, at = cache.head_dim, cache.device, cache._index
    width = (n_heads + 2 * cache.n_kv_heads) * d
    stride = _tokens(qkv, "qkv", (n, T, width), (torch.float32, cache.dtype), at, width)
    for g in (q_gain, k_gain):
        if g is not None and (g.dtype is not torch.bfloat16 or g.shape != (d,) or g.get_device() != at
                              or not g.is_contiguous()):
            raise ValueError("gains must be contiguous bf16 [head_dim]")
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            got = qk_norm_rope(qkv, cache, layer, seqs, n_heads, theta, q_gain, k_gain, eps, n_new, depth, out)
        _lend(stream, cache, qkv, seqs, q_gain, k_gain, n_new, depth, out)
        return got
    if out is None:
        out = torch.empty((n, T, n_heads, d), dtype=cache.dtype, device=dev)
    st = cache.lib.mk_qk_norm_rope(
        cache._ref, layer, qkv.data_ptr(), _TYPES[qkv.dtype], stride, n, T, n_heads, _ints(seqs, "seqs", (n,), at),
        _ints(n_new, "n_new", (n,), at), _ints(depth, "depth", (n, T), at),
        None if q_gain is None else q_gain.data_ptr(), None if k_gain is None else k_gain.data_ptr(), eps, theta,
        out.data_ptr(), _tokens(out, "out", (n, T, n_heads, d), (cache.dtype,), at, n_heads * d), _raw_stream(at))
    if st:
        check(st, None, "mk_qk_norm_rope", op=True)
    return out


def attention_tree(q: torch.Tensor, cache: PagedCache, layer: int, seqs: torch.Tensor,
                   n_new: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, scratch: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Attention of the new tokens q [n, T, n_heads, head_dim] (the cache's
    type) over the pages of sequences seqs: token t < n_new[i] sees the
    committed positions and the new tokens whose bit is set in its row of mask
    (int32 bits [n, T, (T + 31) // 32], see tree_mask), by default those up to
    itself (T = 1: a decode step).  Returns `out` (like q); its rows t >=
    n_new[i] are not written, and those that see a position without a page are
    NaN."""
    if q.dim() != 4:
        raise ValueError("q must be [n, T, n_heads, head_dim]")
    n, T, nq, d = q.shape
    dev, at = cache.device, cache._index
    shape, types = (n, T, nq, cache.head_dim), (cache.dtype,)
    stride = _tokens(q, "q", shape, types, at, nq * d)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            got = attention_tree(q, cache, layer, seqs, n_new, mask, out, scratch)
        _lend(stream, cache, q, seqs, n_new, mask, out, scratch)
        return got
    if out is None:
        out = torch.empty(shape, dtype=cache.dtype, device=dev)
    elif out.data_ptr() == q.data_ptr():
        raise ValueError("out must not be q")
    if scratch is None:
        scratch = cache._state.new_empty(cache._scratch_bytes(T, nq) // 4)
    elif scratch.get_device() != at or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous tensor on the cache's device")
    st = cache.lib.mk_attention_tree(
        cache._ref, layer, q.data_ptr(), stride, n, T, nq, _ints(seqs, "seqs", (n,), at),
        _ints(n_new, "n_new", (n,), at), _ints(mask, "mask", (n, T, (T + 31) // 32), at), out.data_ptr(),
        _tokens(out, "out", shape, types, at, nq * d), scratch.data_ptr(), scratch.nbytes, _raw_stream(at))
    if st:
        check(st, None, "mk_attention_tree", op=True)
    return out
