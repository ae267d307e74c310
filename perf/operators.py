"""Cases of the paged-cache operators: per-head norm + rotation + append, tree
attention over the pages, and page management.

Every case is one pass of one operator as a serving loop calls it.  With
``own`` false, ``run`` computes it from elementary torch operations in 32 bits
(angles in 64); with ``own`` true it calls ``tile_synchronised_b200``.

A paged cache is kv [2, layers, pages, kv_heads, page_size, head_dim] (K, then
V), a page table int32 [seqs, max_pages] (-1: none), lengths int32 [seqs] (the
committed positions) and refs int32 [pages] (sequences that hold the page).
New tokens of a step sit at positions length, length + 1, ... of their
sequence; pages are always allocated lowest index first.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_DEV = "cuda"

# Head layouts: Llama-3.2-1B, Llama-3.1-8B / Qwen3-8B, and the others of the attention tests.
_HEADS = [(32, 8, 64), (32, 8, 128), (12, 4, 256), (8, 1, 128), (8, 8, 128), (4, 2, 64), (16, 8, 128), (14, 2, 64)]

# A drawn case costs no more than these (the largest listed cases).
_MAX_KV = 16 * 16384 * 8 * 128
_MAX_FLOPS = 4.0 * 16 * 64 * 32 * 128 * 12000
_MAX_ROPE = 8 * 1024 * 48 * 128
_MAX_POOL = 200 * 2 ** 20


def listed():
    return [
        # --- attention of the new tokens over the pages
        # one user, the first draft of a small tree behind a 1k prompt: the latency of one call
        dict(name="tree_first", op="tree", nq=32, nkv=8, d=64, dtype="bf16", n=1, T=13, lo=1025, hi=1280, page=16,
             mask="tree"),
        # the single-token step of a batch whose sequences have any length up to 16k
        dict(name="decode_ragged", op="tree", nq=32, nkv=8, d=128, dtype="bf16", n=16, T=1, lo=0, hi=16384, page=64,
             mask="none"),
        # a batch of 8 verifying ragged trees of up to 27 tokens
        dict(name="tree_mid", op="tree", nq=32, nkv=8, d=128, dtype="bf16", n=8, T=27, lo=512, hi=4096, page=32,
             mask="tree"),
        # wide heads, three query heads per KV head, fp16 cache, small pages
        dict(name="tree_wide", op="tree", nq=12, nkv=4, d=256, dtype="fp16", n=3, T=31, lo=1000, hi=2100, page=16,
             mask="tree"),
        # a chunk of a prompt behind a cached prefix: causal, many rows per head
        dict(name="chunk_causal", op="tree", nq=32, nkv=8, d=64, dtype="bf16", n=2, T=500, lo=0, hi=2000, page=64,
             mask="none"),
        # the long end: 64 drafted tokens for each of 16 sequences at 8k to 16k
        dict(name="tree_long", op="tree", nq=32, nkv=8, d=128, dtype="bf16", n=16, T=64, lo=8000, hi=16000, page=128,
             mask="tree"),
        # --- norm + rotation + append
        # one token of each of 16 sequences
        dict(name="rope_step", op="rope", nq=32, nkv=8, d=128, dtype="bf16", src="fp32", norm=True, n=16, T=1, lo=1,
             hi=16000, page=64, theta=1000000.0),
        # trees of 61 tokens, fp16 in and out, no norm
        dict(name="rope_tree", op="rope", nq=12, nkv=4, d=256, dtype="fp16", src="16", norm=False, n=5, T=61, lo=100,
             hi=2100, page=16, theta=500000.0),
        # prompts: 8 x 1024 tokens from a projection's fp32 output
        dict(name="rope_prompt", op="rope", nq=32, nkv=8, d=128, dtype="bf16", src="fp32", norm=True, n=8, T=1024,
             lo=0, hi=900, page=64, theta=1000000.0),
        # --- pages
        # two users forked once each in a small cache: the latency of the bookkeeping
        dict(name="fork_small", op="fork", layers=2, nkv=2, d=64, dtype="bf16", n=2, beams=1, T=5, lo=10, hi=90,
             page=16),
        # 8 prompts, 3 continuations of each, copy on write of every last page (16 layers)
        dict(name="fork_beams", op="fork", layers=16, nkv=8, d=64, dtype="bf16", n=8, beams=3, T=16, lo=65, hi=639,
             page=64),
        # 16 verified drafts brought over from the drafting pool, the accepted path compacted (32 layers)
        dict(name="accept_batch", op="accept", layers=32, nkv=8, d=128, dtype="bf16", n=16, T=24, lo=1, hi=90,
             page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "rope", "fork", "accept"])
    nq, nkv, d = rng.choice(_HEADS)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "tree":
        T = rng.choice([1, _log_int(rng, 1, 130), _log_int(rng, 1, 500)])
        hi = _log_int(rng, 1, 16384)
        lo = rng.choice([0, hi // 2, hi])
        n = _log_int(rng, 1, 32)
        while n > 1 and (n * (hi + T + page) * nkv * d > _MAX_KV or 4.0 * n * T * nq * d * (hi + T) > _MAX_FLOPS):
            n -= 1
        while T > 1 and 4.0 * n * T * nq * d * (hi + T) > _MAX_FLOPS:
            T //= 2
        return dict(op=op, nq=nq, nkv=nkv, d=d, dtype=dtype, n=n, T=T, lo=lo, hi=hi, page=page,
                    mask=rng.choice(["tree", "none"]) if T > 1 else "none")
    if op == "rope":
        T = rng.choice([1, _log_int(rng, 1, 1024)])
        n = _log_int(rng, 1, 64)
        while n > 1 and n * T * (nq + 2 * nkv) * d > _MAX_ROPE:
            n -= 1
        hi = _log_int(rng, 1, 4096)
        while n > 1 and n * (hi + T + page) * nkv * d > _MAX_POOL // 2:
            n -= 1
        return dict(op=op, nq=nq, nkv=nkv, d=d, dtype=dtype, src=rng.choice(["fp32", "16"]),
                    norm=rng.choice([True, False]), n=n, T=T, lo=rng.choice([0, hi]), hi=hi, page=page,
                    theta=rng.choice([500000.0, 1000000.0]))
    layers = _log_int(rng, 1, 32)
    T = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, 600)
    n = _log_int(rng, 1, 16)
    beams = rng.choice([1, 2, 3, 4])
    each = 2 * layers * nkv * page * d
    pages = lambda: n * ((hi + T) // page + 2) * (1 + (beams if op == "fork" else 1))  # noqa: E731
    while n > 1 and pages() * each > _MAX_POOL:
        n -= 1
    while layers > 1 and pages() * each > _MAX_POOL:
        layers //= 2
        each = 2 * layers * nkv * page * d
    c = dict(op=op, layers=layers, nkv=nkv, d=d, dtype=dtype, n=n, T=T, lo=rng.choice([0, hi // 2, hi]), hi=hi,
             page=page)
    return {**c, "beams": beams} if op == "fork" else c


# ------------------------------------------------------------------ inputs
def _cpu(seed, salt):
    g = torch.Generator()
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _normal(shape, seed, salt, dtype, std=1.0):
    g = torch.Generator(device=_DEV)
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    out = torch.empty(shape, dtype=dtype, device=_DEV)
    flat, step = out.view(-1), 1 << 26
    for a in range(0, flat.numel(), step):
        b = min(a + step, flat.numel())
        flat[a:b] = torch.randn(b - a, generator=g, device=_DEV) * std
    return out


def _lengths(case, seed, n):
    g = _cpu(seed, 1)
    return torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g)


def _pool(case, seed, layers, lengths, room, spare=0, extra_rows=0):
    """A cache whose sequence i holds pages for lengths[i] + room[i] positions
    at shuffled page indexes, sized for the case's longest sequences, with
    `spare` more pages and `extra_rows` empty sequences behind."""
    ps, n = case["page"], len(lengths)
    held = (lengths + room + ps - 1) // ps
    width = (case["hi"] + case["T"] + ps - 1) // ps
    total = n * width + spare
    table = torch.full((n + extra_rows, width), -1, dtype=torch.int32)
    order = torch.randperm(total, generator=_cpu(seed, 2)).to(torch.int32)
    refs = torch.zeros(total, dtype=torch.int32)
    at = 0
    for i in range(n):
        k = int(held[i])
        table[i, :k] = order[at:at + k]
        at += k
    refs[order[:at].long()] = 1
    all_lengths = torch.zeros(n + extra_rows, dtype=torch.int32)
    all_lengths[:n] = lengths
    kv = _normal((2, layers, total, case["nkv"], ps, case["d"]), seed, 3, _DTYPES[case["dtype"]])
    return dict(kv=kv, table=table.to(_DEV), lengths=all_lengths.to(_DEV), refs=refs.to(_DEV))


def _tree(case, seed):
    """Parents of a random tree per sequence (a parent comes before its
    children), its ancestor-or-self bits and each token's depth."""
    n, T = case["n"], case["T"]
    g = _cpu(seed, 4)
    parent = torch.minimum((torch.rand((n, T), generator=g) * (torch.arange(T) + 1)).long(), torch.arange(T)) - 1
    seen = torch.zeros((n, T, T), dtype=torch.bool)
    for t in range(T):
        seen[:, t, t] = True
        rows = torch.nonzero(parent[:, t] >= 0).flatten()
        seen[rows, t] |= seen[rows, parent[rows, t]]
    depth = seen.sum(-1).to(torch.int32) - 1
    words = (T + 31) // 32
    bits = torch.zeros((n, T, words * 32), dtype=torch.int64)
    bits[:, :, :T] = seen
    packed = (bits.view(n, T, words, 32) << torch.arange(32)).sum(-1)
    packed = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
    return packed, depth


def _n_new(case, seed):
    n, T = case["n"], case["T"]
    new = torch.randint((T + 1) // 2, T + 1, (n,), generator=_cpu(seed, 5))
    return new.to(torch.int32)


def prepare(case, seed):
    op, n, T = case["op"], case["n"], case["T"]
    lengths = _lengths(case, seed, n)
    room = torch.full((n,), T)
    ps = case["page"]
    dtype = _DTYPES[case["dtype"]]
    if op == "tree":
        s = _pool(case, seed, 1, lengths, room)
        s["seqs"] = torch.randperm(n, generator=_cpu(seed, 6)).to(torch.int32).to(_DEV)
        s["n_new"] = _n_new(case, seed).to(_DEV)
        s["q"] = _normal((n, T, case["nq"], case["d"]), seed, 7, dtype, 2.0)
        s["out"] = torch.zeros_like(s["q"])
        s["mask"] = _tree(case, seed)[0].to(_DEV) if case["mask"] == "tree" else None
    elif op == "rope":
        s = _pool(case, seed, 1, lengths, room)
        nq, nkv, d = case["nq"], case["nkv"], case["d"]
        s["seqs"] = torch.randperm(n, generator=_cpu(seed, 6)).to(torch.int32).to(_DEV)
        s["n_new"] = _n_new(case, seed).to(_DEV)
        s["qkv"] = _normal((n, T, (nq + 2 * nkv) * d), seed, 7, torch.float32 if case["src"] == "fp32" else dtype, 1.5)
        s["depth"] = _tree(case, seed)[1].to(_DEV) if 1 < T <= 128 else None
        s["q_gain"] = (1 + _normal((d,), seed, 8, torch.float32, 0.1)).bfloat16() if case["norm"] else None
        s["k_gain"] = (1 + _normal((d,), seed, 9, torch.float32, 0.1)).bfloat16() if case["norm"] else None
        s["q"] = torch.zeros((n, T, nq, d), dtype=dtype, device=_DEV)
    elif op == "fork":
        beams = case["beams"]
        grow = (T + ps - 1) // ps + 1
        s = _pool(case, seed, case["layers"], lengths, torch.zeros(n, dtype=torch.long), n * beams * grow, n * beams)
        s["src"] = torch.arange(n, dtype=torch.int32).repeat_interleave(beams).to(_DEV)
        s["dst"] = torch.arange(n, n + n * beams, dtype=torch.int32).to(_DEV)
        s["counts"] = torch.full((n * beams,), T, dtype=torch.int32, device=_DEV)
    else:  # accept
        grow = (lengths + T + ps - 1) // ps - lengths // ps  # pages that the drafted positions touch
        s = _pool(case, seed, case["layers"], lengths, torch.zeros(n, dtype=torch.long))
        free = torch.nonzero(s["refs"].cpu() == 0).flatten().to(torch.int32)
        table, dst, at = s["table"].cpu(), [], 0
        for i in range(n):
            a, k = int(lengths[i]) // ps, int(grow[i])
            old = 1 if int(lengths[i]) % ps else 0
            dst += [int(table[i, a])] * old + free[at:at + k - old].tolist()
            at += k - old
        s["dst_pages"] = torch.tensor(dst, dtype=torch.int32).to(_DEV)
        # the drafting pool's pages of the same positions: the committed part is the same
        m = len(dst)
        s["stage"] = _normal((2, case["layers"], m, case["nkv"], ps, case["d"]), seed, 10, dtype)
        s["src_pages"] = torch.randperm(m, generator=_cpu(seed, 11)).to(torch.int32).to(_DEV)
        at = 0
        for i in range(n):
            used = int(lengths[i]) % ps
            if used:
                s["stage"][:, :, s["src_pages"][at].long(), :, :used] = s["kv"][:, :, dst[at], :, :used]
            at += int(grow[i])
        s["seqs"] = torch.arange(n, dtype=torch.int32).to(_DEV)
        s["counts"] = torch.full((n,), T, dtype=torch.int32, device=_DEV)
        s["base"] = lengths.to(torch.int32).to(_DEV)
        keep = torch.stack([torch.randperm(T, generator=_cpu(seed, 12 + i)) for i in range(n)])
        n_keep = torch.randint(1, T + 1, (n,), generator=_cpu(seed, 5))
        ranked = torch.where(torch.arange(T)[None] < n_keep[:, None], keep, T).sort(dim=1).values
        s["keep"] = torch.where(ranked < T, ranked, 0).to(torch.int32).to(_DEV)
        s["n_keep"] = n_keep.to(torch.int32).to(_DEV)
    s["case"] = dict(case)
    if own:
        import tile_synchronised_b200 as mk
        s["cache"] = mk.PagedCache.over(s["kv"], s["table"], s["lengths"], s["refs"])
        if op == "accept":
            m = s["stage"].shape[2]
            none = torch.full((1, 1), -1, dtype=torch.int32, device=_DEV)
            s["drafts"] = mk.PagedCache.over(s["stage"], none, torch.zeros(1, dtype=torch.int32, device=_DEV),
                                             torch.ones(m, dtype=torch.int32, device=_DEV))
    return s


# ------------------------------------------------------------------ the plain form
def _positions(s):
    """K and V of every listed sequence, [n, kv_heads, positions, head_dim] in
    32 bits, and the sequences' lengths."""
    kv, seqs = s["kv"], s["seqs"].long()
    pages = s["table"][seqs].long().clamp_min(0)
    k, v = (kv[h, 0][pages].float().permute(0, 2, 1, 3, 4).flatten(2, 3) for h in (0, 1))
    return k, v, s["lengths"][seqs].long()


def _plain_tree(s):
    c = s["case"]
    n, T, nq, d = s["q"].shape
    k, v, length = _positions(s)
    nkv, S = k.shape[1], k.shape[2]
    new = s["n_new"].long()
    j = torch.arange(S, device=_DEV)[None, None, :]
    t = torch.arange(T, device=_DEV)[None, :, None]
    u = j - length[:, None, None]  # index among the new tokens
    if s["mask"] is None:
        among = u <= t
    else:
        at = u.clamp(0, T - 1).expand(n, T, S)
        among = (s["mask"].gather(2, at // 32) >> (at % 32).to(torch.int32)) & 1 != 0
    seen = (u < 0) | ((u >= 0) & (u < new[:, None, None]) & among)  # [n, T, S]
    v = torch.where((u < new[:, None, None])[:, 0, None, :, None], v, 0.0)
    q = s["q"].float().view(n, T, nkv, nq // nkv, d).permute(0, 2, 1, 3, 4).reshape(n, nkv, -1, d)
    score = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    score = score.view(n, nkv, T, nq // nkv, S)
    score = torch.where(seen[:, None, :, None, :], score, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == float("-inf"), 0.0, top))
    del score
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, nkv, -1, S) @ v).view(n, nkv, T, nq // nkv, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, T, nq, d)
    live = (torch.arange(T, device=_DEV)[None] < new[:, None])[:, :, None, None]
    s["out"].copy_(torch.where(live, o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _plain_rope(s):
    c = s["case"]
    nq, nkv, d, ps = c["nq"], c["nkv"], c["d"], c["page"]
    n, T = s["qkv"].shape[:2]
    x = s["qkv"].float().view(n, T, nq + 2 * nkv, d)
    seqs = s["seqs"].long()
    length = s["lengths"][seqs].long()
    t = torch.arange(T, device=_DEV)
    depth = t.expand(n, T) if s["depth"] is None else s["depth"].long()
    angle = (length[:, None] + depth).double()[:, :, None] * c["theta"] ** (
        torch.arange(d // 2, device=_DEV, dtype=torch.float64) * (-2.0 / d))
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]

    def rotate(h, gain):
        if gain is not None:
            h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * gain.float()
        a, b = h[..., :d // 2], h[..., d // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(s["q"].dtype)

    live = t[None] < s["n_new"].long()[:, None]
    q = rotate(x[:, :, :nq], s["q_gain"])
    s["q"].copy_(torch.where(live[:, :, None, None], q, s["q"]))
    k, v = rotate(x[:, :, nq:nq + nkv], s["k_gain"]), x[:, :, nq + nkv:].to(s["q"].dtype)
    slot = length[:, None] + t[None]
    page = s["table"][seqs].long().gather(1, slot // ps)[live]
    off = (slot % ps)[live]
    s["kv"][0, 0][page, :, off] = k[live]
    s["kv"][1, 0][page, :, off] = v[live]
    return s["q"], s["kv"]


def _plain_free(s, seqs, lengths):
    ps, seqs = s["kv"].shape[4], seqs.long()
    rows = s["table"][seqs].long()
    drop = (torch.arange(rows.shape[1], device=_DEV)[None] >= ((lengths.long() + ps - 1) // ps)[:, None]) & (rows >= 0)
    s["refs"].index_add_(0, rows[drop], torch.full_like(rows[drop], -1, dtype=torch.int32))
    s["table"][seqs] = torch.where(drop, -1, rows).to(torch.int32)
    s["lengths"][seqs] = lengths


def _plain_fork(s, src, dst):
    ps, src, dst = s["kv"].shape[4], src.long(), dst.long()
    length = s["lengths"][src]
    rows = s["table"][src].long()
    rows = torch.where(torch.arange(rows.shape[1], device=_DEV)[None] < ((length.long() + ps - 1) // ps)[:, None],
                       rows, -1)
    shared = rows[rows >= 0]
    s["refs"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    s["table"][dst] = rows.to(torch.int32)
    s["lengths"][dst] = length


def _plain_reserve(s, seqs, counts):
    ps, seqs = s["kv"].shape[4], seqs.long()
    n = len(seqs)
    length = s["lengths"][seqs].long()
    rows = s["table"][seqs].long()
    col = torch.arange(rows.shape[1], device=_DEV)[None]
    first, last = length // ps, (length + counts.long() + ps - 1) // ps
    missing = (col >= first[:, None]) & (col < last[:, None]) & (rows < 0)
    # a partly filled last page is copied while another sequence still holds it
    partial = (length % ps != 0) & (last > first)
    page = rows.gather(1, first.clamp_max(rows.shape[1] - 1)[:, None])[:, 0].clamp_min(0)
    earlier = ((page[None] == page[:, None]) & partial[None] & partial[:, None]).tril(-1).sum(1)
    copied = partial & (s["refs"][page].long() - earlier > 1)
    take = missing | (copied[:, None] & (col == first[:, None]))
    rank = (take.flatten().cumsum(0) - 1).view(n, -1)
    free = torch.sort((s["refs"] != 0).to(torch.int32), stable=True).indices
    fresh = torch.where(take, free[rank.clamp(0, len(free) - 1)], rows)
    old, new = page[copied], fresh.gather(1, first[:, None].clamp_max(rows.shape[1] - 1))[:, 0][copied]
    s["kv"][:, :, new] = s["kv"][:, :, old]
    s["refs"].index_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    s["refs"][fresh[take]] = 1
    s["table"][seqs] = fresh.to(torch.int32)


def _plain_compact(s, seqs, n_keep, keep):
    ps, seqs = s["kv"].shape[4], seqs.long()
    length = s["lengths"][seqs].long()
    j = torch.arange(keep.shape[1], device=_DEV)[None]
    live = j < n_keep.long()[:, None]
    a, b = (length[:, None] + keep.long())[live], (length[:, None] + j)[live]
    row = seqs[:, None].expand(live.shape)[live]
    table = s["table"].long()
    s["kv"][:, :, table[row, b // ps], :, b % ps] = s["kv"][:, :, table[row, a // ps], :, a % ps]
    s["lengths"][seqs] += n_keep


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import tile_synchronised_b200 as mk
        cache = s["cache"]
        if op == "tree":
            return mk.attention_tree(s["q"], cache, 0, s["seqs"], n_new=s["n_new"], mask=s["mask"], out=s["out"])
        if op == "rope":
            q = mk.qk_norm_rope(s["qkv"], cache, 0, s["seqs"], s["case"]["nq"], s["case"]["theta"],
                                q_gain=s["q_gain"], k_gain=s["k_gain"], eps=1e-6, n_new=s["n_new"], depth=s["depth"],
                                out=s["q"])
            return q, s["kv"]
        if op == "fork":
            cache.free(s["dst"])
            cache.fork(s["src"], s["dst"])
            cache.reserve(s["dst"], s["counts"])
        else:
            cache.free(s["seqs"], s["base"])
            cache.reserve(s["seqs"], s["counts"])
            cache.copy(s["src_pages"], s["dst_pages"], source=s["drafts"])
            cache.compact(s["seqs"], s["n_keep"], s["keep"])
        return s["kv"], s["table"], s["lengths"], s["refs"]
    if op == "tree":
        return _plain_tree(s)
    if op == "rope":
        return _plain_rope(s)
    if op == "fork":
        _plain_free(s, s["dst"], torch.zeros_like(s["dst"]))
        _plain_fork(s, s["src"], s["dst"])
        _plain_reserve(s, s["dst"], s["counts"])
    else:
        _plain_free(s, s["seqs"], s["base"])
        _plain_reserve(s, s["seqs"], s["counts"])
        s["kv"][:, :, s["dst_pages"].long()] = s["stage"][:, :, s["src_pages"].long()]
        _plain_compact(s, s["seqs"], s["n_keep"], s["keep"])
    return s["kv"], s["table"], s["lengths"], s["refs"]


def work(case):
    """Bytes and operations of one pass at the mean of the case's lengths."""
    n, T, nkv, d, ps = case["n"], case["T"], case["nkv"], case["d"], case["page"]
    length = (case["lo"] + case["hi"]) / 2
    new = ((T + 1) // 2 + T) / 2
    if case["op"] == "tree":
        nq = case["nq"]
        per = new / 2 if case["mask"] == "none" else min(new, 2 * math.log(new + 1) + 1)
        mask = 0 if case["mask"] == "none" else n * new * ((T + 31) // 32) * 4
        return {"bytes": n * (length + new) * nkv * d * 4 + n * new * nq * d * 4 + mask,
                "flops": 4.0 * n * new * nq * d * (length + per)}
    if case["op"] == "rope":
        nq = case["nq"]
        wide = 4 if case["src"] == "fp32" else 2
        values = n * new * (nq + 2 * nkv) * d
        return {"bytes": values * (wide + 2), "flops": values * (9.0 if case["norm"] else 4.0)}
    each = 2.0 * case["layers"] * nkv * d * 2  # bytes of one position
    if case["op"] == "fork":
        # one last page of each fork read and written (a length that ends a page has none)
        return {"bytes": 2 * n * case["beams"] * each * ps * (ps - 1) / ps + n * (1 + case["beams"]) * 4 * length / ps,
                "flops": 0.0}
    pages = (T + ps - 1) / ps + 0.5
    return {"bytes": 2 * n * each * (pages * ps + (T + 1) / 2), "flops": 0.0}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, n, T, ps = case["op"], case["n"], case["T"], case["page"]
    if op in ("tree", "rope"):
        kv, table = s["kv"], s["table"].cpu()
        seqs, lens, new = s["seqs"].tolist(), s["lengths"].tolist(), s["n_new"].tolist()
    if op == "tree":
        out = s["out"].double()
        for i in range(n):
            L, m = lens[seqs[i]], new[i]
            rows = table[seqs[i]][:(L + m + ps - 1) // ps].long().to(_DEV)
            allowed = torch.zeros((m, L + m), dtype=torch.bool)
            allowed[:, :L] = True
            if s["mask"] is None:
                allowed[:, L:] = torch.ones((m, m), dtype=torch.bool).tril()
            else:
                words = s["mask"][i].cpu().long() & 0xFFFFFFFF
                for u in range(m):
                    allowed[:, L + u] = (words[:m, u // 32] >> (u % 32)) & 1 == 1
            allowed = allowed.to(_DEV)
            for g in range(case["nkv"]):
                K, V = (kv[h, 0, rows, g].reshape(-1, case["d"])[:L + m].double() for h in (0, 1))
                G = case["nq"] // case["nkv"]
                Q = s["q"][i, :m, g * G:(g + 1) * G].double()
                w = torch.einsum("tgd,sd->gts", Q, K) / case["d"] ** 0.5
                w = torch.softmax(w.masked_fill(~allowed, float("-inf")), -1)
                w = torch.where(allowed.any(1)[None, :, None], w, torch.zeros_like(w))
                out[i, :m, g * G:(g + 1) * G] = torch.einsum("gts,sd->tgd", w, V)
        return out
    if op == "rope":
        q, pages = s["q"].double(), s["kv"].double()
        nq, nkv, d = case["nq"], case["nkv"], case["d"]
        freq = torch.tensor([case["theta"] ** (-2 * i / d) for i in range(d // 2)], dtype=torch.float64, device=_DEV)
        for i in range(n):
            L, m = lens[seqs[i]], new[i]
            x = s["qkv"][i, :m].double().view(m, nq + 2 * nkv, d)
            pos = L + (torch.arange(m, device=_DEV) if s["depth"] is None else s["depth"][i, :m])
            turn = torch.polar(torch.ones((), dtype=torch.float64, device=_DEV), pos.double()[:, None] * freq)[:, None]
            heads = []
            for a, b, gain in ((0, nq, s["q_gain"]), (nq, nq + nkv, s["k_gain"])):
                h = x[:, a:b]
                if gain is not None:
                    h = h / ((h ** 2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * gain.double()
                z = torch.complex(h[..., :d // 2].contiguous(), h[..., d // 2:].contiguous()) * turn
                heads.append(torch.cat([z.real, z.imag], -1))
            q[i, :m] = heads[0]
            for t in range(m):
                p, o = int(table[seqs[i], (L + t) // ps]), (L + t) % ps
                pages[0, 0, p, :, o] = heads[1][t]
                pages[1, 0, p, :, o] = x[t, nq + nkv:]
        return q, pages
    return None  # pages: moved, not computed
