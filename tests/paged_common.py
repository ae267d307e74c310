"""Plain 64-bit implementations of the paged-cache operators, and inputs for
their tests.  Everything here is torch / Python on the CPU."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


def generator(seed):
    return torch.Generator().manual_seed(seed)


class Pool:
    """The plain model of a paged cache: the rules of reserve, fork, compact,
    free and copy, one entry after another, on CPU tensors."""

    def __init__(self, layers, nkv, d, ps, n_pages, seqs, width, dtype=torch.bfloat16, seed=0):
        g = generator(seed)
        self.kv = torch.randn((2, layers, n_pages, nkv, ps, d), generator=g).to(dtype)
        self.table = torch.full((seqs, width), -1, dtype=torch.int32)
        self.lengths = torch.zeros(seqs, dtype=torch.int32)
        self.refs = torch.zeros(n_pages, dtype=torch.int32)
        self.ps = ps

    def clone(self):
        o = object.__new__(Pool)
        o.kv, o.table, o.lengths, o.refs = (x.clone() for x in (self.kv, self.table, self.lengths, self.refs))
        o.ps = self.ps
        return o

    def pages(self, positions):
        return -(-positions // self.ps)

    def reserve(self, seqs, counts):
        take, seen, refs = [], {}, self.refs.clone()
        for s, c in zip(seqs, counts):
            L = int(self.lengths[s])
            first, last = L // self.ps, self.pages(L + c) if c else 0
            for j in range(first, last):
                page = int(self.table[s, j])
                if page < 0:
                    take.append((s, j, None))
                elif j == first and L % self.ps and int(refs[page]) > 1:
                    refs[page] -= 1
                    take.append((s, j, page))
        free = [p for p in range(len(self.refs)) if int(self.refs[p]) == 0]
        if len(free) < len(take):
            return False
        for p, (s, j, old) in zip(free, take):
            if old is not None:
                self.kv[:, :, p] = self.kv[:, :, old]
                self.refs[old] -= 1
            self.refs[p] = 1
            self.table[s, j] = p
        return True

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            k = self.pages(int(self.lengths[a]))
            self.table[b, :k] = self.table[a, :k]
            self.refs.index_add_(0, self.table[a, :k].long(), torch.ones(k, dtype=torch.int32))
            self.lengths[b] = self.lengths[a]

    def free(self, seqs, lengths=None):
        for i, s in enumerate(seqs):
            L = 0 if lengths is None else lengths[i]
            for j in range(self.pages(L), self.table.shape[1]):
                if int(self.table[s, j]) >= 0:
                    self.refs[int(self.table[s, j])] -= 1
                    self.table[s, j] = -1
            self.lengths[s] = L

    def at(self, s, pos):
        return int(self.table[s, pos // self.ps]), pos % self.ps

    def compact(self, seqs, keep):
        for s, ks in zip(seqs, keep):
            L = int(self.lengths[s])
            for j, k in enumerate(ks):
                (a, x), (b, y) = self.at(s, L + k), self.at(s, L + j)
                self.kv[:, :, b, :, y] = self.kv[:, :, a, :, x]
            self.lengths[s] += len(ks)

    def rows(self, kv, layer, s, n):
        """Positions 0 .. n - 1 of K (0) or V (1): [nkv, n, d]."""
        pages = self.table[s, :self.pages(n)].long()
        return self.kv[kv, layer][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :n]

    def to_cache(self, device="cuda"):
        import tile_synchronised_b200 as mk
        return mk.PagedCache.over(*(x.clone().to(device) for x in (self.kv, self.table, self.lengths, self.refs)))

    def same_as(self, cache, kv=True):
        assert torch.equal(self.table, cache.table.cpu())
        assert torch.equal(self.lengths, cache.lengths.cpu())
        assert torch.equal(self.refs, cache.refs.cpu())
        if kv:  # bit for bit (NaN included)
            assert torch.equal(self.kv.view(torch.int16), cache.kv.cpu().view(torch.int16))


def filled(lengths, room, layers=1, nkv=2, d=64, ps=16, dtype=torch.bfloat16, seed=0, spare=3, extra=0, poison=True):
    """A pool whose sequence i holds lengths[i] positions and room[i] reserved
    ones on scattered pages; with `poison`, every slot that holds no position
    is NaN."""
    need = [-(-(a + b) // ps) for a, b in zip(lengths, room)]
    total = sum(need) + spare
    p = Pool(layers, nkv, d, ps, max(total, 1), len(lengths) + extra, max(max(need), 1), dtype, seed)
    order = torch.randperm(max(total, 1), generator=generator(seed + 1)).to(torch.int32)
    at = 0
    for i, k in enumerate(need):
        p.table[i, :k] = order[at:at + k]
        p.refs[order[at:at + k].long()] = 1
        p.lengths[i] = lengths[i]
        at += k
    if poison:
        live = torch.zeros((p.kv.shape[2], ps), dtype=torch.bool)
        for i, k in enumerate(lengths):
            for j in range(k + room[i]):
                live[p.at(i, j)] = True
        p.kv.permute(2, 4, 0, 1, 3, 5)[~live] = float("nan")
    return p


def random_tree(T, seed):
    g = generator(seed)
    return [-1 if t == 0 else int(torch.randint(-1, t, (1,), generator=g)) for t in range(T)]


def visible(parents):
    """Ancestor-or-self matrix [T, T] of a tree."""
    T = len(parents)
    seen = torch.zeros((T, T), dtype=torch.bool)
    for t in range(T):
        k = t
        while k >= 0:
            seen[t, k] = True
            k = parents[k]
    return seen


def pack_bits(seen):
    """[..., T, T] booleans as int32 words [..., T, (T + 31) // 32]."""
    T = seen.shape[-1]
    words = (T + 31) // 32
    bits = torch.zeros((*seen.shape[:-1], words * 32), dtype=torch.int64)
    bits[..., :T] = seen.long()
    w = (bits.view(*seen.shape[:-1], words, 32) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def tree_reference(pool, layer, q, seqs, n_new, seen, out):
    """64-bit attention of the new tokens: (out with its live rows replaced,
    the error a correct kernel may have).  seen [n, T, T] or None (causal).

    The bound: the result is rounded to 16 bits once (half a step of it), each
    weight once (half a step of w_j, times |V_j|), and scores carry 32-bit
    error: a dot product of d terms is within (d + 2) 2^-23 sum |q k| / sqrt d
    of its value, the exponent's argument within another 2^-22 of its size, the
    exponential 2^-21.  Weights below half precision's smallest step (2^-24, the
    largest weight being 2^7) add 2^-31 each."""
    dtype = q.dtype
    n, T, nq, d = q.shape
    nkv = pool.kv.shape[3]
    G = nq // nkv
    ref, bound = out.double().clone(), torch.zeros(out.shape, dtype=torch.float64)
    for i in range(n):
        L, m = int(pool.lengths[seqs[i]]), n_new[i]
        if m == 0:
            continue
        K, V = (pool.rows(x, layer, seqs[i], L + m).double() for x in (0, 1))
        see = torch.ones((m, L + m), dtype=torch.bool)
        see[:, L:] = torch.ones((m, m)).tril().bool() if seen is None else seen[i][:m, :m]
        for h in range(nq):
            Q = q[i, :m, h].double()
            k, v = K[h // G], V[h // G]
            s = Q @ k.T / math.sqrt(d)
            size = torch.where(see, Q.abs() @ k.abs().T / math.sqrt(d), 0.0)
            s = torch.where(see, s, float("-inf"))
            top = s.amax(1, keepdim=True)
            w = torch.exp(s - torch.where(torch.isinf(top) & (top < 0), 0.0, top))
            w = torch.where(see, w, 0.0)
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
            # 0 x inf at unseen positions is nothing
            fin = torch.isfinite(v)
            o = w @ torch.where(fin, v, 0.0)
            bad = see.double() @ (~fin).double() > 0
            o = torch.where(bad, float("nan"), o)
            ref[i, :m, h] = o
            exp_err = 2 * ((d + 2) * 2.0 ** -23 * size.amax(1) + 2.0 ** -22 * torch.where(see, s.abs(), 0.0).amax(1)
                           + 2.0 ** -21)
            mass = w @ torch.where(fin, v, 0.0).abs()
            bound[i, :m, h] = (EPS[dtype] * o.abs() + (EPS[dtype] + exp_err[:, None]) * mass
                               + (L + m) * 2.0 ** -31 * torch.where(fin, v, 0.0).abs().amax() + 1e-30)
    return ref, bound


def rope_reference(pool, layer, qkv, nq, theta, q_gain, k_gain, eps, seqs, n_new, depth, q):
    """64-bit q (live rows replaced) and the K/V of the new tokens, with the
    error a correct kernel may have: {"q": (ref, bound), (i, t): (k, v, bound_k)}.

    The bound: one rounding to 16 bits; the norm's 32-bit sum of d squares and
    the products within (d / 2 + 8) 2^-24 of each factor; the angle, reduced in
    64 bits, is rounded to 32 bits in turns (2^-25 of half a turn, 2^-23 in
    radians) and its sine and cosine are within 2^-22 of their values."""
    n, T = qkv.shape[:2]
    nkv, d = pool.kv.shape[3], pool.kv.shape[5]
    dtype = pool.kv.dtype
    x = qkv.double().view(n, T, nq + 2 * nkv, d)
    freq = torch.tensor([theta ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64)
    ref, bound, kv = q.double().clone(), torch.zeros(q.shape, dtype=torch.float64), {}
    rel = (d / 2 + 8) * 2.0 ** -24
    for i in range(n):
        for t in range(n_new[i]):
            pos = int(pool.lengths[seqs[i]]) + (t if depth is None else int(depth[i, t]))
            c, s = torch.cos(pos * freq), torch.sin(pos * freq)
            out = []
            for h, gain in ((x[i, t, :nq], q_gain), (x[i, t, nq:nq + nkv], k_gain)):
                if gain is not None:
                    h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * gain.double()
                a, b = h[:, :d // 2], h[:, d // 2:]
                r = torch.cat([a * c - b * s, b * c + a * s], -1)
                size = a.abs() + b.abs()
                out.append((r, EPS[dtype] * r.abs() + (rel + 2.0 ** -21) * torch.cat([size, size], -1)
                            + (2.0 ** -25 if dtype == torch.float16 else 0) + 1e-30))
            ref[i, t], bound[i, t] = out[0]
            kv[i, t] = (out[1][0], x[i, t, nq + nkv:], out[1][1])
    return ref, bound, kv
