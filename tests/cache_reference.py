"""The key/value cache operators in 64 bits, one sequence and head at a time, from their
definitions (include/ab_attn.h), on host tensors; and the error bounds of the kernels."""

import math

import torch

F64 = torch.float64


class HostCache:
    """A paged cache on the host; to_gpu() gives the KVCache of the same contents."""

    def __init__(self, lengths, Hk, d, page, dtype, spare=0, max_pages=None, seed=0, layout="hpd", scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.g, self.Hk, self.d, self.page, self.dtype, self.layout = g, Hk, d, page, dtype, layout
        self.B = len(lengths)
        need = [-(-n // page) for n in lengths]
        self.max_pages = max_pages if max_pages is not None else max(max(need), 1) + 1
        n_pages = sum(need) + spare + 1
        self.n_pages = n_pages
        self.k = (torch.randn(n_pages, Hk, page, d, generator=g) * scale).to(dtype)
        self.v = torch.randn(n_pages, Hk, page, d, generator=g).to(dtype)
        self.mass = torch.rand(n_pages, Hk, page, generator=g)
        self.pos = torch.zeros(n_pages, Hk, page, dtype=torch.int32)
        self.ksum = torch.randn(n_pages, Hk, d, generator=g) * page / 2
        order = torch.randperm(n_pages, generator=g).tolist()
        self.free = order[sum(need):]
        self.table = torch.full((self.B, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = order[at]
                at += 1
        self.length = torch.tensor(lengths, dtype=torch.int32)

    def allocate(self, b, slots):
        """Give sequence b pages for `slots` slots."""
        for i in range(-(-slots // self.page)):
            if self.table[b, i] < 0:
                self.table[b, i] = self.free.pop()

    def randn(self, *shape, scale=1.0, dtype=None):
        return (torch.randn(*shape, generator=self.g) * scale).to(dtype or self.dtype)

    def slots(self, name, b, h, n):
        """Rows 0 .. n - 1 of sequence b, head h."""
        p = self.table[b, : -(-n // self.page)].long()
        x = getattr(self, name)[p, h]
        return x.reshape(p.numel() * self.page, *x.shape[2:])[:n]

    def to_gpu(self, device="cuda"):
        import block_sparse_attention_ab_b200 as ab

        def pages(t):
            if self.layout == "hpd":
                return t.to(device)
            # [n_pages, page, Hk, d] storage with padded rows
            buf = torch.zeros(self.n_pages, self.page, self.Hk, self.d + 8, dtype=t.dtype, device=device)
            view = buf[..., : self.d].permute(0, 2, 1, 3)
            view.copy_(t.to(device))
            return view

        return ab.KVCache(k=pages(self.k), v=pages(self.v), table=self.table.to(device),
                          length=self.length.to(device), ksum=self.ksum.to(device),
                          mass=self.mass.to(device), pos=self.pos.to(device))


def logit_error(q, k, scale=None):
    """Bound of a logit's absolute error: d products of 16-bit values are exact in fp32, their
    sum is off by at most 2 d half-steps of fp32 relative to the sum of magnitudes (twice: the
    tensor core may truncate), and scaling adds two roundings."""
    d = q.shape[-1]
    mag = (q.abs().to(F64) @ k.abs().to(F64).T).max() if k.numel() and q.numel() else torch.tensor(0.0)
    return float(mag) / math.sqrt(d) * (2 * d + 2) * 2.0 ** -24


def attn(c, q, k=None, v=None, n_tok=None, tree=None, plan=None, per_token=False):
    """(out, lse, bound of |out error| before the output's rounding, bound of |lse error|)."""
    B, Hq, T, d = q.shape
    G = Hq // c.Hk
    out = torch.zeros(B, Hq, T, d, dtype=F64)
    lse = torch.zeros(B, Hq, T, dtype=F64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    u = torch.finfo(c.dtype).eps / 2
    for b in range(B):
        n = T if n_tok is None else int(n_tok[b])
        L = int(c.length[b])
        for h in range(c.Hk):
            kc, vc = c.slots("k", b, h, L), c.slots("v", b, h, L)
            for t in range(n):
                shift = torch.zeros(L, dtype=F64)
                if plan is not None:
                    idx, cnt, w = plan
                    row = t if per_token else 0
                    shift[:] = -math.inf
                    for e in range(int(cnt[b, h, row])):
                        p = int(idx[b, h, row, e])
                        shift[p * c.page : min(L, (p + 1) * c.page)] = \
                            0.0 if w is None else math.log(float(w[b, h, row, e]))
                keys, vals = kc[shift > -math.inf], vc[shift > -math.inf]
                shift = shift[shift > -math.inf]
                if k is not None:
                    js = [j for j in range(n) if (bool(tree[b, t, j]) if tree is not None else j <= t)]
                    keys = torch.cat([keys, k[b, h, js]])
                    vals = torch.cat([vals, v[b, h, js]])
                    shift = torch.cat([shift, torch.zeros(len(js), dtype=F64)])
                rows = q[b, h * G : (h + 1) * G, t]
                if keys.shape[0] == 0:
                    lse[b, h * G : (h + 1) * G, t] = -math.inf
                    continue
                s = rows.to(F64) @ keys.to(F64).T / math.sqrt(d) + shift
                p = torch.softmax(s, dim=-1)
                out[b, h * G : (h + 1) * G, t] = p @ vals.to(F64)
                lse[b, h * G : (h + 1) * G, t] = torch.logsumexp(s, dim=-1)
                # p is rounded to the type (u) and carries the logit's error and that of a
                # base-2 exponential (2^-21), in numerator and denominator
                e = logit_error(rows, keys) + 2.0 ** -22 * float(s.abs().max()) + 2.0 ** -21
                tol[b, h * G : (h + 1) * G, t] = (u + 4 * e) * (p @ vals.to(F64).abs())
                tol_lse[b, h * G : (h + 1) * G, t] = 2 * e + 2.0 ** -21
    return out, lse, tol, tol_lse


def score(c, q, n_tok=None, per_token=True, first=0, recent=0):
    """(scores, bound of their relative error)."""
    B, Hq, T, d = q.shape
    G = Hq // c.Hk
    Tp = T if per_token else 1
    out = torch.zeros(B, c.Hk, Tp, c.max_pages, dtype=F64)
    worst = 0.0
    for b in range(B):
        n = T if n_tok is None else int(n_tok[b])
        L = int(c.length[b])
        P = -(-L // c.page)
        if P == 0 or n == 0:
            continue
        size = torch.tensor([min(c.page, L - p * c.page) for p in range(P)], dtype=F64).unsqueeze(1)
        for h in range(c.Hk):
            mean = c.ksum[c.table[b, :P].long(), h].to(F64) / size
            for t in range(n):
                rows = q[b, h * G : (h + 1) * G, t]
                s = rows.to(F64) @ mean.T / math.sqrt(d)
                worst = max(worst, logit_error(rows, mean) + 2.0 ** -22 * float(s.abs().max()))
                share = torch.softmax(s, dim=-1).mean(dim=0)
                if per_token:
                    out[b, h, t, :P] = share
                else:
                    out[b, h, 0, :P] += share / n
        live = n if per_token else 1
        for p in range(P):
            if p < first or p >= P - recent:
                out[b, :, :live, p] = 2.0
    return out, 4 * worst + 2.0 ** -18


def mass(c, q, lse, n_tok=None, sel=None, plan=None, per_token=False):
    """(mass like c.mass, bound of its absolute error)."""
    B, Hq, T, d = q.shape
    G = Hq // c.Hk
    out = c.mass.to(F64).clone()
    tol = torch.zeros_like(out)
    for b in range(B):
        L = int(c.length[b])
        n = min(T if n_tok is None else int(n_tok[b]), L)
        for h in range(c.Hk):
            keys = c.slots("k", b, h, L)
            got, err = torch.zeros(L, dtype=F64), torch.zeros(L, dtype=F64)
            for i in range(n):
                t = i if sel is None else int(sel[b, i])
                shift = torch.zeros(L, dtype=F64)
                if plan is not None:
                    idx, cnt, w = plan
                    row = t if per_token else 0
                    shift[: L - n] = -math.inf
                    for e in range(int(cnt[b, h, row])):
                        p = int(idx[b, h, row, e])
                        shift[p * c.page : max(p * c.page, min(L - n, (p + 1) * c.page))] = \
                            0.0 if w is None else math.log(float(w[b, h, row, e]))
                shift[L - n + i + 1 :] = -math.inf
                rows = q[b, h * G : (h + 1) * G, t]
                s = rows.to(F64) @ keys.to(F64).T / math.sqrt(d) + shift
                l = lse[b, h * G : (h + 1) * G, t].to(F64).unsqueeze(-1)
                p = torch.where(l == -math.inf, 0.0, torch.exp(s - l)).sum(dim=0)
                got += p
                span = torch.where(s == -math.inf, 0.0, s).abs().max() + l[l > -math.inf].abs().max() \
                    if bool((l > -math.inf).any()) else 0.0
                err += p * (2 * logit_error(rows, keys) + 2.0 ** -20 * (1 + float(span)))
            pg = c.table[b, torch.arange(L) // c.page].long()
            off = torch.arange(L) % c.page
            out[pg, h, off] += got
            # sums over the rows and the addition to the old mass, in fp32
            tol[pg, h, off] = err + (n * G + 2) * 2.0 ** -24 * out[pg, h, off].abs()
    return out, tol


def keep(c, budget, recent=0, next_pos=None, score=None):
    """(src, n_keep)."""
    x = c.mass if score is None else score
    src = torch.full((c.B, c.Hk, budget), -1, dtype=torch.int32)
    count = torch.zeros(c.B, dtype=torch.int32)
    for b in range(c.B):
        L = int(c.length[b])
        m = min(L, budget)
        count[b] = m
        for h in range(c.Hk):
            old = c.mass
            c.mass = x
            val = c.slots("mass", b, h, L).clone()
            c.mass = old
            if recent > 0:
                val[c.slots("pos", b, h, L) >= int(next_pos[b]) - recent] = math.inf
            order = sorted(range(L), key=lambda s: (-float(val[s]), s))
            kept = sorted(order[:m])
            stay = set(s for s in kept if s < m)
            movers = iter(s for s in kept if s >= m)
            for j in range(m):
                src[b, h, j] = j if j in stay else next(movers)
    return src, count


def compact(c, src, count):
    """Moves slots of the host cache; returns the set of (page, head) whose sum is due."""
    due = set()
    for b in range(c.B):
        m = int(count[b])
        for h in range(c.Hk):
            for j in range(m):
                s = int(src[b, h, j])
                if s != j:
                    to = (int(c.table[b, j // c.page]), h, j % c.page)
                    frm = (int(c.table[b, s // c.page]), h, s % c.page)
                    for name in ("k", "v", "mass", "pos"):
                        t = getattr(c, name)
                        t[to] = t[frm].clone()
                    due.add((to[0], h, min(c.page, m - j // c.page * c.page)))
            if m % c.page:
                due.add((int(c.table[b, m // c.page]), h, m % c.page))
        c.length[b] = m
    return due
